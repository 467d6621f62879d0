"""The operators around the scan on the GPU, through the C ABI and the binding: forms that the
wider tests do not reach."""

import ctypes

import numpy as np
import pytest

import layer_ref as ref
from test_layer_ops_gpu import _dev, _strided, ssd  # noqa: F401  (ssd is the built package)

pytestmark = pytest.mark.gpu


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# rows and widths that take each way a row comes in: bulk copies, single vectors, pairs, elements
@pytest.mark.parametrize("R,D", [(37, 2560), (300, 512), (9, 64), (21, 34), (50, 97)])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_without_d_residual(ssd, R, D, with_dh, kind):  # noqa: F811
    """ssd_norm_backward with bf16 rows, a float32 h and no d_residual (the final norm of a network
    has neither the stream's gradient nor a use for its own): dx, d_weight and d_bias are those of
    the call that asks for it, and right."""
    import torch
    from state_space_model_ssd_gb300 import _lib
    rng = np.random.default_rng(R + D)
    dy, dy64 = _dev(rng.standard_normal((R, D)), "bf16")
    h, h64 = _dev(rng.standard_normal((R, D)) + 0.5, "f32")
    dh, dh64 = _dev(rng.standard_normal((R, D)), "f32") if with_dh else (None, None)
    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    layer = kind == "layer"
    _, _, st = ref.norm(h64, w64, None, None, 1e-5, layer)
    stats = torch.from_numpy(st.astype(np.float32)).cuda()
    p = _lib.NormProblem(R, D, D, D, D, D, 0 if layer else 1, 1, 0, 0, 1e-5)
    n = ctypes.c_size_t()
    assert _lib.lib().ssd_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")

    def call(dres):
        dx, dw, db = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
        assert _lib.lib().ssd_norm_backward(
            ctypes.byref(p), _p(dy), _p(h), _p(dh), _p(w), _p(stats), _p(dx), _p(dres), _p(dw), _p(db), _p(ws),
            n.value, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        return dx, dw, db

    dres = torch.empty_like(h)
    without, full = call(None), call(dres)
    for a, b in zip(without, full):
        assert bool((a == b).all())
    dv, dw, db = ref.norm_bwd(dy64, h64, w64, stats.double().cpu().numpy(), dh64, layer)
    ref.assert_close(without[0], dv, "bf16", "dx")
    ref.assert_close(dres, dv, "f32", "d_residual")
    ref.assert_close(without[1], dw, "f32", "d_weight")
    ref.assert_close(without[2], db, "f32", "d_bias")
    # the binding's form of it
    g = ssd.norm_backward(dy, h, w, stats, dh=dh, kind=kind)
    assert bool((g["dx"] == full[0]).all()) and bool((g["d_residual"] == dres).all())


# dy, h: their types
@pytest.mark.parametrize("dt,ht", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("R,D", [(40, 768), (21, 34), (50, 97)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_backward_writes_what_out_brings(ssd, dt, ht, R, D, with_dh):  # noqa: F811
    """Every buffer in ``out`` gets the call's result, also d_residual in the type of dx and d_bias
    without ``bias``; the dict of an earlier call serves again."""
    import torch
    rng = np.random.default_rng(R * D)
    dy, dy64 = _dev(rng.standard_normal((R, D)), dt)
    h, h64 = _dev(rng.standard_normal((R, D)), ht)
    dh, dh64 = _dev(rng.standard_normal((R, D)), ht) if with_dh else (None, None)
    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    _, _, st = ref.norm(h64, w64, None, None, 1e-5, True)
    stats = torch.from_numpy(st.astype(np.float32)).cuda()
    dv, dw, db = ref.norm_bwd(dy64, h64, w64, stats.double().cpu().numpy(), dh64, True)
    out = {"dx": torch.full_like(dy, float("nan")), "d_residual": torch.full_like(h, float("nan")),
           "d_weight": torch.full_like(w, float("nan")), "d_bias": torch.full_like(w, float("nan"))}
    mine = dict(out)
    g = ssd.norm_backward(dy, h, w, stats, dh=dh, bias=False, out=out)
    assert set(g) == set(mine) and all(g[k] is mine[k] for k in mine)
    ref.assert_close(g["dx"], dv, dt, "dx")
    ref.assert_close(g["d_residual"], dv, ht, "d_residual")
    ref.assert_close(g["d_weight"], dw, "f32", "d_weight")
    ref.assert_close(g["d_bias"], db, "f32", "d_bias")
    # without buffers: the same bits, and only what was asked for
    f = ssd.norm_backward(dy, h, w, stats, dh=dh, bias=False)
    assert "d_bias" not in f and ("d_residual" in f) == (with_dh or dt != ht)
    assert all(bool((f[k] == g[k]).all()) for k in f)
    # the dict of an earlier call
    for t in f.values():
        t.fill_(float("nan"))
    before = dict(f)
    f2 = ssd.norm_backward(dy, h, w, stats, dh=dh, bias=False, out=f)
    assert all(f2[k] is before[k] and bool((f2[k] == g[k]).all()) for k in before)
    if dt == ht:  # one buffer for both, under two tensors
        one = torch.full_like(dy, float("nan"))
        f3 = ssd.norm_backward(dy, h, w, stats, dh=dh, out={"dx": one, "d_residual": one[:]})
        assert bool((one == g["dx"]).all()) and bool((f3["d_residual"] == g["dx"]).all())
    with pytest.raises(ValueError):
        ssd.norm_backward(dy, h, w, stats, dh=dh, out={"d_residual": torch.empty(R, D + 1, dtype=h.dtype,
                                                                               device="cuda")})


def test_conv_backward_writes_what_out_brings(ssd):  # noqa: F811
    """d_initial_state in ``out`` is written without being asked for; d_bias without a bias, which
    has no meaning, is refused."""
    import torch
    rng = np.random.default_rng(4)
    u, _ = _dev(rng.standard_normal((2, 30, 24)), "bf16")
    w, _ = _dev(rng.standard_normal((24, 4)), "f32")
    init, _ = _dev(rng.standard_normal((2, 4, 24)), "bf16")
    want = ssd.conv_backward(u, w, None, u, initial_state=init, d_initial_state=True)
    buf = torch.full_like(init, float("nan"))
    g = ssd.conv_backward(u, w, None, u, initial_state=init, out={"d_initial_state": buf})
    assert g["d_initial_state"] is buf
    assert set(g) == set(want) and all(bool((g[k] == want[k]).all()) for k in want)
    with pytest.raises(ValueError):
        ssd.conv_backward(u, w, None, u, out={"d_bias": torch.empty(24, device="cuda")})


# silu'(v) = s + v s (1 - s) where s is 1 to the last bit: 1, however large v is.  Each row or
# sequence has gates of one size, so that a tolerance of its own largest value judges it.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gated_backward_at_large_gates(ssd, dt):  # noqa: F811
    import torch
    rng = np.random.default_rng(31)
    scales = np.array([1e-3, 1.0, 9.0, 14.0, 30.0, 1e4, 2.0 ** 24, 3e7, 1e9, 1e12])
    R, D = len(scales), 64
    z, z64 = _dev(scales[:, None] * rng.uniform(0.5, 1.5, (R, D)), dt)
    y, y64 = _dev(rng.standard_normal((R, D)), dt)
    dout, dout64 = _dev(rng.standard_normal((R, D)), dt)
    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    _, rstd = ssd.gated_norm_forward(y, z, w)
    _, wr = ref.gated(y64, z64, w64, 1e-5, 1)
    assert np.abs(rstd.double().cpu().numpy() / wr - 1).max() <= ref.CHAIN
    # a gradient that survives the norm's own factor 1 / (y z): that of a unit rstd
    one = torch.ones_like(rstd)
    for r in (rstd, one):
        g = ssd.gated_norm_backward(dout, y, z, w, r)
        # a - xh mean(a xh) of the formula, with xh = y z rstd: finite for either rstd
        dy, dz, _ = ref.gated_bwd(dout64, y64, z64, w64, r.double().cpu().numpy(), 1)
        for i in range(R):
            ref.assert_close(g["dy"][i], dy[i], dt, "dy at gates of %g" % scales[i])
            ref.assert_close(g["dz"][i], dz[i], dt, "dz at gates of %g" % scales[i])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_conv_backward_at_large_inputs(ssd, dt):  # noqa: F811
    import torch
    rng = np.random.default_rng(32)
    L, C, K = 48, 16, 4
    w, w64 = _dev(rng.uniform(0.5, 1.0, (C, K)), "f32")
    b, b64 = _dev(rng.standard_normal(C), "f32")
    # runs of one sign: a sum that crosses zero between them takes a large step over it
    sign = np.repeat([1.0, -1.0, 1.0], L // 3)
    for scale in (9.0, 30.0, 1e4, 2.0 ** 24, 3e7, 1e12):
        u, u64 = _dev(sign[None, :, None] * scale * rng.uniform(0.5, 1.5, (1, L, C)), dt)
        init, init64 = _dev(scale * rng.uniform(0.5, 1.5, (1, K, C)), dt)
        dy, dy64 = _dev(rng.standard_normal((1, L, C)), dt)
        pos = torch.tensor([6], dtype=torch.int32, device="cuda")
        g = ssd.conv_backward(u, w, b, dy, initial_state=init, positions=pos, d_initial_state=True)
        with np.errstate(over="ignore"):
            du, dw, db, d0 = ref.conv_bwd(u64[0], w64, b64, dy64[0], 6, init64[0])
        ref.assert_close(g["du"], du[None], dt, "du at %g" % scale)
        ref.assert_close(g["d_weight"], dw, "f32", "d_weight at %g" % scale)
        ref.assert_close(g["d_bias"], db, "f32", "d_bias at %g" % scale)
        ref.assert_close(g["d_initial_state"], d0[None], dt, "d_initial_state at %g" % scale)


def test_norm_forward_refuses_a_residual_out_without_a_residual(ssd):  # noqa: F811
    """h is x itself then: a buffer for it would be left unwritten."""
    import torch
    x, w = torch.randn(3, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        ssd.norm_forward(x, w, residual_out=torch.empty_like(x))


# Rows of one column.  rms: dx = rstd a (1 - xh^2) with xh^2 = 1 - eps rstd^2, layer: xh = 0 and
# dx = rstd (a - a): the terms cancel, so that the bound is the chain's roundings of the terms
# before they do, rstd max|a| with a = w dy (and of dh, which does not cancel).
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt,ht,with_dh", [("f32", "f32", False), ("f32", "f32", True), ("bf16", "f32", True),
                                           ("bf16", "bf16", False), ("bf16", "bf16", True)])
@pytest.mark.parametrize("R", [1, 300])
def test_norm_backward_of_one_column(ssd, R, kind, dt, ht, with_dh):  # noqa: F811
    import torch
    rng = np.random.default_rng(41)
    dy, dy64 = _dev(rng.standard_normal((R, 1)), dt)
    h, h64 = _dev(2 + rng.random((R, 1)), ht)
    dh, dh64 = _dev(rng.standard_normal((R, 1)), ht) if with_dh else (None, None)
    w, w64 = _dev([1.3], "f32")
    _, _, st = ref.norm(h64, w64, None, None, 1e-5, kind == "layer")
    stats = torch.from_numpy(st.astype(np.float32)).cuda()
    st = stats.double().cpu().numpy()
    g = ssd.norm_backward(dy, h, w, stats, dh=dh, kind=kind)
    dv, dw, db = ref.norm_bwd(dy64, h64, w64, st, dh64, kind == "layer")
    terms = np.abs(st[:, 1:] * w64 * dy64).max() + (np.abs(dh64).max() if with_dh else 0.0)
    for key, d in [("dx", dt)] + ([("d_residual", ht)] if "d_residual" in g else []):
        off = np.abs(g[key].double().cpu().numpy() - dv)
        assert (off <= ref.ROUND[d] * np.abs(dv) + ref.CHAIN * terms).all(), key
    # xh is 0 (layer) or 1 (rms), to a rounding or two
    ref.assert_close(g["d_weight"], dw, "f32", "d_weight")
    ref.assert_close(g["d_bias"], db, "f32", "d_bias")


@pytest.mark.parametrize("dt,wdt,has_b", [("bf16", "bf16", True), ("bf16", "bf16", False), ("f32", "bf16", False),
                                          ("bf16", "f32", False), ("f32", "f32", False)])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_step_parameters(ssd, dt, wdt, has_b, K):  # noqa: F811
    """The step's weights and bias in either type, and no bias: what the prompt's convolution and
    the formulas of the scan give."""
    import torch
    B, H, P, N, G = 5, 6, 16, 32, 2
    C = H * P + 2 * G * N
    rng = np.random.default_rng(42)
    st, st64 = _dev(rng.standard_normal((B, H, P, N)), "f32")
    win, win64 = _dev(rng.standard_normal((B, K, C)), dt)
    u, u64 = _dev(rng.standard_normal((B, C)), dt)
    w, w64 = _dev(rng.uniform(-1, 1, (C, K)), wdt)
    b, b64 = _dev(rng.uniform(-1, 1, C), wdt) if has_b else (None, np.zeros(C))
    raw = rng.standard_normal((B, H)).astype(np.float32)
    pos = rng.integers(0, 50, B)
    y = ssd.conv_decode_step(st, win, u, torch.from_numpy(raw).cuda(), w, b,
                             torch.from_numpy(pos.astype(np.int32)).cuda(), -4.6, ngroups=G)
    want = np.zeros((B, H, P))
    for i in range(B):
        o, s, _ = ref.conv(u64[i:i + 1], w64, b64, int(pos[i]), win64[i])
        win64[i, int(pos[i]) % K] = s[int(pos[i]) % K]
        x = o[0, :H * P].reshape(H, P)
        Bm, Cm = (np.repeat(o[0, H * P + k * G * N:H * P + (k + 1) * G * N].reshape(G, N), H // G, 0)
                  for k in (0, 1))
        delta = np.log1p(np.exp(raw[i].astype(np.float64) - 4.6))
        st64[i] = np.exp(-delta)[:, None, None] * st64[i] + (delta[:, None] * x)[..., None] * Bm[:, None]
        want[i] = np.einsum("hpn,hn->hp", st64[i], Cm)
    ref.assert_close(y, want, dt, "y")
    ref.assert_close(st, st64, "f32", "state")
    assert np.array_equal(win.double().cpu().numpy(), win64)


def test_every_operator_on_a_stream_of_its_own(ssd):  # noqa: F811
    """``stream=``: a chain of calls there, ordered behind a long copy by that stream alone, gives what
    the current stream gives."""
    import torch
    H, P, N, K, T = 8, 64, 64, 4, 3000
    C, D = H * P + 2 * N, H * P
    gen = torch.Generator(device="cuda").manual_seed(6)

    def rnd(*s, dt=torch.bfloat16):
        return torch.randn(*s, generator=gen, device="cuda").to(dt)

    src = rnd(1, T, C)
    w, b, gw = rnd(C, K, dt=torch.float32), rnd(C, dt=torch.float32), rnd(D, dt=torch.float32)
    z, tok, raw = rnd(1, T, D), rnd(3, C), rnd(3, H, dt=torch.float32)
    state, win = rnd(3, H, P, N, dt=torch.float32), rnd(3, K, C)
    pos = torch.tensor([4, 9, 2], dtype=torch.int32, device="cuda")
    big = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()

    def chain(u, s_, w_, stream):
        kw = {} if stream is None else {"stream": stream}
        o, f = ssd.conv_forward(u, w, b, split=((H, P), (1, N), (1, N)), final_state=True, **kw)
        y, r = ssd.gated_norm_forward(o[0], z, gw, **kw)
        gn = ssd.gated_norm_backward(y, o[0], z, gw, r, **kw)
        gc = ssd.conv_backward(u, w, b, (gn["dy"], o[1], o[2]), **kw)
        n, _, st = ssd.norm_forward(y, gw, **kw)
        nb = ssd.norm_backward(n, y, gw, st, **kw)
        t = ssd.conv_decode_step(s_, w_, tok, raw, w, b, pos, -4.6, **kw)
        return [*o, f, y, r, *gn.values(), *gc.values(), n, st, *nb.values(), t, s_, w_]

    want = chain(src, state.clone(), win.clone(), None)
    u = torch.zeros_like(src)
    s2, w2 = state.clone(), win.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # what the chain reads arrives late on its stream
        for _ in range(8):
            big.fill_(1.0)
        u.copy_(src)
    got = chain(u, s2, w2, s)
    s.synchronize()
    for x, y in zip(got, want):
        assert bool((x == y).all())


def test_norm_offsets_beyond_32_bits(ssd):  # noqa: F811
    """2,100,000 rows of 1152 columns, 2.4e9 elements a tensor: the last rows' gradients, and the sums
    over all rows, of which only the first and the last are not zero."""
    import torch
    R, D, G, n = 2_100_000, 1152, 2, 32
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    rng = np.random.default_rng(43)
    at = np.r_[0:n, R - n:R]
    rows = torch.from_numpy(at).cuda()

    def tensor(dt):
        t = torch.zeros(R, D, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device="cuda")
        v, v64 = _dev(rng.standard_normal((2 * n, D)), dt)
        t[rows] = v
        return t, v64

    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    (y, y64), (z, z64), (do, do64) = tensor("bf16"), tensor("bf16"), tensor("bf16")
    out, rstd = ssd.gated_norm_forward(y, z, w, groups=G)
    wo, wr = ref.gated(y64, z64, w64, 1e-5, G)
    ref.assert_close(out[rows], wo, "bf16", "out")
    ref.assert_close(rstd[rows], wr, "f32", "rstd")
    del out
    g = ssd.gated_norm_backward(do, y, z, w, rstd, groups=G)
    dy, dz, dw = ref.gated_bwd(do64, y64, z64, w64, rstd[rows].double().cpu().numpy(), G)
    ref.assert_close(g["dy"][rows], dy, "bf16", "dy")
    ref.assert_close(g["dz"][rows], dz, "bf16", "dz")
    ref.assert_close(g["d_weight"], dw, "f32", "d_weight")
    del g, y, z, rstd
    h, h64 = tensor("f32")
    dh, dh64 = tensor("f32")
    _, _, st = ref.norm(h64, w64, None, None, 1e-5, True)
    stats = torch.zeros(R, 2, device="cuda")
    stats[rows] = torch.from_numpy(st.astype(np.float32)).cuda()
    g = ssd.norm_backward(do, h, w, stats, dh=dh)
    dv, dw, db = ref.norm_bwd(do64, h64, w64, stats[rows].double().cpu().numpy(), dh64, True)
    ref.assert_close(g["dx"][rows], dv, "bf16", "dx")
    ref.assert_close(g["d_residual"][rows], dv, "f32", "d_residual")
    ref.assert_close(g["d_weight"], dw, "f32", "d_weight")
    ref.assert_close(g["d_bias"], db, "f32", "d_bias")


# More rows than the GPU holds at once, so that every block goes round its ring.
@pytest.mark.parametrize("dt,rdt,D", [("f32", "f32", 12288), ("bf16", "f32", 16384), ("bf16", "bf16", 9000),
                                      ("f32", None, 16384), ("bf16", None, 12000)])
def test_long_rows(ssd, dt, rdt, D):  # noqa: F811
    import torch
    R = 700
    rng = np.random.default_rng(D)
    x, x64 = _dev(rng.standard_normal((R, D)), dt)
    res, res64 = _dev(rng.standard_normal((R, D)), rdt) if rdt else (None, None)
    dy, dy64 = _dev(rng.standard_normal((R, D)), dt)
    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    y, h, stats = ssd.norm_forward(x, w, residual=res)
    wy, wh, _ = ref.norm(x64, w64, None, res64, 1e-5, True)
    ref.assert_close(y, wy, dt, "y")
    h64 = h.double().cpu().numpy()
    ref.assert_close(h, wh, rdt or dt, "h")
    g = ssd.norm_backward(dy, h, w, stats, dh=res)
    dv, dw, db = ref.norm_bwd(dy64, h64, w64, stats.double().cpu().numpy(), res64, True)
    ref.assert_close(g["dx"], dv, dt, "dx")
    ref.assert_close(g["d_weight"], dw, "f32", "d_weight")
    ref.assert_close(g["d_bias"], db, "f32", "d_bias")
    z, z64 = _dev(rng.standard_normal((R, D)), dt)
    out, rstd = ssd.gated_norm_forward(x, z, w)
    wo, _ = ref.gated(x64, z64, w64, 1e-5, 1)
    ref.assert_close(out, wo, dt, "out")
    gg = ssd.gated_norm_backward(dy, x, z, w, rstd)
    ey, ez, ew = ref.gated_bwd(dy64, x64, z64, w64, rstd.double().cpu().numpy(), 1)
    ref.assert_close(gg["dy"], ey, dt, "dy")
    ref.assert_close(gg["dz"], ez, dt, "dz")
    ref.assert_close(gg["d_weight"], ew, "f32", "gated d_weight")
