"""Linear attention: borders that are not what they should be, rows of no sequence, and which of the
kernels takes a call."""

import contextlib
import ctypes

import pytest

from test_linear_attention_gpu import _backward, _forward, _make, ssd  # noqa: F401  (ssd is the built package)

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _launches(ssd, names):  # noqa: F811
    """The names of the kernels launched meanwhile, into the list ``names``."""
    ssd.profiler.reset()
    ssd.profiler.enable(True)
    try:
        yield
        names += ssd.profiler.read()
    finally:
        ssd.profiler.enable(False)
        ssd.profiler.reset()


def _workspace_size(s, bwd):
    from state_space_model_ssd_gb300 import _lib
    q, k, v = s["q"], s["k"], s["v"]
    (B, L, H, N), G, P = q.shape, k.shape[2], v.shape[3]
    p = _lib.LinAttnProblem(B, L, q.stride(1), k.stride(1), v.stride(1), H * P, *((H * N, G * N, G * P) if bwd else (0, 0, 0)),
                            H, G, P, N, 0 if s["cu"] is None else s["n"], 1 if q.dtype.itemsize == 2 else 0, s["scale"])
    n = ctypes.c_size_t()
    assert _lib.lib().ssd_linear_attention_workspace_size(ctypes.byref(p), bwd, ctypes.byref(n)) == 0
    return n.value


# few tokens, plain cores, tensor cores uncut and cut, rows laid out anew; heads of their own and shared
@pytest.mark.parametrize("L,H,G,P,N,cu", [
    (12, 3, 3, 16, 12, [4, 4, 9]), (300, 2, 2, 13, 20, [37, 100, 290]), (300, 4, 2, 13, 20, [37, 100, 290]),
    (300, 2, 2, 64, 64, [130, 140, 300]), (2000, 4, 2, 64, 128, [700, 701, 1900]),
    (2100, 8, 8, 80, 96, [515, 1900, 2100]), (2100, 8, 2, 33, 65, [1, 1900, 2050])])
def test_tokens_before_the_first_sequence(ssd, L, H, G, P, N, cu):  # noqa: F811
    """Borders cut out of a longer list start behind 0: outputs and gradients of the tokens before
    are zero, whatever the workspace held."""
    import torch
    s = _make(1, L, H, G, P, N, "bf16", cu, True, seed=23)
    tc = L * H >= 16384 or (P % 64 == 0 and N % 64 == 0)
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")   # NaN in either type
    outs = {n: torch.full_like(s[x], 7.0) for n, x in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    o, _ = _forward(ssd, s, tc, out=torch.full_like(s["do"], 7.0), workspace=ws)
    ws.fill_(255)
    _backward(ssd, s, tc, out=outs, workspace=ws)
    for t in (o, *(outs[n] for n in ("dq", "dk", "dv"))):
        assert not t[:, :cu[0]].any() and not t[:, cu[-1]:].any()


# an odd number of elements beside q, k and v; whole rows on 16 bytes, but q, k and v off them
@pytest.mark.parametrize("L,H,G,P,N,cu", [(2100, 8, 8, 64, 128, None), (2100, 8, 2, 128, 64, [0, 1290, 1290, 1300, 1428]),
                                          (4200, 4, 4, 64, 64, None)])
@pytest.mark.parametrize("offset", [3, 4])
def test_rows_off_16_bytes(ssd, L, H, G, P, N, cu, offset):  # noqa: F811
    """Many rows of 64 and 128 channels reach the tensor cores by copies, as those of other channels do."""
    import torch
    s = _make(1, L, H, G, P, N, "bf16", cu, True, True, seed=29, offset=offset)
    assert (s["q"].stride(1) % 8 == 0) == (offset == 4) and s["q"].data_ptr() % 16
    names = []
    with _launches(ssd, names):
        _forward(ssd, s, True)
        _backward(ssd, s, True)
    assert {"linattn_pad", "linattn_tc_walk", "linattn_unpad"} <= set(names) and "linattn_walk" not in names
    # a workspace of the size asked for by the strides does
    names = []
    with _launches(ssd, names):
        _forward(ssd, s, True, workspace=torch.empty(_workspace_size(s, 0), dtype=torch.uint8, device="cuda"))
        _backward(ssd, s, True, workspace=torch.empty(_workspace_size(s, 1), dtype=torch.uint8, device="cuda"))
    assert ("linattn_pad" in names) == (offset == 3) and ("linattn_walk" in names) == (offset == 4)


@pytest.mark.parametrize("offset", [3, 4])
def test_few_rows_off_16_bytes(ssd, offset):  # noqa: F811
    """Too few rows for copies: cut for the plain cores, which go through 32 tokens at a time, not for the
    tensor cores."""
    s = _make(1, 400, 2, 2, 64, 64, "bf16", None, True, True, offset=offset)
    names = []
    with _launches(ssd, names):
        _forward(ssd, s, False)
        _backward(ssd, s, False)
    assert set(names) == {"linattn_sums", "linattn_scan", "linattn_walk"}


# the tests of the tensor cores take them, directly or by copies
@pytest.mark.parametrize("L,H,G,P,N,cu,names", [
    (1500, 3, 3, 64, 64, None, {"linattn_tc_sums", "linattn_scan", "linattn_tc_walk"}),
    (130, 2, 1, 128, 64, None, {"linattn_tc_walk", "linattn_shared_sum"}),
    (257, 4, 2, 128, 128, [0, 0, 1, 64, 191, 257], {"linattn_tc_walk", "linattn_shared_sum"}),
    (2100, 8, 8, 80, 96, None, {"linattn_pad", "linattn_tc_sums", "linattn_scan", "linattn_tc_walk", "linattn_unpad"}),
    (2047, 8, 8, 33, 65, None, {"linattn_sums", "linattn_scan", "linattn_walk"}),
    (2100, 8, 8, 12, 10, None, {"linattn_sums", "linattn_scan", "linattn_walk"})])
def test_which_kernels_run(ssd, L, H, G, P, N, cu, names):  # noqa: F811
    s = _make(1, L, H, G, P, N, "bf16", cu, True, seed=5)
    got = []
    with _launches(ssd, got):
        ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"], final_state=True)
        ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], cu_seqlens=s["cu"])
    assert set(got) == names


def test_step_on_states_off_16_bytes(ssd):  # noqa: F811
    """One layer's part of a cache for all layers, with rows that no 16 bytes divide: as by itself."""
    import torch
    s = _make(3, 1, 3, 3, 5, 21, "bf16", seed=37)
    cache = torch.randn(4, 5, 3, 5, 21, device="cuda")
    before = cache.clone()
    assert cache[1].data_ptr() % 16
    args = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0], s["ld"]
    alone = cache[1].clone()
    want = ssd.linear_attention_step(alone, *args)
    assert torch.equal(ssd.linear_attention_step(cache[1], *args), want)
    before[1] = alone
    assert torch.equal(cache, before)


def _guarded(n, dtype, shape):
    """A tensor in the middle of a buffer of 7, 256-byte aligned, and a check that what is around it is left."""
    import torch
    size = torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * 4096 // size,), 7, dtype=dtype, device="cuda")
    lo = 4096 // size

    def left():
        return bool((buf[:lo] == 7).all()) and bool((buf[lo + n:] == 7).all())

    return buf[lo:lo + n].view(shape), left


# plain cores, tensor cores cut and uncut, rows laid out anew, shared heads, a few tokens
@pytest.mark.parametrize("L,H,G,P,N,dtype", [(14, 2, 2, 20, 20, "bf16"), (300, 2, 2, 20, 20, "f32"),
                                             (2000, 2, 2, 64, 64, "bf16"), (2000, 4, 2, 64, 128, "bf16"),
                                             (300, 4, 4, 128, 64, "bf16"), (2100, 8, 4, 80, 96, "bf16")])
@pytest.mark.parametrize("kind", ["falls", "far", "backwards", "saw"])
def test_borders_that_fall_write_nothing_outside(ssd, L, H, G, P, N, dtype, kind):  # noqa: F811
    """Both directions, with states, in workspaces and outputs of exactly their sizes, in the middle of
    others' memory; afterwards a sound call gives what it should."""
    import torch
    m = L - 1
    cu = {"falls": [0, m, m // 4, m // 2], "far": [-5, m // 3, 9 * L, m], "backwards": [m, m // 2, m // 3, 0],
          "saw": [0, m, 1, L, 2, m // 2, m // 3, L]}[kind]
    s = _make(1, L, H, G, P, N, dtype, cu, True, seed=41)
    n, dt = len(cu) - 1, s["q"].dtype
    checks = []

    def out(dtype, *shape):
        size = 1
        for d in shape:
            size *= d
        t, left = _guarded(size, dtype, shape)
        checks.append(left)
        return t

    o, final = out(dt, 1, L, H, P), out(torch.float32, n, H, P, N)
    ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], scale=s["scale"], cu_seqlens=s["cu"],
                                 initial_state=s["init"], out=o, final_state_out=final,
                                 workspace=out(torch.uint8, _workspace_size(s, 0)))
    grads = {"dq": out(dt, 1, L, H, N), "dk": out(dt, 1, L, G, N), "dv": out(dt, 1, L, G, P),
             "d_initial_state": out(torch.float32, n, H, P, N)}
    ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], scale=s["scale"], cu_seqlens=s["cu"],
                                  initial_state=s["init"], d_final_state=s["dfinal"], out=grads,
                                  workspace=out(torch.uint8, _workspace_size(s, 1)))
    torch.cuda.synchronize()
    assert all(left() for left in checks)
    assert ssd.layer_status() == 0
    s = _make(1, L, H, G, P, N, dtype, [0, m // 2, m], True, seed=43)
    _forward(ssd, s, dtype == "bf16")
    _backward(ssd, s, dtype == "bf16")


@pytest.mark.parametrize("L,H,G,P,N", [(2100, 8, 8, 80, 96), (2100, 8, 2, 33, 65), (2100, 8, 8, 64, 64)])
def test_a_sequence_of_nan_stays_alone_in_copies(ssd, L, H, G, P, N):  # noqa: F811
    """NaN and infinities of one sequence, its states among them, stay out of the others' outputs and
    gradients where rows are laid out anew."""
    import torch
    a, b = 700, 1413
    s = _make(1, L, H, G, P, N, "bf16", [0, a, b, L], True, P == 64, seed=47, offset=3)

    def run():
        names = []
        with _launches(ssd, names):
            o, f = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"],
                                                initial_state=s["init"], final_state=True)
            g = ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], cu_seqlens=s["cu"],
                                              initial_state=s["init"], d_final_state=s["dfinal"], d_initial_state=True)
        assert "linattn_pad" in names
        return (o, g["dq"], g["dk"], g["dv"]), (f, g["d_initial_state"])

    rows0, states0 = run()
    for x in "qv":
        s[x][:, a:b] = float("nan")
    s["k"][:, a:b] = float("inf")
    s["do"][:, a:b] = float("-inf")
    s["init"][1] = s["dfinal"][1] = float("nan")
    rows1, states1 = run()
    for x, y in zip(rows0, rows1):
        assert torch.isfinite(x).all() and torch.equal(x[:, :a], y[:, :a]) and torch.equal(x[:, b:], y[:, b:])
    for x, y in zip(states0, states1):
        assert torch.equal(x[[0, 2]], y[[0, 2]])


@pytest.mark.parametrize("B,L,H,G,P,N,cu", [(1, 1, 2, 2, 64, 128, None), (3, 4, 4, 2, 128, 128, None),
                                            (1, 14, 2, 2, 64, 128, list(range(15))), (2, 16, 3, 1, 128, 64, None),
                                            (1, 101, 1, 1, 128, 64, None), (1, 128, 2, 2, 64, 64, [0, 50, 50, 120]),
                                            (50, 70, 8, 8, 64, 64, None)])
@pytest.mark.parametrize("strided", [False, True])
def test_short_sequences_keep_their_scores(ssd, B, L, H, G, P, N, cu, strided):  # noqa: F811
    """Sequences within one block of tokens, which no state enters: off by half a step of bfloat16 and
    float32 roundings alone.  (Two bfloat16 terms hold a score to 2^-18, less than the float32 sums' bound:
    two hundred roundings and more of 2^-24.)"""
    s = _make(B, L, H, G, P, N, "bf16", cu, False, strided, seed=53)
    _forward(ssd, s, False)
    _backward(ssd, s, False)
