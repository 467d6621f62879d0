"""Linear attention with a decay for each head against all pairs of tokens in 64 bits.

Bounds: each output is off by half a step of its type, and by the roundings of the terms it adds
up: ``roundings`` of float32 and, on the tensor cores, one of bfloat16 (the masked product, or the
state that meets q), each relative to the sum of the terms' absolute values."""

import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import state_space_model_ssd_gb300 as m
    return m


def _make(B, L, H, G, P, N, dtype, cu=None, state=False, strided=False, seed=0, fast=2.0, offset=0):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if strided:
        w = H * N + G * (N + P) + 2 * offset
        rows = r(B, L, w).to(dt)[..., offset:]
        q = rows[..., :H * N].unflatten(2, (H, N))
        k = rows[..., H * N:H * N + G * N].unflatten(2, (G, N))
        v = rows[..., H * N + G * N:H * N + G * (N + P)].unflatten(2, (G, P))
    else:
        q, k, v = r(B, L, H, N).to(dt), r(B, L, G, N).to(dt), r(B, L, G, P).to(dt)
    ld = -fast * torch.exp2(-8.0 * torch.arange(H, device="cuda") / max(1, H - 1)).float()
    n = B if cu is None else len(cu) - 1
    s = dict(q=q, k=k, v=v, ld=ld, scale=N ** -0.5, n=n,
             cu=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
             cuts=ref.borders(B, L, cu), do=r(B, L, H, P).to(dt),
             init=r(n, H, P, N) if state else None, dfinal=r(n, H, P, N) if state else None)
    return s


def _bound(s, exact, total, tc, kind):
    """Half a step of the output's type, and the terms' roundings."""
    N, P = s["q"].shape[3], s["v"].shape[3]
    longest = max([b - a for a, b in zip(s["cuts"], s["cuts"][1:])] + [0])
    terms = ref.roundings(N, P, longest) * ref.EPS32
    if kind == "state":
        return terms * total + ref.EPS32 * exact.abs()
    half = ref.EPS16 if s["q"].dtype.itemsize == 2 else ref.EPS32
    # a state that meets q in bfloat16 was itself summed in float32
    return (terms + (ref.EPS16 * (1 + ref.EPS16) if tc else 0.0)) * total * (1 + half) + half * exact.abs()


def _check(name, got, exact, bound):
    import torch
    d = (got.double() - exact).abs()
    assert torch.isfinite(got.double()).all(), name
    worst = (d - bound).max().item() if d.numel() else 0.0
    assert worst <= 0.0, "%s: off by up to %.3g more than its bound (max %.3g)" % (name, worst, d.max().item())


def _forward(ssd, s, tc, **kw):
    o, final = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], scale=s["scale"],
                                            cu_seqlens=s["cu"], initial_state=s["init"], final_state=True, **kw)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    a = lambda t: None if t is None else t.double().abs()  # noqa: E731
    args = (s["ld"].double(), s["scale"], s["cuts"])
    eo, ef = ref.attention(d(s["q"]), d(s["k"]), d(s["v"]), *args, d(s["init"]))
    to, tf = ref.attention(a(s["q"]), a(s["k"]), a(s["v"]), *args, a(s["init"]))
    _check("o", o, eo, _bound(s, eo, to, tc, "o"))
    _check("final", final, ef, _bound(s, ef, tf, tc, "state"))
    return o, final


def _backward(ssd, s, tc, **kw):
    state = s["init"] is not None
    g = ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], scale=s["scale"],
                                      cu_seqlens=s["cu"], initial_state=s["init"], d_final_state=s["dfinal"],
                                      d_initial_state=state, **kw)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    a = lambda t: None if t is None else t.double().abs()  # noqa: E731
    args = (s["ld"].double(), s["scale"], s["cuts"])
    exact = ref.gradients(d(s["q"]), d(s["k"]), d(s["v"]), *args, d(s["do"]), d(s["init"]), d(s["dfinal"]))
    total = ref.gradients(a(s["q"]), a(s["k"]), a(s["v"]), *args, a(s["do"]), a(s["init"]), a(s["dfinal"]))
    for name, e, t in zip(("dq", "dk", "dv", "d_initial_state"), exact, total):
        _check(name, g[name], e, _bound(s, e, t, tc, "state" if name == "d_initial_state" else "o"))
    return g


# B, L, H, G, P, N, cu, state, strided, offset
SHAPES = [
    (1, 1, 1, 1, 1, 1, None, False, False, 0),
    (2, 33, 3, 3, 13, 21, None, True, False, 0),
    (1, 100, 4, 2, 33, 65, None, True, True, 0),
    (1, 77, 2, 1, 128, 128, [0, 0, 5, 6, 38, 70, 70], True, False, 0),
    (3, 1, 5, 5, 7, 128, None, True, False, 0),
    (1, 64, 3, 1, 100, 3, None, False, True, 3),
    (1, 700, 2, 2, 16, 8, None, True, False, 0),           # more than one segment
    (1, 1300, 3, 1, 20, 12, [0, 600, 600, 601, 1250], True, True, 0),
]
TC = [
    (1, 1, 2, 2, 64, 64, None, True, False, 0),
    (1, 128, 3, 3, 64, 128, None, True, True, 0),
    (2, 130, 2, 1, 128, 64, None, False, False, 0),
    (1, 257, 4, 2, 128, 128, [0, 0, 1, 64, 191, 257], True, False, 0),
    (1, 1500, 3, 3, 64, 64, None, True, False, 0),
    (1, 2100, 4, 1, 64, 128, [0, 1290, 1290, 1300, 1428], True, True, 0),
    (2, 700, 2, 2, 128, 128, None, True, True, 0),
    (1, 200, 2, 2, 64, 64, None, True, True, 4),           # rows off 16 bytes: the plain cores
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_any_size(ssd, shape, dtype):
    *sizes, cu, state, strided, offset = shape
    s = _make(*sizes, dtype, cu, state, strided, offset=offset)
    # the one of 128 x 128 channels takes the tensor cores in bfloat16, and has their roundings
    tc = dtype == "bf16" and sizes[4] == sizes[5] == 128
    _forward(ssd, s, tc)
    _backward(ssd, s, tc)


@pytest.mark.parametrize("shape", TC)
def test_tensor_cores(ssd, shape):
    *sizes, cu, state, strided, offset = shape
    s = _make(*sizes, "bf16", cu, state, strided, offset=offset)
    _forward(ssd, s, True)
    _backward(ssd, s, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,cu", [(1, None), (2, None), (16, None), (17, None), (16, [0, 0, 5, 5, 12]), (9, [0, 9])])
@pytest.mark.parametrize("B,H,G,P,N", [(1, 4, 2, 64, 128), (3, 2, 1, 100, 12), (2, 3, 3, 5, 7), (1, 80, 80, 64, 64)])
def test_a_few_tokens(ssd, B, H, G, P, N, L, cu, dtype):
    """Up to sixteen tokens a sequence are stepped through, in float32; one more is a walk."""
    if cu is not None and B > 1:
        B = 1
    s = _make(B, L, H, G, P, N, dtype, cu, True, L % 2 == 1)
    walk = L > 16 and dtype == "bf16" and P % 64 == 0 and N % 64 == 0
    o, _ = _forward(ssd, s, walk)
    if cu is not None:
        assert not o[:, cu[-1]:].any()


# the forms of the launch: whole sequences by the pass, states of 128 channels by sums of their own, cut
# sequences with their final states from the scan, one long sequence of many segments
@pytest.mark.parametrize("B,L,H,G,P,N,state,strided", [(4, 2100, 26, 26, 64, 64, True, False),
                                                       (4, 2100, 26, 13, 64, 64, False, True),
                                                       (8, 1100, 20, 20, 128, 128, True, False),
                                                       (6, 1024, 30, 10, 64, 128, True, True),
                                                       (2, 5000, 3, 1, 64, 128, True, False)])
def test_forms_of_the_launch(ssd, B, L, H, G, P, N, state, strided):
    s = _make(B, L, H, G, P, N, "bf16", None, state, strided, seed=11)
    _forward(ssd, s, True)
    _backward(ssd, s, True)


# enough tokens of other channels for their rows to be laid out anew for the tensor cores; the last two
# just too few, and too narrow, for that
@pytest.mark.parametrize("B,L,H,G,P,N,cu,state,strided,offset,tc", [
    (2, 1030, 8, 8, 90, 15, None, True, False, 0, True),
    (1, 2100, 8, 2, 33, 65, None, True, True, 3, True),
    (1, 2100, 8, 4, 80, 96, [0, 1290, 1290, 1300, 1428], True, True, 0, True),
    (9, 130, 15, 5, 127, 64, None, False, True, 1, True),
    (950, 18, 1, 1, 31, 17, None, True, False, 0, True),
    (1, 2047, 8, 2, 33, 65, None, True, False, 0, False),
    (1, 2100, 8, 8, 12, 10, None, True, True, 0, False)])
def test_rows_laid_out_anew(ssd, B, L, H, G, P, N, cu, state, strided, offset, tc):
    import torch
    s = _make(B, L, H, G, P, N, "bf16", cu, state, strided, seed=17, offset=offset)
    o, final = _forward(ssd, s, tc)
    g = _backward(ssd, s, tc)
    # into slices of wider rows, what lies beside them left as it is
    rows = torch.full((B, L, H * N + G * (N + P) + 5), 7.0, device="cuda", dtype=torch.bfloat16)
    views = {"dq": rows[..., 1:1 + H * N].unflatten(2, (H, N)),
             "dk": rows[..., 2 + H * N:2 + (H + G) * N].unflatten(2, (G, N)),
             "dv": rows[..., 4 + (H + G) * N:4 + (H + G) * N + G * P].unflatten(2, (G, P))}
    ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], scale=s["scale"], cu_seqlens=s["cu"],
                                  initial_state=s["init"], d_final_state=s["dfinal"], d_initial_state=state,
                                  out=dict(views))
    for name, view in views.items():
        assert torch.equal(view, g[name]), name
    beside = [0, 1 + H * N, 2 + (H + G) * N, 3 + (H + G) * N, rows.shape[2] - 1]
    assert (rows[..., beside] == 7).all()
    if cu is not None:
        assert not o[:, cu[-1]:].any() and not views["dq"][:, cu[-1]:].any()
    # captured on a stream of its own, without the states
    call = lambda: ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], scale=s["scale"],  # noqa: E731
                                                cu_seqlens=s["cu"], initial_state=s["init"])
    o2, none = call()
    assert none is None and torch.isfinite(o2).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, _ = call()
    o3.fill_(7.0)
    graph.replay()
    assert torch.equal(o2, o3)


@pytest.mark.parametrize("B,L,H,P,N", [(8, 4096, 20, 128, 128), (2, 4096, 32, 128, 64), (1, 16384, 8, 64, 64),
                                       (4, 4096, 40, 64, 64)])
def test_states_of_slow_decays_keep_their_bits(ssd, B, L, H, P, N):
    """States that thousands of tokens are summed into: off by 2^-19 of their size at most, in each
    direction.  The weighted values are split to 2^-25.  The tensor cores' sums may cut off instead of
    rounding: 512 tokens are 96 additions of 16, each of which loses half of 2^-23 of a sum in the mean
    that is itself half its size in the mean: 96 * 2^-25 = 2^-18.4 of that run's part, and a run is at
    most half of what a state of 4096 tokens and these decays holds."""
    import torch
    s = _make(B, L, H, H, P, N, "bf16", state=True, seed=13)
    ld = -torch.exp2(-6 - 6 * torch.arange(H, device="cuda") / (H - 1)).float()
    _, final = ssd.linear_attention_forward(s["q"], s["k"], s["v"], ld, initial_state=s["init"], final_state=True,
                                            scale=s["scale"])
    back = ssd.linear_attention_backward(s["q"], s["k"], s["v"], ld, s["do"], scale=s["scale"],
                                         initial_state=s["init"], d_final_state=s["dfinal"], d_initial_state=True)
    a = ld.double()

    def walk(S, rows, cols, blocks, weight):
        for lo in blocks:
            hi = min(lo + 64, L)
            t = torch.arange(hi - lo, device="cuda", dtype=torch.float64)
            w = torch.exp(a[:, None] * weight(t, hi - lo))
            S = S * torch.exp(a * (hi - lo))[:, None, None] + torch.einsum(
                "bthp,ht,bthn->bhpn", rows[:, lo:hi].double(), w, cols[:, lo:hi].double())
        return S

    ends = {"final": (final, walk(s["init"].double(), s["v"], s["k"], range(0, L, 64), lambda t, m: m - 1 - t)),
            "d_initial": (back["d_initial_state"],
                          walk(s["dfinal"].double(), s["do"].double() * s["scale"], s["q"],
                               reversed(range(0, L, 64)), lambda t, m: t + 1))}
    for name, (got, exact) in ends.items():
        off = (got.double() - exact).norm(dim=(2, 3)) / exact.norm(dim=(2, 3))
        assert off.max().item() <= 2.0 ** -19, (name, off.max().item())


def test_offsets_beyond_32_bits(ssd):
    """Tokens whose elements lie beyond 2^31: the end of a long sequence is that of a short one that goes
    on from its state."""
    import torch
    T, H, N, P = 290000, 60, 128, 64
    assert T * H * N > 2 ** 31
    q = torch.randn(1, T, H, N, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(1, T, H, N, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1, T, H, P, device="cuda", dtype=torch.bfloat16)
    ld = -torch.exp2(-2.0 - 6.0 * torch.arange(H, device="cuda") / H).float()
    o, final = ssd.linear_attention_forward(q, k, v, ld, final_state=True)
    cut = T - 1000
    _, state = ssd.linear_attention_forward(q[:, cut - 20000:cut], k[:, cut - 20000:cut], v[:, cut - 20000:cut], ld,
                                            final_state=True)   # e^(-20000 / 256) of what was before is gone
    o1, final1 = ssd.linear_attention_forward(q[:, cut:], k[:, cut:], v[:, cut:], ld, initial_state=state,
                                              final_state=True)
    # two float32 sums of thousands of terms in other orders; outputs rounded to bfloat16 thrice
    assert (final - final1).norm() <= 1e-5 * final.norm()
    d = (o[:, cut:].float() - o1.float()).norm()
    assert d <= 3 * ref.EPS16 * o1.float().norm()
    g = ssd.linear_attention_backward(q, k, v, ld, o)
    g1 = ssd.linear_attention_backward(q[:, cut:], k[:, cut:], v[:, cut:], ld, o[:, cut:], initial_state=state)
    for n in ("dq", "dk", "dv"):
        a, b = g[n][:, cut:].float(), g1[n].float()
        assert (a - b).norm() <= 3 * ref.EPS16 * b.norm(), n


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128), (24, 40)])
@pytest.mark.parametrize("ld", [0.0, -1e-6, -30.0, -1e9, float("-inf")])
def test_decays(ssd, ld, P, N):
    """From no decay at all to one that forgets at once, in one call with others."""
    s = _make(1, 300, 2, 2, P, N, "bf16", [0, 200, 300], True)
    s["ld"][0] = ld
    _forward(ssd, s, P % 64 == 0)
    _backward(ssd, s, P % 64 == 0)


def test_chunks_of_a_prompt(ssd):
    """A prompt in pieces, each from the state of the last, then token by token over cache slots: the
    same outputs as in one go, within the bounds of both."""
    import torch
    s = _make(1, 517, 6, 3, 64, 128, "bf16", None, True)
    o, final = _forward(ssd, s, True)
    state, parts = s["init"], []
    for lo, hi in ((0, 128), (128, 129), (129, 500)):
        p, state = ssd.linear_attention_forward(s["q"][:, lo:hi], s["k"][:, lo:hi], s["v"][:, lo:hi], s["ld"],
                                                scale=s["scale"], initial_state=state, final_state=True)
        parts.append(p)
    cache = torch.randn(3, *state.shape[1:], device="cuda")
    cache[2] = state[0]
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in range(500, 517):
        parts.append(ssd.linear_attention_step(cache, s["q"][:, t], s["k"][:, t], s["v"][:, t], s["ld"],
                                               scale=s["scale"], slots=slots)[:, None])
    d = lambda t: t.double()  # noqa: E731
    a = lambda t: t.double().abs()  # noqa: E731
    args = (s["ld"].double(), s["scale"], s["cuts"])
    eo, ef = ref.attention(d(s["q"]), d(s["k"]), d(s["v"]), *args, d(s["init"]))
    to, tf = ref.attention(a(s["q"]), a(s["k"]), a(s["v"]), *args, a(s["init"]))
    _check("o", torch.cat(parts, 1), eo, _bound(s, eo, to, True, "o"))
    _check("final", cache[2:], ef, _bound(s, ef, tf, True, "state"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,P,N,strided", [(1, 1, 1, 1, 1, False), (5, 3, 1, 13, 21, True), (4, 2, 2, 64, 128, True),
                                               (40, 80, 80, 64, 128, False), (3, 4, 2, 128, 12, False),
                                               (2, 2, 1, 100, 127, True)])
def test_step(ssd, B, H, G, P, N, strided, dtype):
    import torch
    s = _make(B, 1, H, G, P, N, dtype, None, False, strided, seed=3)
    q, k, v = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
    nslots = B + 2
    state = torch.randn(nslots, H, P, N, device="cuda")
    before = state.clone()
    slots = torch.randperm(nslots, device="cuda")[:B].to(torch.int32)
    dead = []
    if B > 2:
        slots[1], slots[2] = -1, nslots
        dead = [1, 2]
    o = ssd.linear_attention_step(state, q, k, v, s["ld"], scale=s["scale"], slots=slots)
    live = [i for i in range(B) if i not in dead]
    sl = slots.long()[live]
    kk = k.double().repeat_interleave(H // G, 1)[live]
    vv = v.double().repeat_interleave(H // G, 1)[live]
    a = torch.exp(s["ld"].double())[:, None, None]
    e = a * before[sl].double() + vv[..., None] * kk[:, :, None, :]
    t = a * before[sl].double().abs() + vv.abs()[..., None] * kk.abs()[:, :, None, :]
    # expf within two units, a product and a sum
    assert ((state[sl].double() - e).abs() <= 8 * ref.EPS32 * t).all()
    qq = q.double()[live][:, :, None, :]
    eo, to = (e * qq).sum(-1) * s["scale"], (t * qq.abs()).sum(-1) * s["scale"]
    half = ref.EPS16 if dtype == "bf16" else ref.EPS32
    assert ((o[live].double() - eo).abs() <= (N + 16) * ref.EPS32 * to * (1 + half) + half * eo.abs()).all()
    assert not o[dead].any()
    others = [i for i in range(nslots) if i not in sl.tolist()]
    assert torch.equal(state[others], before[others])


def test_directional_derivative(ssd):
    """The gradients against differences of the forward in float32: the loss is linear in each of q, k
    and v alone, so that a central difference has no error but rounding."""
    import torch
    s = _make(1, 90, 3, 3, 24, 20, "f32", None, True, seed=7)
    g = _backward(ssd, s, False)

    def loss(**kw):
        t = {**s, **kw}
        o, final = ssd.linear_attention_forward(t["q"], t["k"], t["v"], t["ld"], scale=t["scale"],
                                                initial_state=t["init"], final_state=True)
        return (o.double() * s["do"].double()).sum() + (final.double() * s["dfinal"].double()).sum()

    for x, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("init", "d_initial_state")):
        u = torch.randn_like(s[x])
        diff = (loss(**{x: s[x] + u}) - loss(**{x: s[x] - u})) / 2
        total = float((g[name].double().abs() * u.double().abs()).sum())
        assert abs(float(diff - (g[name].double() * u.double()).sum())) <= 2e-5 * total


def test_tokens_behind_the_last_sequence(ssd):
    import torch
    for sizes in ((1, 300, 2, 1, 64, 64), (1, 300, 2, 1, 24, 40), (1, 2000, 2, 1, 64, 64)):
        s = _make(*sizes, "bf16", [0, 100, 150])
        s["q"][:, 150:] = float("nan")
        outs = {n: torch.full_like(s[x], 7.0) for n, x in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
        o = torch.full_like(s["do"], 7.0)
        ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"], out=o)
        g = ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], cu_seqlens=s["cu"], out=outs)
        assert torch.isfinite(o).all() and not o[:, 150:].any()
        for n in ("dq", "dk", "dv"):
            assert torch.isfinite(g[n]).all() and not g[n][:, 150:].any(), n


@pytest.mark.parametrize("P,N,L", [(64, 64, 300), (64, 128, 1500), (13, 20, 300)])
def test_a_sequence_of_nan_stays_alone(ssd, P, N, L):
    import torch
    s = _make(1, L, 2, 2, P, N, "bf16", [0, 90, 170, L], True)
    o0, f0 = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"],
                                          initial_state=s["init"], final_state=True)
    args = dict(cu_seqlens=s["cu"], initial_state=s["init"], d_final_state=s["dfinal"], d_initial_state=True)
    g0 = ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], **args)
    for x in "qkv":
        s[x][:, 90:170] = float("nan") if x != "k" else float("inf")
    s["do"][:, 90:170] = float("nan")
    o1, f1 = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"],
                                          initial_state=s["init"], final_state=True)
    g1 = ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["ld"], s["do"], **args)
    for a, b in ((o0, o1), (g0["dq"], g1["dq"]), (g0["dk"], g1["dk"]), (g0["dv"], g1["dv"])):
        assert torch.equal(a[:, :90], b[:, :90]) and torch.equal(a[:, 170:], b[:, 170:])
    for a, b in ((f0, f1), (g0["d_initial_state"], g1["d_initial_state"])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


@pytest.mark.parametrize("cu", [[0, 400, 100, 300], [-5, 100, 9999, 300], [300, 200, 100, 0]])
@pytest.mark.parametrize("P,N", [(64, 64), (20, 20)])
def test_malformed_borders_stay_in_range(ssd, cu, P, N):
    """Wrong values, but none outside the tensors: those around them keep theirs."""
    import torch
    s = _make(1, 300, 2, 2, P, N, "bf16", cu, True)
    big = torch.full((3, 300, 2, P), 7.0, device="cuda", dtype=torch.bfloat16)
    ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["ld"], cu_seqlens=s["cu"], initial_state=s["init"],
                                 out=big[1:2])
    torch.cuda.synchronize()
    assert (big[0] == 7).all() and (big[2] == 7).all()


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (24, 20, "f32")])
def test_same_bits_in_a_graph_on_another_stream_and_strided_outputs(ssd, P, N, dtype):
    import torch
    s = _make(1, 900, 4, 2, P, N, dtype, None, True)
    run = lambda **kw: ssd.linear_attention_backward(  # noqa: E731
        s["q"], s["k"], s["v"], s["ld"], s["do"], initial_state=s["init"], d_final_state=s["dfinal"],
        d_initial_state=True, **kw)
    fwd = lambda **kw: ssd.linear_attention_forward(  # noqa: E731
        s["q"], s["k"], s["v"], s["ld"], initial_state=s["init"], final_state=True, **kw)
    g0, (o0, f0) = run(), fwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g1, (o1, f1) = run(stream=side), fwd(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    wide = torch.zeros(1, 900, 4 * N + 2 * (N + P), device="cuda", dtype=s["q"].dtype)
    out = {"dq": wide[..., :4 * N].unflatten(2, (4, N)), "dk": wide[..., 4 * N:6 * N].unflatten(2, (2, N)),
           "dv": wide[..., 6 * N:].unflatten(2, (2, P))}
    g2 = run(out=out)
    assert g2 is out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g3, (o3, f3) = run(), fwd()
    for t in (*g3.values(), o3, f3):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n in g0:
        assert torch.equal(g0[n], g1[n]) and torch.equal(g0[n], g2[n]) and torch.equal(g0[n], g3[n]), n
    assert torch.equal(o0, o1) and torch.equal(f0, f1) and torch.equal(o0, o3) and torch.equal(f0, f3)
    assert ssd.layer_status() == 0


def test_no_tokens(ssd):
    import torch
    for P, N, dt in ((64, 64, torch.bfloat16), (5, 9, torch.float32)):
        q = torch.zeros(2, 0, 3, N, device="cuda", dtype=dt)
        k, v = q[..., :1, :], torch.zeros(2, 0, 1, P, device="cuda", dtype=dt)
        ld = torch.zeros(3, device="cuda")
        init = torch.randn(2, 3, P, N, device="cuda")
        o, final = ssd.linear_attention_forward(q, k, v, ld, initial_state=init, final_state=True)
        assert o.shape == (2, 0, 3, P) and torch.equal(final, init)
        g = ssd.linear_attention_backward(q, k, v, ld, o, d_final_state=init, d_initial_state=True)
        assert torch.equal(g["d_initial_state"], init)
