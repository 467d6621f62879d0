"""Beam search over cached states against plain loops in 64 bits."""

import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import state_space_model_ssd_gb300 as m
    return m


def _same(got, want, finished=None):
    """Whole numbers are equal; scores are off by half a step and by the logarithm's sum: float32
    sums of exponentials, each within 2^-20 of its value (its argument's rounding included)."""
    import torch
    scores, parents, tokens = got
    assert torch.equal(parents.long(), want[1]) and torch.equal(tokens.long(), want[2])
    low = torch.isinf(want[0])
    assert torch.equal(scores[low].double(), want[0][low])
    d = (scores.double() - want[0])[~low].abs()
    assert (d <= 2.0 ** -20 + ref.EPS32 * want[0][~low].abs()).all()


def _make(B, K, V, dtype, strided=False, seed=0, scale=2.5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, K, V + (7 if strided else 0), generator=g, device="cuda") * scale
    return x.to(dtype)[..., :V], -3 + 2 * torch.randn(B, K, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,K,V,keep,strided", [(1, 1, 1, 1, False), (2, 3, 5, 15, False), (3, 4, 1000, 8, True),
                                               (1, 4, 50277, 8, False), (20, 8, 9001, 16, True),
                                               (2, 16, 70001, 32, False), (1, 64, 300, 64, True),
                                               (40, 2, 2048, 64, False)])
def test_select(ssd, B, K, V, keep, strided, dtype):
    import torch
    x, s = _make(B, K, V, getattr(torch, dtype), strided)
    _same(ssd.beam_select(x, s, keep), ref.beam_select(x, s, keep))


def test_select_ties(ssd):
    """Few values, equal beams: the lowest beam, then the lowest token; the same beam at other
    alignments scores the same."""
    import torch
    x, s = _make(3, 4, 5001, torch.float32, seed=2)
    x = torch.round(x)
    s[:] = -1.0
    x[:, 1:] = x[:, :1]
    _same(ssd.beam_select(x, s, 16), ref.beam_select(x, s, 16))
    x[:] = 0.0
    _same(ssd.beam_select(x, s, 64), ref.beam_select(x, s, 64))


@pytest.mark.parametrize("V", [4095, 4096, 4097, 8192, 12289])
def test_select_slices(ssd, V):
    """Borders of slices, with enough rows for the wide ones; slices of equal logits, which outnumber
    the list of candidates, take the long way."""
    import torch
    x, s = _make(40, 4, V, torch.float32, seed=V)
    x[3] = torch.round(x[3])
    x[4] = 0.0
    x[5, :, ::2] = -torch.inf
    x[6] = -torch.inf
    x[6, :, 17] = 1.0
    x[7] = x[7, :1]
    s[7] = -1.0
    for keep in (1, 9, 64):
        _same(ssd.beam_select(x, s, keep), ref.beam_select(x, s, keep))


def test_select_order_of_the_vocabulary(ssd):
    """Rising and falling logits, and the best in one thread's reach."""
    import torch
    V = 20000
    up = torch.arange(V, device="cuda", dtype=torch.float32) / 1000
    x = torch.stack([up, up.flip(0), torch.where(torch.arange(V, device="cuda") % 256 == 3, up + 9, up)])[None]
    s = torch.tensor([[-1.0, -1.5, -2.0]], device="cuda")
    for keep in (1, 7, 64):
        _same(ssd.beam_select(x, s, keep), ref.beam_select(x, s, keep))


def test_select_masks(ssd):
    """Masked tokens, beams with nothing left, dead beams, NaN and infinities, ended beams."""
    import torch
    x, s = _make(6, 4, 900, torch.float32, seed=4)
    x[0, :, 3:] = -torch.inf                  # fewer tokens than are kept
    x[1, 0] = -torch.inf                      # a beam with nothing
    s[2, 1:] = -torch.inf                     # the first step of a search
    x[3, 2, 500] = float("nan")
    x[3, 3, 7] = torch.inf
    s[4, 0], s[4, 1] = torch.inf, float("nan")
    x[5] = -torch.inf
    for keep in (4, 16):
        _same(ssd.beam_select(x, s, keep), ref.beam_select(x, s, keep))
    f = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    f[0, 1] = f[1, 0] = f[2, 2] = f[3, 2] = True
    f[5] = True
    for pad in (0, 5, 899):
        _same(ssd.beam_select(x, s, 16, finished=f, pad_token=pad), ref.beam_select(x, s, 16, f, pad))
        _same(ssd.beam_select(x, s, 16, finished=f.to(torch.uint8), pad_token=pad), ref.beam_select(x, s, 16, f, pad))


def test_select_large_logits(ssd):
    import torch
    x, s = _make(2, 3, 3000, torch.float32, seed=5, scale=1.0)
    x = x * 1000 + 3e4
    _same_scores = ref.beam_select(x, s, 8)
    got = ssd.beam_select(x, s, 8)
    assert torch.equal(got[1].long(), _same_scores[1]) and torch.equal(got[2].long(), _same_scores[2])
    assert torch.allclose(got[0].double(), _same_scores[0], atol=1e-2, rtol=0)


@pytest.mark.parametrize("B,K", [(1, 1), (1, 4), (5, 7), (40, 16), (2, 64)])
@pytest.mark.parametrize("kind", ["random", "one", "swap", "bad"])
def test_reorder(ssd, B, K, kind):
    import torch
    g = torch.Generator().manual_seed(B * 100 + K)
    n = B * K + 4
    slots = torch.randperm(n, generator=g)[:B * K].view(B, K).to(torch.int32)
    parents = {"random": torch.randint(0, K, (B, K), generator=g), "one": torch.full((B, K), K - 1),
               "swap": torch.arange(K).flip(0).repeat(B, 1), "bad": torch.randint(-2, K + 2, (B, K), generator=g)}[kind]
    wide = torch.randn(n, 3000, device="cuda")
    caches = [torch.randn(n, 3, 16, 32, device="cuda"), torch.randn(n, 4, 77, device="cuda").bfloat16(),
              torch.randint(0, 255, (n, 13), device="cuda", dtype=torch.uint8), wide[:, 5:2500],
              torch.randn(n, device="cuda").double(), torch.zeros(n, 0, device="cuda")]
    before = [c.clone() for c in caches]
    rest = wide.clone()
    new = ssd.beam_reorder(caches, slots.cuda(), parents.to(torch.int32).cuda())
    want, copies = ref.beam_reorder(slots, parents)
    assert new.tolist() == want
    for c, b in zip(caches, before):
        for frm, to in copies:
            b[to] = b[frm]
        assert torch.equal(c, b)
    assert torch.equal(wide[:, :5], rest[:, :5]) and torch.equal(wide[:, 2500:], rest[:, 2500:])


def test_select_on_another_stream_into_given_outputs(ssd):
    import torch
    x, s = _make(3, 4, 3000, torch.bfloat16, seed=8)
    want = ssd.beam_select(x, s, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tuple(torch.empty_like(t) for t in want)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    got = ssd.beam_select(x, s, 6, out=out, workspace=ws, stream=side)
    new = ssd.beam_reorder([], want[1][:, :4].contiguous(), want[1][:, :4].contiguous(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(want, got, out):
        assert torch.equal(a, b) and b.data_ptr() == c.data_ptr()
    assert new.shape == (3, 4)


def test_reorder_leaves_slots_outside_the_cache(ssd):
    import torch
    cache = torch.randn(6, 100, device="cuda")
    before = cache.clone()
    slots = torch.tensor([[-1, 2, 9, 4]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[0, 0, 1, 1]], dtype=torch.int32, device="cuda")
    new = ssd.beam_reorder([cache], slots, parents)
    assert new.tolist() == [[-1, 9, 2, 4]]   # the pad's copy and the copy to 9 are not made
    before[4] = before[2]
    assert torch.equal(cache, before)


def test_reorder_many_caches(ssd):
    import torch
    caches = [torch.randn(8, 10 + i, device="cuda") for i in range(201)]
    want = [c.clone() for c in caches]
    slots = torch.tensor([[3, 1], [0, 7]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[1, 1], [0, 1]], dtype=torch.int32, device="cuda")
    new = ssd.beam_reorder(tuple(caches), slots, parents)
    assert new.tolist() == [[1, 3], [0, 7]]
    for c, w in zip(caches, want):
        w[3] = w[1]
        assert torch.equal(c, w)
    assert ssd.beam_reorder([], slots, parents).tolist() == [[1, 3], [0, 7]]


def test_a_search_over_recurrent_states(ssd):
    """Prompts, then beam search: the states of two layers (linear attention, the scan with its
    convolution's window) are stepped, chosen from and reordered, in a captured graph; at the end each
    beam's states are those of its own tokens gone through one by one."""
    import torch
    B, K, V, H, P, N, steps = 2, 3, 97, 2, 64, 64, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ld = -torch.tensor([0.02, 0.3], device="cuda")
    emb = (r(V, H * (2 * N + P)) * 0.5).bfloat16()
    head = r(H * P, V).bfloat16()
    C = H * P + 2 * N
    emb2, w, bias = (r(V, C) * 0.5).bfloat16(), r(C, 4), r(C)
    raw = r(V, H)

    def parts(tok):
        x = emb[tok]
        q, k, v = x.split([H * N, H * N, H * P], -1)
        return q.unflatten(-1, (H, N)), k.unflatten(-1, (H, N)), v.unflatten(-1, (H, P))

    prompt = torch.randint(0, V, (B, 9), generator=g, device="cuda")
    q, k, v = parts(prompt)
    _, first = ssd.linear_attention_forward(q, k, v, ld, final_state=True)
    n = B * K + 1
    state, scan, window = torch.zeros(n, H, P, N, device="cuda"), torch.zeros(n, H, P, N, device="cuda"), \
        torch.zeros(n, 4, C, device="cuda").bfloat16()
    slots = torch.arange(n - 1, device="cuda", dtype=torch.int32).flip(0).view(B, K).contiguous()
    state[slots.long()] = first[:, None]
    scores = torch.full((B, K), -torch.inf, device="cuda")
    scores[:, 0] = 0.0
    tok = torch.randint(0, V, (B, 1), generator=g, device="cuda").repeat(1, K)
    pos = torch.zeros(B * K, dtype=torch.int32, device="cuda")
    hist = tok[..., None].clone()

    def step(tok, slots, scores, pos):
        t = tok.flatten()
        q, k, v = parts(t)
        o = ssd.linear_attention_step(state, q, k, v, ld, slots=slots.flatten())
        y = ssd.conv_decode_step(scan, window, emb2[t], raw[t], w, bias, pos, -1.0, slots=slots.flatten())
        logits = ((o + y).flatten(1) @ head).unflatten(0, (B, K))
        s, par, new = ssd.beam_select(logits, scores)
        return s, par, new, ssd.beam_reorder([state, scan, window], slots, par)

    buf = [tok.clone(), slots.clone(), scores.clone(), pos.clone()]
    saved = [t.clone() for t in (state, scan, window)]
    step(*buf)                                        # warm-up
    for t, b in zip((state, scan, window), saved):
        t.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*buf)
    for t, b in zip((state, scan, window), saved):
        t.copy_(b)
    for _ in range(steps):
        graph.replay()
        s, par, new, sl = outs
        hist = torch.cat([hist.gather(1, par.long()[..., None].expand_as(hist)), new.long()[..., None]], -1)
        buf[0].copy_(new)
        buf[1].copy_(sl)
        buf[2].copy_(s)
        buf[3].add_(1)
    assert ((buf[2][:, :-1] >= buf[2][:, 1:]).all())
    state1, scan1, window1 = torch.zeros_like(state), torch.zeros_like(scan), torch.zeros_like(window)
    flat = buf[1].flatten()
    state1[flat.long()] = first.repeat_interleave(K, 0)
    for i in range(steps):
        t = hist[..., i].flatten()
        q, k, v = parts(t)
        ssd.linear_attention_step(state1, q, k, v, ld, slots=flat)
        ssd.conv_decode_step(scan1, window1, emb2[t], raw[t], w, bias,
                             torch.full((B * K,), i, dtype=torch.int32, device="cuda"), -1.0, slots=flat)
    for a, b in ((state, state1), (scan, scan1), (window, window1)):
        assert torch.equal(a[flat.long()], b[flat.long()])
