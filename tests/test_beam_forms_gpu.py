"""Beam search: orders that hang on the last bits, masked vocabularies, slices of either width."""

import pytest

import attn_ref as ref
from test_beam_gpu import _make, _same, ssd  # noqa: F401  (ssd is the built package)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [300, 3000, 20000])
@pytest.mark.parametrize("score", [-1e5, -7e8, 3e20, -3e38])
def test_one_beam_by_its_logits(ssd, V, score):  # noqa: F811
    """Logits closer to one another than their sums with the score can tell apart: still by the
    logits, equal ones by token."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randperm(V, generator=g, device="cuda").float() * 2.0 ** -40
    x[V // 2:V // 2 + 40] = x[::V // 40][:40]     # some twice
    x = x[None, None].repeat(1, 3, 1)
    s = torch.full((1, 3), score, device="cuda")
    s[:, 0] = s[:, 2] = -torch.inf
    for keep in (1, 8, 64):
        _, parents, tokens = ssd.beam_select(x, s, keep)
        assert (parents == 1).all()
        assert torch.equal(tokens[0].long(), torch.sort(x[0, 1], descending=True, stable=True).indices[:keep])


@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-6])
def test_each_beam_by_its_logits(ssd, scale):  # noqa: F811
    """Whatever the beams' scores do to one another, each beam's tokens come in the order of its logits."""
    import torch
    B, K, V = 16, 8, 5000
    x, s = _make(B, K, V, torch.float32, seed=31, scale=scale)
    s = s * 1e4
    s[:, 1::2] = s[:, ::2]
    _, parents, tokens = ssd.beam_select(x, s, 64)
    for b in range(B):
        for i in range(K):
            mine = tokens[b][parents[b] == i].long()
            assert torch.equal(mine, torch.sort(x[b, i], descending=True, stable=True).indices[:len(mine)])


def test_scores_at_the_end_of_the_range(ssd):  # noqa: F811
    """Sums beyond float32 come out as infinities, in their right order."""
    import torch
    x = -1e37 * torch.arange(34, device="cuda", dtype=torch.float32).flip(0).repeat(1, 2, 1)
    s = torch.tensor([[-3e38, -2.9e38]], device="cuda")
    want = ref.beam_select(x, s, 64)
    scores, parents, tokens = ssd.beam_select(x, s, 64)
    assert torch.equal(parents.long(), want[1]) and torch.equal(tokens.long(), want[2])
    assert torch.equal(scores, want[0].float())


def _masked(x, kind):
    import torch
    V = x.shape[-1]
    t = torch.arange(V, device="cuda")
    if isinstance(kind, float):
        open_ = torch.rand(V, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") < kind
    else:
        open_ = {"runs": t % 256 < 128, "few": (t >= V // 3) & (t < V // 3 + 20), "last": t == V - 1,
                 "threads": t % 256 < 40, "one warp": t % 256 >= 32}[kind]
    return x.masked_fill(~open_, -torch.inf)


# the smaller batch takes slices of 2048 elements, the larger one of 4096
@pytest.mark.parametrize("B,K,V,dtype", [(1, 4, 9001, "float32"), (90, 4, 12289, "float32"), (40, 8, 8190, "bfloat16")])
@pytest.mark.parametrize("kind", [0.5, 0.1, 0.01, 0.001, "runs", "few", "last", "threads", "one warp"])
def test_masked_vocabularies(ssd, kind, B, K, V, dtype):  # noqa: F811
    """Constrained decoding: most tokens at -inf, at random and in patterns that leave some threads and
    warps without any; some beams ended or without a choice."""
    import torch
    x, s = _make(B, K, V, getattr(torch, dtype), seed=3)
    x = _masked(x, kind)
    x[0, 1] = -torch.inf
    f = torch.zeros(B, K, dtype=torch.bool, device="cuda")
    f[0, 2] = f[-1, 0] = True
    for keep in (1, 16, 64):
        _same(ssd.beam_select(x, s, keep, finished=f, pad_token=3), ref.beam_select(x, s, keep, f, 3))


@pytest.mark.parametrize("V", [4095, 4096, 8191, 8192, 12289])
def test_wide_slices(ssd, V):  # noqa: F811
    """Borders of the slices of 4096 elements; equal and rounded logits, of which more reach the bound
    than are ranked."""
    import torch
    x, s = _make(80, 4, V, torch.float32, seed=V)
    x[1] = 0.0
    x[2] = torch.round(x[2])
    x[3] = x[3, :1]
    s[3] = -1.0
    x[4] = torch.round(x[4] / 4)
    x[5, :, :100] = 3.0
    for keep in (1, 9, 64):
        _same(ssd.beam_select(x, s, keep), ref.beam_select(x, s, keep))


def _time(f):
    """Microseconds of a call in a replayed graph: the least of five runs of twenty."""
    import torch
    f()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    graph.replay()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 50)
    return best


@pytest.mark.parametrize("B,K,keep", [(1, 4, 8), (64, 8, 16)])
def test_masks_cost_little(ssd, B, K, keep):  # noqa: F811
    """A masked vocabulary takes no more than twice the time of an open one (ranking what is at -inf
    took ten to sixty times as long)."""
    import torch
    x, s = _make(B, K, 50277, torch.float32, seed=6)
    whole = _time(lambda: ssd.beam_select(x, s, keep))
    for kind in (0.5, 0.01, 0.001, "runs", "few", "threads"):
        y = _masked(x, kind)
        assert _time(lambda: ssd.beam_select(y, s, keep)) <= 2 * whole, kind


@pytest.mark.parametrize("shape", [(1,), (3,), (4, 1791), (8193,), (20001,)])
def test_reorder_slots_of_odd_elements(ssd, shape):  # noqa: F811
    """Slots of two-byte elements that are off four bytes, contiguous and in wider rows."""
    import torch
    n = 12
    row = 1
    for d in shape:
        row *= d
    wide = torch.randn(n, row + 1, device="cuda").half()
    caches = [torch.randn(n, *shape, device="cuda").bfloat16(), wide[:, 1:], wide.clone()[:, :row]]
    slots = torch.arange(n, dtype=torch.int32, device="cuda").view(3, 4)
    parents = torch.tensor([[1, 1, 2, 3], [0, 0, 0, 0], [3, 2, 2, 3]], dtype=torch.int32, device="cuda")
    want, copies = ref.beam_reorder(slots, parents)
    after = [c.clone() for c in caches]
    for c in after:
        for frm, to in copies:
            c[to] = c[frm]
    edge = wide[:, :1].clone()
    assert ssd.beam_reorder(caches, slots, parents).tolist() == want
    for c, a in zip(caches, after):
        assert torch.equal(c, a)
    assert torch.equal(wide[:, :1], edge)


def test_reorder_moves_two_bytes_at_a_time(ssd):  # noqa: F811
    """Odd numbers of two-byte elements go faster than as many single bytes."""
    import torch
    n, row = 64, 400001
    slots = torch.arange(n, dtype=torch.int32, device="cuda").view(16, 4)
    parents = torch.tensor([[0, 0, 1, 1]] * 16, dtype=torch.int32, device="cuda")
    two = [torch.zeros(n, row, device="cuda", dtype=torch.bfloat16)]
    one = [torch.zeros(n, 2 * row + 1, device="cuda", dtype=torch.uint8)]
    assert _time(lambda: ssd.beam_reorder(two, slots, parents)) <= 0.9 * _time(lambda: ssd.beam_reorder(one, slots, parents))
