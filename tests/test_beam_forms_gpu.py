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
