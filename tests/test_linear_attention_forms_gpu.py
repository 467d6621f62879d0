"""Linear attention: borders that are not what they should be, rows of no sequence, and which of the
kernels takes a call."""

import pytest

from test_linear_attention_gpu import _backward, _forward, _make, ssd  # noqa: F401  (ssd is the built package)

pytestmark = pytest.mark.gpu


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
