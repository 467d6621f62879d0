"""The block of examples/mamba_block.py: its operators together, forward and backward against
torch's own differentiation of the same formulas in 64 bits, and one token at a time against
the whole prompt."""

import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_ssd_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("mamba_block", os.path.join(ROOT, "examples", "mamba_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(blk, p, x, res, cuts):
    """The block token by token in 64 bits on the CPU, with torch's autograd."""
    import torch
    H, P, N, G, K = blk.H, blk.P, blk.N, blk.G, blk.K
    v = x + res
    mu = v.mean(-1, keepdim=True)
    n = (v - mu) / torch.sqrt(((v - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    proj = n @ p["w_in"]
    i, c = blk.inner, blk.channels
    z, u, raw = proj[:, :i], proj[:, i:i + c], proj[:, i + c:i + c + H]
    ys = []
    for lo, hi in zip(cuts, cuts[1:]):
        S = torch.zeros(H, P, N, dtype=torch.float64)
        pad = torch.cat([torch.zeros(K - 1, c, dtype=torch.float64), u[lo:hi]])
        for t in range(hi - lo):
            pre = p["conv_b"] + (p["conv_w"] * pad[t:t + K].t()).sum(-1)
            a = pre * torch.sigmoid(pre)
            xt = a[:i].view(H, P)
            B = a[i:i + G * N].view(G, N).repeat_interleave(H // G, 0)
            C = a[i + G * N:].view(G, N).repeat_interleave(H // G, 0)
            delta = torch.nn.functional.softplus(raw[lo + t] + blk.delta_init)
            S = torch.exp(-delta)[:, None, None] * S + (delta[:, None] * xt)[..., None] * B[:, None]
            ys.append((S * C[:, None]).sum(-1).reshape(-1))
    y = torch.stack(ys)
    g = y * z * torch.sigmoid(z)
    gated = g / torch.sqrt((g ** 2).mean(-1, keepdim=True) + 1e-5) * p["gate_w"]
    return gated @ p["w_out"], v


def test_block_against_autograd(example):
    """Float32 throughout (a bfloat16 chain would drown the comparison in its roundings)."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    blk = example.Block(4, headdim=16, dstate=16, groups=2, d_model=40, dtype=torch.float32)
    T, cuts = 75, [0, 30, 31, 75]
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, T, 40, generator=gen, device="cuda")
    res = torch.randn(1, T, 40, generator=gen, device="cuda")
    d_out = torch.randn(1, T, 40, generator=gen, device="cuda")
    d_h = torch.randn(1, T, 40, generator=gen, device="cuda")
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    out, h, _, _, saved = blk.forward(x, res, cu)
    dx, dres, g = blk.backward(d_out, d_h, saved, cu)
    names = ["w_in", "w_out", "conv_w", "conv_b", "norm_w", "norm_b", "gate_w"]
    p = {k: getattr(blk, k).double().cpu().requires_grad_() for k in names}
    x64 = x[0].double().cpu().requires_grad_()
    r64 = res[0].double().cpu().requires_grad_()
    o64, h64 = _reference(blk, p, x64, r64, cuts)
    ((o64 * d_out[0].double().cpu()).sum() + (h64 * d_h[0].double().cpu()).sum()).backward()

    def rel(a, b):
        b = b.detach().numpy()
        return np.abs(a.double().cpu().numpy().reshape(b.shape) - b).max() / np.abs(b).max()

    # a dozen float32 operators in a row, each good to a few 1e-6 of its largest value
    assert rel(out, o64) <= 1e-4 and rel(h, h64) <= 1e-6
    assert rel(dx, x64.grad) <= 1e-4 and rel(dres, r64.grad) <= 1e-4
    for k in names:
        assert rel(g[k], p[k].grad) <= 1e-4, k


@pytest.mark.parametrize("heads,groups", [(24, 1), (6, 2)])
def test_tokens_one_by_one(example, heads, groups):
    """bfloat16: the tokens after a prompt, from its states, give what the longer prompt gives
    (each within the roundings of a few bfloat16 tensors)."""
    import torch
    blk = example.Block(heads, groups=groups)
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, cut = 90, 71
    x = torch.randn(2, n, blk.d_model, generator=gen, device="cuda").bfloat16()
    res = torch.randn(2, n, blk.d_model, generator=gen, device="cuda")
    full, _, _, _, _ = blk.forward(x, res)
    _, _, window, state, _ = blk.forward(x[:, :cut].contiguous(), res[:, :cut].contiguous())
    # the two rows live in slots 2 and 0 of a cache; a third row is padding
    cache_s = torch.zeros(3, *state.shape[1:], device="cuda")
    cache_w = torch.zeros(3, *window.shape[1:], dtype=window.dtype, device="cuda")
    cache_s[[2, 0]], cache_w[[2, 0]] = state, window
    slots = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
    pad = torch.zeros(1, blk.d_model, device="cuda")
    for t in range(cut, n):
        pos = torch.full((3,), t, dtype=torch.int32, device="cuda")
        o, _ = blk.step(torch.cat([x[:, t], pad.bfloat16()]), torch.cat([res[:, t], pad]), cache_w, cache_s,
                        pos, slots)
        d = (o[:2] - full[:, t]).float().norm() / full[:, t].float().norm()
        assert float(d) <= 2e-2, t


def test_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["mamba_block.py", "--tokens", "300", "--heads", "8"])
    example.main()
    assert "one by one" in capsys.readouterr().out
