"""A residual block of a language model around the scan: one training step over packed
sequences, then a prompt and generated tokens from cached states.

    n, h      = norm(x + residual)
    z, u, dt  = n W_in                      (torch.matmul)
    x, B, C   = conv(u)                     short causal convolution, SiLU
    y         = scan(x, dt, B, C)
    out       = gated_norm(y, z) W_out      (torch.matmul)

Every step but the two projections is an operator of this package, forward and backward; the
gradients go straight into slices of the projection's gradient.  Run as

    python examples/mamba_block.py [--tokens 4096] [--heads 24]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_model_ssd_gb300 as ssd  # noqa: E402


class Block:
    """Parameters of one block (float32 norms and convolution, bfloat16 projections)."""

    def __init__(self, heads: int, headdim: int = 64, dstate: int = 128, groups: int = 1, width: int = 4,
                 d_model=None, delta_init: float = -4.6, dtype=torch.bfloat16, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.H, self.P, self.N, self.G, self.K = heads, headdim, dstate, groups, width
        self.inner, self.delta_init, self.dtype = heads * headdim, delta_init, dtype
        self.d_model = d_model or self.inner // 2
        self.channels = self.inner + 2 * groups * dstate
        # the step sizes take a multiple of 16 bytes, so that every slice of a row starts on one
        self.step_cols = -(-heads // 8) * 8
        self.split = ((heads, headdim), (groups, dstate), (groups, dstate))

        def normal(*shape, scale, dt=torch.float32):
            return (torch.randn(*shape, generator=gen, device=device) * scale).to(dt)

        cols = self.inner + self.channels + self.step_cols
        self.w_in = normal(self.d_model, cols, scale=self.d_model ** -0.5, dt=dtype)
        self.w_out = normal(self.inner, self.d_model, scale=self.inner ** -0.5, dt=dtype)
        self.conv_w = normal(self.channels, width, scale=width ** -0.5)
        self.conv_b = normal(self.channels, scale=0.1)
        self.norm_w = 1 + normal(self.d_model, scale=0.1)
        self.norm_b = normal(self.d_model, scale=0.1)
        self.gate_w = 1 + normal(self.inner, scale=0.1)

    def _slices(self, proj):
        """z, u and the raw step sizes of the projection's rows."""
        i, c = self.inner, self.channels
        return proj[..., :i], proj[..., i:i + c], proj[..., i + c:i + c + self.H]

    def forward(self, x, residual, cu_seqlens=None, conv_state=None, state=None, positions=None):
        """x ``[batch, L, d_model]``, residual float32.  Returns the block's output, the residual
        stream after it took x in, the final window and scan state, and what backward needs."""
        n, h, stats = ssd.norm_forward(x, self.norm_w, self.norm_b, residual=residual)
        proj = n @ self.w_in
        z, u, raw = self._slices(proj)
        raw = raw.float().contiguous()
        (xs, B, C), window = ssd.conv_forward(u, self.conv_w, self.conv_b, split=self.split,
                                              cu_seqlens=cu_seqlens, initial_state=conv_state,
                                              positions=positions, final_state=True)
        y, final = ssd.forward(xs, raw, B, C, self.delta_init, cu_seqlens=cu_seqlens, initial_state=state)
        gated, rstd = ssd.gated_norm_forward(y, z, self.gate_w)
        return gated @ self.w_out, h, window, final, (n, h, stats, proj, raw, xs, B, C, y, gated, rstd)

    def backward(self, d_out, d_h, saved, cu_seqlens=None):
        """Gradients of x, of the residual that came in, and of every parameter."""
        n, h, stats, proj, raw, xs, B, C, y, gated, rstd = saved
        z, u, _ = self._slices(proj)
        g = {"w_out": gated.flatten(0, 1).t() @ d_out.flatten(0, 1)}
        d_proj = torch.zeros_like(proj)
        dz, du, draw = self._slices(d_proj)
        gn = ssd.gated_norm_backward(d_out @ self.w_out.t(), y, z, self.gate_w, rstd, out={"dz": dz})
        gs = ssd.backward(xs, raw, B, C, gn["dy"], self.delta_init, cu_seqlens=cu_seqlens)
        draw.copy_(gs["d_raw_dt"])
        gc = ssd.conv_backward(u, self.conv_w, self.conv_b, (gs["dx"], gs["dB"], gs["dC"]),
                               cu_seqlens=cu_seqlens, out={"du": du})
        g["w_in"] = n.flatten(0, 1).t() @ d_proj.flatten(0, 1)
        nb = ssd.norm_backward(d_proj @ self.w_in.t(), h, self.norm_w, stats, dh=d_h)
        g.update(conv_w=gc["d_weight"], conv_b=gc["d_bias"], gate_w=gn["d_weight"], norm_w=nb["d_weight"],
                 norm_b=nb["d_bias"])
        return nb["dx"], nb["d_residual"], g

    def step(self, x, residual, conv_state, state, positions, slots=None):
        """One token for each row: x ``[batch, d_model]``; the states are updated in place."""
        n, h, _ = ssd.norm_forward(x, self.norm_w, self.norm_b, residual=residual, stats=False)
        z, u, raw = self._slices(n @ self.w_in)
        y = ssd.conv_decode_step(state, conv_state, u, raw.float().contiguous(), self.conv_w, self.conv_b,
                                 positions, self.delta_init, ngroups=self.G, slots=slots)
        gated, _ = ssd.gated_norm_forward(y, z, self.gate_w)
        return gated @ self.w_out, h


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=24)
    args = ap.parse_args()
    blk = Block(args.heads)
    T, D = args.tokens, blk.d_model
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, T, D, generator=gen, device="cuda").bfloat16()
    res = torch.randn(1, T, D, generator=gen, device="cuda")
    cu = torch.tensor([0, T // 5, T // 2, T], dtype=torch.int32, device="cuda")
    out, h, _, _, saved = blk.forward(x, res, cu)
    dx, dres, grads = blk.backward(torch.ones_like(out), torch.zeros_like(h), saved, cu)
    print("training step over %d tokens in 3 sequences: |dx| %.3g, |d residual| %.3g" %
          (T, dx.float().norm(), dres.norm()))
    for k, v in sorted(grads.items()):
        print("  d %-7s %-18s norm %.4g" % (k, list(v.shape), v.float().norm()))

    # a prompt, then its last tokens again one by one from the states before them
    n = min(T, 200)
    full, _, _, _, _ = blk.forward(x[:, :n], res[:, :n])
    _, _, window, state, _ = blk.forward(x[:, :n - 4], res[:, :n - 4])
    worst = 0.0
    for t in range(n - 4, n):
        pos = torch.full((1,), t, dtype=torch.int32, device="cuda")
        o, _ = blk.step(x[:, t], res[:, t], window, state, pos)
        worst = max(worst, float((o - full[:, t]).float().norm() / full[:, t].float().norm()))
    print("4 tokens after a prompt of %d, one by one against the whole prompt: off by %.2g" % (n - 4, worst))


if __name__ == "__main__":
    main()
