"""Linear attention and beam search in 64 bits, written out plainly, and bounds of rounding."""

import torch

EPS32 = 2.0 ** -24   # half a step of float32, relative
EPS16 = 2.0 ** -8    # of bfloat16


def borders(batch, L, cu):
    return [i * L for i in range(batch + 1)] if cu is None else [int(x) for x in cu]


def attention(q, k, v, ld, scale, cuts, init=None):
    """o and final states of sequences ``cuts[s] .. cuts[s + 1]`` from all pairs of their tokens;
    differentiable.  Tokens outside the sequences have o = 0."""
    B, L, H, N = q.shape
    P, r = v.shape[3], H // k.shape[2]
    q, k, v = q.flatten(0, 1), k.flatten(0, 1).repeat_interleave(r, 1), v.flatten(0, 1).repeat_interleave(r, 1)
    parts, finals, at = [], [], 0
    for lo, hi in zip(cuts, cuts[1:]):
        parts.append(q.new_zeros(lo - at, H, P))
        n, at = hi - lo, hi
        t = torch.arange(n, dtype=torch.float64, device=q.device)
        gap = t[:, None] - t[None, :]
        a = torch.where(gap[..., None] >= 0, torch.exp(ld * gap[..., None].clamp(min=0).nan_to_num()), 0.0)
        a = torch.where((gap == 0)[..., None], torch.ones_like(a), a)   # 0 times -inf
        qs, ks, vs = q[lo:hi], k[lo:hi], v[lo:hi]
        o = torch.einsum("ihn,jhn,ijh,jhp->ihp", qs, ks, a, vs) if n else q.new_zeros(0, H, P)
        down = a[n - 1] if n else q.new_zeros(0, H)
        final = torch.einsum("jhp,jh,jhn->hpn", vs, down, ks) if n else q.new_zeros(H, P, N)
        if init is not None and n:
            o = o + torch.einsum("ihn,ih,hpn->ihp", qs, torch.exp(ld * (t[:, None] + 1)), init[len(finals)])
            final = final + torch.exp(ld * n)[:, None, None] * init[len(finals)]
        elif init is not None:
            final = init[len(finals)]
        parts.append(o)
        finals.append(final)
    parts.append(q.new_zeros(B * L - at, H, P))
    return scale * torch.cat(parts).view(B, L, H, P), torch.stack(finals)


def gradients(q, k, v, ld, scale, cuts, do, init=None, dfinal=None):
    """By torch's differentiation of the above."""
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    s = init.detach().clone().requires_grad_() if init is not None else None
    o, final = attention(*leaves, ld, scale, cuts, s)
    loss = (o * do).sum()
    if dfinal is not None:
        loss = loss + (final * dfinal).sum()
    loss.backward()
    return [t.grad for t in leaves] + ([s.grad] if s is not None else [])


def roundings(N, P, longest):
    """How many float32 roundings a term of any of the sums goes through, at most: products and
    sums over channels, over a block's tokens, over the chunks and segments of the states."""
    return 2 * max(N, P) + 2 * 128 + longest // 8 + 64


def beam_select(logits, scores, keep, finished=None, pad=0):
    """Scores in 64 bits, parents and tokens, candidate by candidate."""
    B, K, V = logits.shape
    out = []
    for b in range(B):
        cand = []
        for i in range(K):
            x = logits[b, i].double()
            s = scores[b, i].double().item()
            ended = finished is not None and bool(finished[b, i])
            z = torch.full_like(x, -torch.inf)
            if ended:
                if abs(s) < float("inf"):
                    z[pad] = s
            else:
                lse = torch.logsumexp(x, 0)
                if torch.isfinite(lse) and abs(s) < float("inf"):
                    z = s - lse + x
            cand.append(z)
        z = torch.cat(cand)
        order = torch.sort(z, descending=True, stable=True)
        out.append((order.values[:keep], order.indices[:keep] // V, order.indices[:keep] % V))
    return [torch.stack(x) for x in zip(*out)]


def beam_reorder(slots, parents):
    """New slots and the copies (from, to), beam by beam."""
    new, copies = [], []
    for row, par in zip(slots.tolist(), parents.tolist()):
        K = len(row)
        free = [row[i] for i in range(K) if i not in par]
        seen, n = set(), []
        for p in par:
            if not 0 <= p < K:
                n.append(-1)
            elif p in seen:
                n.append(free.pop(0))
                copies.append((row[p], n[-1]))
            else:
                n.append(row[p])
                seen.add(p)
        new.append(n)
    return new, copies
