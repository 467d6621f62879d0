"""The operators around the scan in 64 bits, in numpy, token by token and row by row, for the
GPU tests; and the comparison they use."""

import numpy as np


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def conv(u, w, b, p0=0, before=None, silu=True):
    """One sequence u [n, C]: output, state rows [K, C] after it, and pre-activations."""
    n, C = u.shape
    K = w.shape[1]
    hist = {}
    if before is not None:
        for m in range(1, K + 1):
            hist[p0 - m] = before[(p0 - m) % K]
    for i in range(n):
        hist[p0 + i] = u[i]
    zero = np.zeros(C)
    pre = np.zeros((n, C))
    for i in range(n):
        pre[i] = b
        for j in range(K):
            pre[i] += w[:, K - 1 - j] * hist.get(p0 + i - j, zero)
    state = np.zeros((K, C))
    for p in range(p0 + n - K, p0 + n):
        state[p % K] = hist.get(p, zero)
    out = pre * sigmoid(pre) if silu else pre
    return out, state, pre


def conv_bwd(u, w, b, dout, p0=0, before=None, dstate=None, silu=True):
    """Reverse of conv: du, dw, db, d_before."""
    n, C = u.shape
    K = w.shape[1]
    _, _, pre = conv(u, w, b, p0, before, silu)
    s = sigmoid(pre)
    g = dout * s * (1 + pre * (1 - s)) if silu else dout
    hist = {p0 + i: u[i] for i in range(n)}
    for m in range(1, K + 1):
        hist[p0 - m] = before[(p0 - m) % K] if before is not None else np.zeros(C)
    d = {p: np.zeros(C) for p in hist}
    dw = np.zeros_like(w)
    for i in range(n):
        for j in range(K):
            d[p0 + i - j] += w[:, K - 1 - j] * g[i]
            dw[:, K - 1 - j] += g[i] * hist[p0 + i - j]
    if dstate is not None:
        for p in range(p0 + n - K, p0 + n):
            d[p] += dstate[p % K]
    du = np.stack([d[p0 + i] for i in range(n)]) if n else np.zeros((0, C))
    db4 = np.zeros((K, C))
    for m in range(1, K + 1):
        db4[(p0 - m) % K] = d[p0 - m]
    return du, dw, g.sum(0), db4


def norm(x, w, b, res, eps, layer):
    v = x + (res if res is not None else 0.0)
    mu = v.mean(-1, keepdims=True) if layer else np.zeros(v.shape[:-1] + (1,))
    rstd = 1.0 / np.sqrt(((v - mu) ** 2).mean(-1, keepdims=True) + eps)
    y = (v - mu) * rstd * w + (b if b is not None else 0.0)
    return y, v, np.concatenate([mu, rstd], -1)


def norm_bwd(dy, h, w, stats, dh, layer):
    mu, rstd = stats[:, :1], stats[:, 1:]
    xh = (h - mu) * rstd
    a = dy * w
    dv = a - xh * (a * xh).mean(-1, keepdims=True)
    if layer:
        dv = dv - a.mean(-1, keepdims=True)
    dv = dv * rstd + (dh if dh is not None else 0.0)
    return dv, (dy * xh).sum(0), dy.sum(0)


def gated(y, z, w, eps, groups):
    R, D = y.shape
    v = (y * z * sigmoid(z)).reshape(R, groups, D // groups)
    rstd = 1.0 / np.sqrt((v ** 2).mean(-1) + eps)
    return (v * rstd[..., None]).reshape(R, D) * w, rstd


def gated_bwd(dout, y, z, w, rstd, groups):
    R, D = y.shape
    s = sigmoid(z)
    gate = z * s
    xh = (y * gate).reshape(R, groups, -1) * rstd[..., None]
    a = (dout * w).reshape(R, groups, -1)
    dv = ((a - xh * (a * xh).mean(-1, keepdims=True)) * rstd[..., None]).reshape(R, D)
    return dv * gate, dv * y * s * (1 + z * (1 - s)), (dout * xh.reshape(R, D)).sum(0)


# A float32 result is a chain of a few dozen roundings of 2^-24 whose terms are no larger than
# a small multiple of the tensor's largest value; 128 of them bound it at every size here (the
# longest fixed-order chain is a 64-token run, then 8 and 32 partial sums).  The bfloat16 path's
# exponential and quotient are good to a few 2^-22, which the same bound holds.  A bfloat16
# result adds its own rounding, half of 2^-8 of the value; twice that covers a float32 value
# that lands on the other side of a rounding boundary.
CHAIN = 128 * 2.0 ** -24
ROUND = {"f32": 0.0, "bf16": 2.0 ** -8}


def assert_close(got, ref, dtype, what):
    got = got.detach().double().cpu().numpy().reshape(np.shape(ref))
    ref = np.asarray(ref, np.float64)
    assert np.isfinite(got).all(), what + ": not finite"
    if ref.size == 0:
        return
    top = np.abs(ref).max()
    bound = ROUND[dtype] * np.abs(ref) + CHAIN * top + 1e-30
    bad = np.abs(got - ref) - bound
    at = np.unravel_index(np.argmax(bad), bad.shape)
    assert bad[at] <= 0, "%s: %r instead of %r at %s (largest %r)" % (what, got[at], ref[at], at, top)
