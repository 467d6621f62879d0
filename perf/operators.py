"""The operators around the scan (short causal convolution, single-token step, norms) as cases
that can be timed and compared: inputs, one pass, the work it cannot do without, and its values
in 64 bits.

``own`` false: elementary torch operations in float32, rounded once at the end.  ``own`` true:
the calls a program makes of ``state_space_model_ssd_gb300``.
"""

from __future__ import annotations

import torch

own = False

DELTA_INIT = -4.6
EPS = 1e-5
_NO_LAYER_OF_OURS = 48 * 64  # a width that none of this package's workloads has: not drawn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the packed 64K-token batch of the 24-head layer: lengths from a few tokens to thousands,
        # every sequence continuing from a carried window (a chunked prompt)
        {"name": "conv_fwd_packed_64k", "op": "conv_fwd", "dtype": "bf16", "batch": 1, "seqlen": 65536,
         "nseq": 24, "heads": 24, "headdim": 64, "groups": 1, "dstate": 128, "width": 4, "state": True,
         "strided": True},
        # the last seven tokens of a prompt on the 80-head layer: latency
        {"name": "conv_fwd_tail", "op": "conv_fwd", "dtype": "bf16", "batch": 1, "seqlen": 7, "nseq": 0,
         "heads": 80, "headdim": 64, "groups": 1, "dstate": 128, "width": 4, "state": True,
         "strided": True},
        # the training step of the 80-head layer at 32K tokens; u is a slice of the projection's rows
        {"name": "conv_bwd_32k", "op": "conv_bwd", "dtype": "bf16", "batch": 1, "seqlen": 32768, "nseq": 0,
         "heads": 80, "headdim": 64, "groups": 1, "dstate": 128, "width": 4, "state": False,
         "strided": True},
        # float32 with an odd number of tokens and of channels, three taps, carried state
        {"name": "conv_bwd_odd_f32", "op": "conv_bwd", "dtype": "f32", "batch": 2, "seqlen": 333, "nseq": 0,
         "heads": 5, "headdim": 13, "groups": 1, "dstate": 16, "width": 3, "state": True,
         "strided": False},
        # one token for one user of the 80-head layer: latency
        {"name": "step_1", "op": "step", "dtype": "bf16", "batch": 1, "slots": 1, "heads": 80,
         "headdim": 64, "groups": 1, "dstate": 128, "width": 4},
        # one token for 128 rows of a serving batch (some of them padding) out of 160 cache slots
        {"name": "step_128", "op": "step", "dtype": "bf16", "batch": 128, "slots": 160, "heads": 80,
         "headdim": 64, "groups": 1, "dstate": 128, "width": 4},
        # the norm in front of the 80-head layer (d_model 2560) with a float32 residual stream
        {"name": "norm_fwd_32k", "op": "norm_fwd", "dtype": "bf16", "rows": 32768, "dim": 2560,
         "kind": "layer", "residual": "f32"},
        # the same for a handful of generated tokens: latency
        {"name": "norm_fwd_5", "op": "norm_fwd", "dtype": "bf16", "rows": 5, "dim": 2560, "kind": "rms",
         "residual": "bf16"},
        # its backward in training, the gradient of the residual stream added
        {"name": "norm_bwd_32k", "op": "norm_bwd", "dtype": "bf16", "rows": 32768, "dim": 2560,
         "kind": "layer", "residual": "f32"},
        # float32, odd row count and width, no residual
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "dtype": "f32", "rows": 517, "dim": 1001,
         "kind": "layer", "residual": "none"},
        # after the scan of the 2 x 2048-token, 24-head layer; z is a slice of the projection's rows
        {"name": "gated_fwd_4k", "op": "gated_fwd", "dtype": "bf16", "rows": 4096, "dim": 1536, "groups": 1,
         "strided": True},
        # the training step of the 80-head layer, eight norm groups
        {"name": "gated_bwd_32k", "op": "gated_bwd", "dtype": "bf16", "rows": 32768, "dim": 5120, "groups": 8,
         "strided": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["conv_fwd", "conv_bwd", "step", "norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op in ("conv_fwd", "conv_bwd"):
            heads = _log(rng, 1, 80)
            headdim, dstate = (64, rng.choice([64, 128])) if rng.random() < 0.7 else (rng.randint(1, 96),
                                                                                   rng.randint(1, 96))
            batch = rng.choice([1, 1, 2, 5])
            seqlen = _log(rng, 1, 65536)
            nseq = rng.choice([0, min(seqlen, _log(rng, 1, 60))]) if batch == 1 else 0
            c = {"op": op, "dtype": dtype, "batch": batch, "seqlen": seqlen, "nseq": nseq, "heads": heads,
                 "headdim": headdim, "groups": rng.choice([1, 1, 2]), "dstate": dstate,
                 "width": rng.choice([2, 3, 4, 4]), "state": rng.random() < 0.5,
                 "strided": rng.random() < 0.5}
        elif op == "step":
            batch = _log(rng, 1, 192)
            groups = rng.choice([1, 1, 2])
            c = {"op": op, "dtype": dtype, "batch": batch, "slots": batch + rng.randint(0, 9),
                 "heads": groups * _log(rng, 1, 40), "headdim": rng.choice([16, 32, 64, 64, 128]),
                 "groups": groups, "dstate": rng.choice([16, 64, 128, 128]),
                 "width": rng.choice([2, 3, 4, 4])}
        elif op in ("norm_fwd", "norm_bwd"):
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 65536),
                 "dim": rng.choice([_log(rng, 24, 8192), 64 * rng.randint(1, 47)]),
                 "kind": rng.choice(["layer", "rms"]), "residual": rng.choice(["none", dtype, "f32"])}
        else:
            groups = rng.choice([1, 1, 2, 8])
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 65536),
                 "dim": groups * rng.choice([_log(rng, 8, 960), 64 * rng.randint(1, 10)]), "groups": groups,
                 "strided": rng.random() < 0.5}
        sizes = [c.get("seqlen"), c.get("rows"), c.get("dim"), _channels(c) if "heads" in c else 0]
        if work(c)["bytes"] <= most and _NO_LAYER_OF_OURS not in sizes:
            return c


def _channels(c):
    return c["heads"] * c["headdim"] + 2 * c["groups"] * c["dstate"]


def _split(c):
    bc = (c["groups"], c["dstate"])
    return ((c["heads"], c["headdim"]), bc, bc)


def work(case):
    """Every input read once, every output written once; flops counted per element."""
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op in ("conv_fwd", "conv_bwd"):
        C, K = _channels(c), c["width"]
        T = c["batch"] * c["seqlen"]
        st = (c["nseq"] or c["batch"]) * K * C * e if c["state"] else 0
        par = C * (K + 1) * 4
        if op == "conv_fwd":
            return {"bytes": 2 * T * C * e + 2 * st + par, "flops": T * C * (2 * K + 5)}
        return {"bytes": 3 * T * C * e + 3 * st + 2 * par, "flops": T * C * (6 * K + 12)}
    if op == "step":
        C, K = _channels(c), c["width"]
        pn = c["heads"] * c["headdim"] * c["dstate"]
        row = 2 * 4 * pn + (K - 1 + 2) * C * e + c["heads"] * (4 + c["headdim"] * e)
        return {"bytes": c["batch"] * row + C * (K + 1) * 4, "flops": c["batch"] * (5 * pn + C * (2 * K + 5))}
    R, D = c["rows"], c["dim"]
    if op in ("norm_fwd", "norm_bwd"):
        r = SIZE.get(c["residual"], 0)
        if op == "norm_fwd":
            return {"bytes": R * D * (2 * e + 2 * r) + R * 8 + 2 * D * 4, "flops": 8 * R * D}
        both = r and c["residual"] != c["dtype"]
        return {"bytes": R * D * (2 * e + (r or e) + r + (r if both else 0)) + R * 8 + 4 * D * 4,
                "flops": 14 * R * D}
    g = c["groups"]
    if op == "gated_fwd":
        return {"bytes": 3 * R * D * e + R * g * 4 + D * 4, "flops": 10 * R * D}
    return {"bytes": 5 * R * D * e + R * g * 4 + 2 * D * 4, "flops": 22 * R * D}


# ------------------------------------------------------------------ inputs

def _lengths(total, n, seed):
    """n sequence lengths that add up to total: spread over a wide range, some of one token."""
    g = torch.Generator().manual_seed(seed + 17)
    w = torch.exp(2.0 * torch.randn(n, generator=g)).double()
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * (total - n)).long()
    cut[-1] = total - n
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)) + 1
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(lens, 0)]).to(torch.int32)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dt = DT[c["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    def uniform(*shape, scale):
        return (torch.rand(*shape, generator=gen, device=dev) * 2 - 1) * scale

    s = {"case": dict(c)}
    op = c["op"]
    if op in ("conv_fwd", "conv_bwd"):
        b, L, C, K = c["batch"], c["seqlen"], _channels(c), c["width"]
        if c["strided"]:  # a slice of the in-projection's rows: gate before it, step sizes after it
            inner = c["heads"] * c["headdim"]
            wide = normal(b, L, inner + C + c["heads"])
            s["u"] = wide[..., inner:inner + C]
        else:
            s["u"] = normal(b, L, C)
        s["weight"] = uniform(C, K, scale=K ** -0.5)
        s["bias"] = uniform(C, scale=K ** -0.5)
        s["cu"] = _lengths(L, c["nseq"], seed).to(dev) if c["nseq"] else None
        n = c["nseq"] or b
        s["init"] = normal(n, K, C) if c["state"] else None
        s["positions"] = (torch.randint(0, 5000, (n,), generator=gen, device=dev, dtype=torch.int32)
                          if c["state"] else None)
        if op == "conv_bwd":
            s["dy"] = tuple(normal(b, L, h, p) for h, p in _split(c))
            s["dfinal"] = normal(n, K, C) if c["state"] else None
    elif op == "step":
        b, n, C, K = c["batch"], c["slots"], _channels(c), c["width"]
        s["state"] = normal(n, c["heads"], c["headdim"], c["dstate"], scale=0.5, dtype=torch.float32)
        s["conv_state"] = normal(n, K, C)
        s["u"] = normal(b, C)
        s["raw_dt"] = normal(b, c["heads"], scale=0.5, dtype=torch.float32)
        s["weight"] = uniform(C, K, scale=K ** -0.5)
        s["bias"] = uniform(C, scale=K ** -0.5)
        s["positions"] = torch.randint(0, 5000, (b,), generator=gen, device=dev, dtype=torch.int32)
        slots = torch.randperm(n, generator=gen, device=dev)[:b].to(torch.int32)
        if b > 16:  # a batch padded to its captured size
            slots[-(b // 32):] = -1
        s["slots"] = slots
    elif op in ("norm_fwd", "norm_bwd"):
        R, D = c["rows"], c["dim"]
        rdt = DT.get(c["residual"])
        # a residual stream: a few channels much larger than the rest
        big = torch.where(torch.rand(D, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        s["weight"] = 1 + 0.1 * normal(D, dtype=torch.float32)
        s["bias"] = 0.1 * normal(D, dtype=torch.float32) if c["kind"] == "layer" else None
        if op == "norm_fwd":
            s["x"] = normal(R, D)
            s["residual"] = None if rdt is None else (normal(R, D, dtype=torch.float32) * big + 0.3).to(rdt)
        else:
            h = normal(R, D, dtype=torch.float32) * big + 0.3
            s["h"] = h.to(rdt or dt)
            s["dy"] = normal(R, D)
            s["dh"] = None if rdt is None else normal(R, D, dtype=rdt)
            h = s["h"].float()
            mean = h.mean(-1) if c["kind"] == "layer" else torch.zeros(R, device=dev)
            rstd = torch.rsqrt((h - mean[:, None]).square().mean(-1) + EPS)
            s["stats"] = torch.stack([mean, rstd], -1).contiguous()
    else:
        R, D, g = c["rows"], c["dim"], c["groups"]
        s["y"] = normal(R, D)
        if c["strided"]:
            s["z"] = normal(R, 2 * D + 192)[:, :D]
        else:
            s["z"] = normal(R, D)
        s["weight"] = 1 + 0.1 * normal(D, dtype=torch.float32)
        if op == "gated_bwd":
            s["dout"] = normal(R, D)
            z = s["z"].float()
            v = (s["y"].float() * z * torch.sigmoid(z)).view(R, g, D // g)
            s["rstd"] = torch.rsqrt(v.square().mean(-1) + EPS)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _own_conv_fwd(s):
    import state_space_model_ssd_gb300 as ssd
    outs, final = ssd.conv_forward(s["u"], s["weight"], s["bias"], split=_split(s["case"]), cu_seqlens=s["cu"],
                                   initial_state=s["init"], positions=s["positions"],
                                   final_state=s["case"]["state"])
    return {"outs": outs, "final": final}


def _own_conv_bwd(s):
    import state_space_model_ssd_gb300 as ssd
    return ssd.conv_backward(s["u"], s["weight"], s["bias"], s["dy"], cu_seqlens=s["cu"],
                             initial_state=s["init"], positions=s["positions"], d_final_state=s["dfinal"],
                             d_initial_state=s["case"]["state"])


def _own_step(s):
    import state_space_model_ssd_gb300 as ssd
    y = ssd.conv_decode_step(s["state"], s["conv_state"], s["u"], s["raw_dt"], s["weight"], s["bias"],
                             s["positions"], DELTA_INIT, ngroups=s["case"]["groups"], slots=s["slots"])
    return {"y": y, "state": s["state"], "conv_state": s["conv_state"]}


def _own_norm_fwd(s):
    import state_space_model_ssd_gb300 as ssd
    y, h, stats = ssd.norm_forward(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS,
                                   kind=s["case"]["kind"])
    return {"y": y, "h": h if s["residual"] is not None else None, "stats": stats}


def _own_norm_bwd(s):
    import state_space_model_ssd_gb300 as ssd
    return ssd.norm_backward(s["dy"], s["h"], s["weight"], s["stats"], dh=s["dh"], kind=s["case"]["kind"],
                             bias=s["bias"] is not None)


def _own_gated_fwd(s):
    import state_space_model_ssd_gb300 as ssd
    out, rstd = ssd.gated_norm_forward(s["y"], s["z"], s["weight"], eps=EPS, groups=s["case"]["groups"])
    return {"out": out, "rstd": rstd}


def _own_gated_bwd(s):
    import state_space_model_ssd_gb300 as ssd
    return ssd.gated_norm_backward(s["dout"], s["y"], s["z"], s["weight"], s["rstd"],
                                   groups=s["case"]["groups"])


def _window(s):
    """Per token: taps [T, C] for j = 0 .. K-1 back, in float32, and what the gather went by."""
    c = s["case"]
    K, C = c["width"], _channels(c)
    u = s["u"].float().reshape(-1, C)
    T = u.shape[0]
    t = torch.arange(T, device=u.device)
    if s["cu"] is not None:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:], t, right=True)
        start, end = cu[seq], cu[seq + 1]
    else:
        seq = t // c["seqlen"]
        start = seq * c["seqlen"]
        end = start + c["seqlen"]
    taps = [u]
    for j in range(1, K):
        inside = t - j >= start
        tap = torch.where(inside[:, None], u[(t - j).clamp(min=0)], torch.zeros((), device=u.device))
        if s["init"] is not None:
            row = torch.remainder(s["positions"].long()[seq] + t - start - j, K)
            tap = torch.where(inside[:, None], tap, s["init"][seq, row].float())
        taps.append(tap)
    return u, t, seq, start, end, taps


def _bounds(s, device):
    """First token, length and first position of each sequence."""
    c = s["case"]
    if s["cu"] is not None:
        cu = s["cu"].long()
        first, n = cu[:-1], torch.diff(cu)
    else:
        first = torch.arange(c["batch"], device=device) * c["seqlen"]
        n = torch.full_like(first, c["seqlen"])
    p0 = s["positions"].long() if s["positions"] is not None else torch.zeros_like(first)
    return first, n, p0


def _plain_conv_fwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    K = c["width"]
    u, t, seq, start, end, taps = _window(s)
    pre = s["bias"].float() + sum(s["weight"][:, K - 1 - j].float() * taps[j] for j in range(K))
    out = (pre * torch.sigmoid(pre)).to(dt)
    shape = s["u"].shape[:2]
    outs = tuple(p.contiguous().view(*shape, *d)
                 for p, d in zip(out.split([h * p for h, p in _split(c)], -1), _split(c)))
    final = None
    if c["state"]:
        first, n, p0 = _bounds(s, u.device)
        rows = []
        for r in range(K):  # the last position that falls on row r
            p = p0 + n - 1 - torch.remainder(p0 + n - 1 - r, K)
            here = p >= p0
            tok = u[(first + p - p0).clamp(min=0, max=u.shape[0] - 1)]
            rows.append(torch.where(here[:, None], tok, s["init"].float()[:, r]))
        final = torch.stack(rows, 1).to(dt)
    return {"outs": outs, "final": final}


def _plain_conv_bwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    K, C = c["width"], _channels(c)
    u, t, seq, start, end, taps = _window(s)
    T = u.shape[0]
    w = s["weight"].float()
    pre = s["bias"].float() + sum(w[:, K - 1 - j] * taps[j] for j in range(K))
    sig = torch.sigmoid(pre)
    dy = torch.cat([p.reshape(T, -1).float() for p in s["dy"]], -1)
    g = dy * sig * (1 + pre * (1 - sig))
    du = g * w[:, K - 1]
    for j in range(1, K):
        ok = t + j < end
        du = du + torch.where(ok[:, None], g[(t + j).clamp(max=T - 1)] * w[:, K - 1 - j],
                              torch.zeros((), device=u.device))
    dw = torch.stack([(g * taps[K - 1 - k]).sum(0) for k in range(K)], 1)
    out = {"d_weight": dw, "d_bias": g.sum(0)}
    if c["state"]:
        first, n, p0 = _bounds(s, u.device)
        df = s["dfinal"].float()
        d0 = torch.zeros(df.shape, device=u.device)
        seqs = torch.arange(df.shape[0], device=u.device)
        for m in range(0, K):
            # position p0 + n - 1 - m, among the last K: in this call's tokens, or the carried state's
            p = p0 + n - 1 - m
            row = torch.remainder(p, K)
            d = df[seqs, row]
            here, none = (p >= p0)[:, None], torch.zeros((), device=u.device)
            du.index_add_(0, (first + p - p0).clamp(min=0, max=T - 1), torch.where(here, d, none))
            d0[seqs, row] += torch.where(here, none, d)
        for m in range(1, K):
            row = torch.remainder(p0 - m, K)
            for i in range(0, K - m):
                ok = (i < n)[:, None]
                d0[seqs, row] += torch.where(ok, g[(first + i).clamp(max=T - 1)] * w[:, K - 1 - (i + m)],
                                             torch.zeros((), device=u.device))
        out["d_initial_state"] = d0.to(dt)
    out["du"] = du.to(dt).view(s["u"].shape)
    return out


def _plain_step(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    H, P, G, N, K = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
    # a padding row repeats row 0 (which is never one), so that no write of its own is needed
    live = s["slots"] >= 0
    row = torch.where(live, torch.arange(c["batch"], device=live.device), 0)
    slot, pos = s["slots"].long()[row], s["positions"].long()[row]
    u = s["u"].float()[row]
    w = s["weight"].float()
    pre = s["bias"].float() + w[:, K - 1] * u
    for j in range(1, K):
        pre = pre + w[:, K - 1 - j] * s["conv_state"][slot, torch.remainder(pos - j, K)].float()
    s["conv_state"][slot, torch.remainder(pos, K)] = s["u"][row]
    v = pre * torch.sigmoid(pre)
    x, B, C = v.split([H * P, G * N, G * N], -1)
    x = x.view(-1, H, P)
    B = B.view(-1, G, N).repeat_interleave(H // G, 1)
    C = C.view(-1, G, N).repeat_interleave(H // G, 1)
    zz = s["raw_dt"][row] + DELTA_INIT
    delta = torch.clamp(zz, min=0) + torch.log1p(torch.exp(-zz.abs()))
    S = torch.exp(-delta)[..., None, None] * s["state"][slot] + (delta[..., None] * x)[..., None] * B[..., None, :]
    s["state"][slot] = S
    y = torch.where(live[:, None, None], (S * C[..., None, :]).sum(-1), torch.zeros((), device=u.device))
    return {"y": y.to(dt), "state": s["state"], "conv_state": s["conv_state"]}


def _plain_norm_fwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    v = s["x"].float()
    h = None
    if s["residual"] is not None:
        v = v + s["residual"].float()
        h = v.to(s["residual"].dtype)
    mean = v.mean(-1, keepdim=True) if c["kind"] == "layer" else torch.zeros(v.shape[0], 1, device=v.device)
    d = v - mean
    rstd = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    y = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(dt), "h": h, "stats": torch.cat([mean, rstd], -1)}


def _plain_norm_bwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    dy, h = s["dy"].float(), s["h"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (h - mean) * rstd
    wd = dy * s["weight"].float()
    dv = wd - xh * (wd * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dv = dv - wd.mean(-1, keepdim=True)
    dv = dv * rstd
    if s["dh"] is not None:
        dv = dv + s["dh"].float()
    out = {"dx": dv.to(dt), "d_weight": (dy * xh).sum(0)}
    if s["bias"] is not None:
        out["d_bias"] = dy.sum(0)
    if s["dh"] is not None:
        out["d_residual"] = dv.to(s["dh"].dtype)
    return out


def _plain_gated_fwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    R, D, g = c["rows"], c["dim"], c["groups"]
    z = s["z"].float()
    v = (s["y"].float() * z * torch.sigmoid(z)).view(R, g, D // g)
    rstd = torch.rsqrt(v.square().mean(-1) + EPS)
    out = (v * rstd[..., None]).view(R, D) * s["weight"].float()
    return {"out": out.to(dt), "rstd": rstd}


def _plain_gated_bwd(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    R, D, g = c["rows"], c["dim"], c["groups"]
    y, z, do = s["y"].float(), s["z"].float(), s["dout"].float()
    sig = torch.sigmoid(z)
    gate = z * sig
    rstd = s["rstd"][..., None]
    xh = (y * gate).view(R, g, D // g) * rstd
    wd = (do * s["weight"].float()).view(R, g, D // g)
    dv = ((wd - xh * (wd * xh).mean(-1, keepdim=True)) * rstd).view(R, D)
    return {"dy": (dv * gate).to(dt), "dz": (dv * y * sig * (1 + z * (1 - sig))).to(dt),
            "d_weight": (do * xh.view(R, D)).sum(0)}


_own = {"conv_fwd": _own_conv_fwd, "conv_bwd": _own_conv_bwd, "step": _own_step, "norm_fwd": _own_norm_fwd,
        "norm_bwd": _own_norm_bwd, "gated_fwd": _own_gated_fwd, "gated_bwd": _own_gated_bwd}
_plain = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "step": _plain_step,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "gated_fwd": _plain_gated_fwd,
          "gated_bwd": _plain_gated_bwd}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv_fwd": _exact_conv, "conv_bwd": _exact_conv, "step": _exact_step, "norm_fwd": _exact_norm_fwd,
            "norm_bwd": _exact_norm_bwd, "gated_fwd": _exact_gated, "gated_bwd": _exact_gated}[case["op"]](s)


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_conv(s):
    """One sequence at a time: the carried tokens in front of its own, then the sum over taps."""
    c = s["case"]
    K, C, L = c["width"], _channels(c), c["seqlen"]
    bwd = c["op"] == "conv_bwd"
    w, b = s["weight"].double(), s["bias"].double()
    flat = s["u"].reshape(-1, C)
    T = flat.shape[0]
    cuts = s["cu"].tolist() if s["cu"] is not None else [i * L for i in range(c["batch"] + 1)]
    widths = [h * p for h, p in _split(c)]
    out = torch.empty(T, C, dtype=torch.float64, device=flat.device)
    state = torch.zeros(len(cuts) - 1, K, C, dtype=torch.float64, device=flat.device)
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    if bwd:
        dy = torch.cat([p.reshape(T, -1) for p in s["dy"]], -1)
    for q in range(len(cuts) - 1):
        lo, hi = cuts[q], cuts[q + 1]
        p0 = int(s["positions"][q]) if c["state"] else 0
        before = torch.zeros(K, C, dtype=torch.float64, device=flat.device)  # positions p0-K .. p0-1
        if c["state"]:
            order = [(p0 - K + i) % K for i in range(K)]
            before = s["init"][q].double()[order]
        ext = torch.cat([before, flat[lo:hi].double()])  # token i at K + i
        n = hi - lo
        pre = b.expand(n, C).clone()
        for k in range(K):
            pre.addcmul_(ext[k + 1:k + 1 + n], w[:, k].expand(n, C))
        if not bwd:
            out[lo:hi] = _silu64(pre)
            for i in range(K):
                state[q, (p0 + n - K + i) % K] = ext[n + i]
            continue
        e = torch.exp(-pre)
        g = dy[lo:hi].double() * (1 / (1 + e) + pre * e / (1 + e) ** 2)
        g = torch.where(torch.isfinite(e), g, torch.zeros_like(g))
        dext = torch.zeros_like(ext)
        for k in range(K):
            dext[k + 1:k + 1 + n] += g * w[:, k]
            dw[:, k] += (g * ext[k + 1:k + 1 + n]).sum(0)
        db += g.sum(0)
        if c["state"]:
            for i in range(K):
                dext[n + i] += s["dfinal"][q, (p0 + n - K + i) % K].double()
            for i in range(K):
                state[q, (p0 - K + i) % K] = dext[i]
        out[lo:hi] = dext[K:]
    if bwd:
        r = {"d_weight": dw, "d_bias": db, "du": out.view(s["u"].shape)}
        if c["state"]:
            r["d_initial_state"] = state
        return r
    outs = tuple(p.reshape(*s["u"].shape[:2], *d) for p, d in zip(out.split(widths, -1), _split(c)))
    return {"outs": outs, "final": state if c["state"] else None}


def _exact_step(s):
    c = s["case"]
    H, P, G, N, K = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
    state, window = s["state"].double(), s["conv_state"].double()
    y = torch.zeros(c["batch"], H, P, dtype=torch.float64, device=state.device)
    w, b = s["weight"].double(), s["bias"].double()
    slots, pos = s["slots"].tolist(), s["positions"].tolist()
    for i in range(c["batch"]):
        q, p = slots[i], pos[i]
        if q < 0:
            continue
        window[q, p % K] = s["u"][i].double()
        v = b.clone()
        for k in range(K):
            v += w[:, k] * window[q, (p + 1 + k - K) % K]
        v = _silu64(v)
        x, B, C = v[:H * P].view(H, P), v[H * P:H * P + G * N].view(G, N), v[H * P + G * N:].view(G, N)
        delta = torch.log1p(torch.exp(s["raw_dt"][i].double() + DELTA_INIT))
        for g in range(G):
            hs = slice(g * (H // G), (g + 1) * (H // G))
            state[q, hs] *= torch.exp(-delta[hs])[:, None, None]
            state[q, hs] += torch.einsum("h,hp,n->hpn", delta[hs], x[hs], B[g])
            y[i, hs] = state[q, hs] @ C[g]
    return {"y": y, "state": state, "conv_state": window}


def _exact_norm_fwd(s):
    v = s["x"].double()
    h = None
    if s["residual"] is not None:
        v = h = v + s["residual"].double()
    mean = v.mean(-1) if s["case"]["kind"] == "layer" else v.new_zeros(v.shape[0])
    var = ((v - mean[:, None]) ** 2).mean(-1)
    rstd = (var + EPS) ** -0.5
    y = (v - mean[:, None]) * rstd[:, None] * s["weight"].double()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return {"y": y, "h": h, "stats": torch.stack([mean, rstd], -1)}


def _exact_norm_bwd(s):
    """dv = J^T (w dy) with J = rstd (I - 1 1^T / D - xh xh^T / D)."""
    dy, h, st = s["dy"].double(), s["h"].double(), s["stats"].double()
    D = dy.shape[1]
    xh = (h - st[:, :1]) * st[:, 1:]
    a = dy * s["weight"].double()
    dot = torch.einsum("rd,rd->r", a, xh) / D
    dv = a - dot[:, None] * xh
    if s["case"]["kind"] == "layer":
        dv = dv - (a.sum(-1) / D)[:, None]
    dv = dv * st[:, 1:]
    if s["dh"] is not None:
        dv = dv + s["dh"].double()
    out = {"dx": dv, "d_weight": torch.einsum("rd,rd->d", dy, xh)}
    if s["bias"] is not None:
        out["d_bias"] = dy.sum(0)
    if s["dh"] is not None:
        out["d_residual"] = dv
    return out


def _exact_gated(s):
    c = s["case"]
    R, D, g = c["rows"], c["dim"], c["groups"]
    n = D // g
    y, z, w = s["y"].double(), s["z"].double(), s["weight"].double()
    gate = _silu64(z)
    outs, stats, dys, dzs, dws = [], [], [], [], []
    for k in range(g):
        at = slice(k * n, (k + 1) * n)
        v = y[:, at] * gate[:, at]
        if c["op"] == "gated_fwd":
            rstd = (torch.einsum("rd,rd->r", v, v) / n + EPS) ** -0.5
            outs.append(v * rstd[:, None] * w[at])
            stats.append(rstd)
            continue
        rstd = s["rstd"][:, k].double()[:, None]
        xh = v * rstd
        do = s["dout"][:, at].double()
        a = do * w[at]
        dv = rstd * (a - xh * (torch.einsum("rd,rd->r", a, xh) / n)[:, None])
        e = torch.exp(-z[:, at])
        dys.append(dv * gate[:, at])
        dzs.append(dv * y[:, at] * (1 / (1 + e) + z[:, at] * e / (1 + e) ** 2))
        dws.append(torch.einsum("rd,rd->d", do, xh))
    if c["op"] == "gated_fwd":
        return {"out": torch.cat(outs, 1), "rstd": torch.stack(stats, 1)}
    return {"dy": torch.cat(dys, 1), "dz": torch.cat(dzs, 1), "d_weight": torch.cat(dws)}
