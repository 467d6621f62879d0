"""Linear attention with a decay for each head (prompts, their backward, single tokens) and beam
search over cached states (selection, reordering of cache slots) as cases that can be timed and
compared: inputs, one pass, the work it cannot do without, and its values in 64 bits.

``own`` false: elementary torch operations in float32 (in float64 where borders between
candidates and powers of far positions need it), rounded once at the end.  ``own`` true: the
calls a program makes of ``state_space_model_ssd_gb300``.
"""

from __future__ import annotations

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
CHUNK = 128  # tokens per diagonal block of the plain form


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a 32K-token document through the 80-head layer (values of 64, keys of 128 channels);
        # q, k and v are slices of one projection's rows
        {"name": "attn_fwd_32k", "op": "attn_fwd", "dtype": "bf16", "batch": 1, "seqlen": 32768, "nseq": 0,
         "heads": 80, "groups": 80, "headdim": 64, "dstate": 128, "state": False, "strided": True},
        # the packed 64K-token batch of the 24-head layer: prompts of a few to thousands of tokens,
        # each continuing from a carried state
        {"name": "attn_fwd_packed_64k", "op": "attn_fwd", "dtype": "bf16", "batch": 1, "seqlen": 65536,
         "nseq": 24, "heads": 24, "groups": 24, "headdim": 64, "dstate": 64, "state": True,
         "strided": False},
        # the last seven tokens of a prompt on the 80-head layer: latency
        {"name": "attn_fwd_tail", "op": "attn_fwd", "dtype": "bf16", "batch": 1, "seqlen": 7, "nseq": 0,
         "heads": 80, "groups": 80, "headdim": 64, "dstate": 128, "state": True, "strided": True},
        # the training step of the 80-head layer at 32K tokens
        {"name": "attn_bwd_32k", "op": "attn_bwd", "dtype": "bf16", "batch": 1, "seqlen": 32768, "nseq": 0,
         "heads": 80, "groups": 80, "headdim": 64, "dstate": 128, "state": False, "strided": True},
        # training with keys and values shared by four heads each, 128 x 128 states, carried states
        # and their gradients (a sequence trained in pieces)
        {"name": "attn_bwd_shared_8k", "op": "attn_bwd", "dtype": "bf16", "batch": 2, "seqlen": 4096,
         "nseq": 0, "heads": 32, "groups": 8, "headdim": 128, "dstate": 128, "state": True,
         "strided": False},
        # float32 with odd sizes everywhere
        {"name": "attn_bwd_odd_f32", "op": "attn_bwd", "dtype": "f32", "batch": 2, "seqlen": 333, "nseq": 0,
         "heads": 5, "groups": 5, "headdim": 13, "dstate": 21, "state": True, "strided": False},
        # one token for one user of the 80-head layer: latency
        {"name": "attn_step_1", "op": "attn_step", "dtype": "bf16", "batch": 1, "slots": 1, "heads": 80,
         "groups": 80, "headdim": 64, "dstate": 128},
        # one token for 128 rows of a serving batch (some of them padding) out of 160 cache slots
        {"name": "attn_step_128", "op": "attn_step", "dtype": "bf16", "batch": 128, "slots": 160, "heads": 80,
         "groups": 80, "headdim": 64, "dstate": 128},
        # one user with four beams over a vocabulary of odd size: latency
        {"name": "select_1x4", "op": "select", "dtype": "bf16", "batch": 1, "beams": 4, "vocab": 50277,
         "keep": 8, "strided": False},
        # 64 users with eight beams, twice as many candidates kept (some will have ended); the
        # logits are a slice of a head padded to a multiple of 64 columns
        {"name": "select_64x8", "op": "select", "dtype": "f32", "batch": 64, "beams": 8, "vocab": 50277,
         "keep": 16, "strided": True},
        # one user with four beams, one of them doubled, four layers of eight heads: latency
        {"name": "reorder_1x4", "op": "reorder", "dtype": "bf16", "batch": 1, "beams": 4, "copies": 1,
         "layers": 4, "heads": 8, "headdim": 64, "dstate": 64, "channels": 0},
        # 16 users with four beams, half of the beams replaced, the states and windows of 24 layers
        # of 24 heads
        {"name": "reorder_16x4", "op": "reorder", "dtype": "bf16", "batch": 16, "beams": 4, "copies": 2,
         "layers": 24, "heads": 24, "headdim": 64, "dstate": 128, "channels": 1792},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "select", "reorder"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if op == "reorder":
            beams = rng.randint(2, 16)
            c = {"op": op, "dtype": dtype, "batch": _log(rng, 1, 32), "beams": beams,
                 "copies": rng.randint(1, beams - 1), "layers": _log(rng, 1, 24), "heads": _log(rng, 1, 80),
                 "headdim": rng.choice([64, 64, 128, rng.randint(5, 100)]),
                 "dstate": rng.choice([64, 128, rng.randint(5, 100)]),
                 "channels": rng.choice([0, _log(rng, 16, 6000)])}
            if 2 * c["beams"] * c["batch"] * work(c)["bytes"] / (c["copies"] * c["batch"]) > 40e9:
                continue
        elif op == "select":
            beams = _log(rng, 1, 16)
            c = {"op": op, "dtype": dtype, "batch": _log(rng, 1, 128), "beams": beams,
                 "vocab": _log(rng, 300, 131072), "keep": beams * rng.choice([1, 2]),
                 "strided": rng.random() < 0.5}
            if c["batch"] * beams * c["vocab"] > 64 * 8 * 65536:
                continue
        else:
            heads = _log(rng, 1, 80)
            groups = heads if rng.random() < 0.6 else rng.choice([g for g in range(1, heads + 1) if heads % g == 0])
            P, N = rng.choice([(64, 64), (64, 128), (128, 128), (128, 64), (64, 128), (128, 128),
                               (rng.randint(1, 128), rng.randint(1, 128))])
            c = {"op": op, "dtype": dtype, "batch": rng.choice([1, 1, 2, 5])}
            if op == "attn_step":
                c["batch"] = _log(rng, 1, 192)
                c["slots"] = c["batch"] + rng.randint(0, 9)
            else:
                c["seqlen"] = _log(rng, 1, 65536)
                c["nseq"] = min(c["seqlen"], _log(rng, 1, 60)) if c["batch"] == 1 and rng.random() < 0.5 else 0
            c |= {"heads": heads, "groups": groups, "headdim": P, "dstate": N}
            if op != "attn_step":
                c |= {"state": rng.random() < 0.5, "strided": rng.random() < 0.5}
                # float32 and sizes of any kind: what a tenth of the largest costs
                if (dtype == "f32" or P % 64 or N % 64) and work(c)["bytes"] > most / 10:
                    continue
        if work(c)["bytes"] <= most:
            return c


def work(case):
    """Every input read once, every output written once; flops of the recurrence."""
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "reorder":
        slot = c["layers"] * (c["heads"] * c["headdim"] * c["dstate"] * 4 + 4 * c["channels"] * e)
        return {"bytes": 2 * c["batch"] * c["copies"] * slot + 12 * c["batch"] * c["beams"], "flops": 0}
    if c["op"] == "select":
        n = c["batch"] * c["beams"]
        return {"bytes": n * (c["vocab"] * e + 4) + 12 * c["batch"] * c["keep"], "flops": 4 * n * c["vocab"]}
    H, G, P, N = c["heads"], c["groups"], c["headdim"], c["dstate"]
    if c["op"] == "attn_step":
        live = c["batch"] - (c["batch"] // 32 if c["batch"] > 16 else 0)
        row = 2 * 4 * H * P * N + (H * (N + P) + G * (N + P)) * e
        return {"bytes": live * row, "flops": 5 * live * H * P * N}
    T = c["batch"] * c["seqlen"]
    st = (c["nseq"] or c["batch"]) * H * P * N * 4 if c["state"] else 0
    if c["op"] == "attn_fwd":
        return {"bytes": T * (H + G) * (N + P) * e + 2 * st, "flops": 5 * T * H * P * N}
    return {"bytes": T * ((2 * N + P) * H + 2 * (N + P) * G) * e + 3 * st, "flops": 15 * T * H * P * N}


# ------------------------------------------------------------------ inputs

def _lengths(total, n, seed):
    """n sequence lengths that add up to total: spread over a wide range, some of one token."""
    g = torch.Generator().manual_seed(seed + 17)
    w = torch.exp(2.0 * torch.randn(n, generator=g)).double()
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * (total - n)).long()
    cut[-1] = total - n
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)) + 1
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(lens, 0)])


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dt = DT[c["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    s = {"case": dict(c)}
    op = c["op"]
    if op == "reorder":
        B, K = c["batch"], c["beams"]
        n = B * K + 3  # a cache with a few slots to spare
        s["slots"] = torch.randperm(n, generator=gen, device=dev)[:B * K].to(torch.int32).view(B, K)
        # the beams that go on, `copies` of them more than once
        kept = torch.rand(B, K, generator=gen, device=dev).argsort(-1)[:, :K - c["copies"]]
        again = torch.randint(0, kept.shape[1], (B, c["copies"]), generator=gen, device=dev)
        parents = torch.cat([kept, kept.gather(1, again)], 1)
        mixed = torch.rand(B, K, generator=gen, device=dev).argsort(-1)
        s["parents"] = parents.gather(1, mixed).to(torch.int32)
        s["caches"] = [normal(n, c["heads"], c["headdim"], c["dstate"], dtype=torch.float32)
                       for _ in range(c["layers"])]
        if c["channels"]:
            s["caches"] += [normal(n, 4, c["channels"]) for _ in range(c["layers"])]
        return s
    if op == "select":
        B, K, V = c["batch"], c["beams"], c["vocab"]
        wide = -(-V // 64) * 64 if c["strided"] else V
        s["logits"] = normal(B, K, wide, scale=2.5)[..., :V]
        s["scores"] = -5.0 + normal(B, K, scale=2.0, dtype=torch.float32)
        s["finished"] = torch.rand(B, K, generator=gen, device=dev) < 0.05
        return s
    H, G, P, N = c["heads"], c["groups"], c["headdim"], c["dstate"]
    # each head its own memory, from two tokens to thousands
    s["log_decay"] = -torch.exp2(-1.0 - 11.0 * torch.arange(H, device=dev) / max(1, H - 1)).float()
    s["scale"] = N ** -0.5
    if op == "attn_step":
        b, n = c["batch"], c["slots"]
        s["state"] = normal(n, H, P, N, scale=2.0, dtype=torch.float32)
        rows = normal(b, H * N + G * (N + P))  # a row of the projection
        s["q"] = rows[:, :H * N].unflatten(1, (H, N))
        s["k"] = rows[:, H * N:H * N + G * N].unflatten(1, (G, N))
        s["v"] = rows[:, H * N + G * N:].unflatten(1, (G, P))
        slots = torch.randperm(n, generator=gen, device=dev)[:b].to(torch.int32)
        if b > 16:  # a batch padded to its captured size
            slots[-(b // 32):] = -1
        s["slots"] = slots
        return s
    B, L = c["batch"], c["seqlen"]
    if c["strided"]:  # slices of one projection's rows
        rows = normal(B, L, H * N + G * (N + P))
        s["q"] = rows[..., :H * N].unflatten(2, (H, N))
        s["k"] = rows[..., H * N:H * N + G * N].unflatten(2, (G, N))
        s["v"] = rows[..., H * N + G * N:].unflatten(2, (G, P))
    else:
        s["q"], s["k"], s["v"] = normal(B, L, H, N), normal(B, L, G, N), normal(B, L, G, P)
    # the borders of the sequences, on the host too: a program packs them there
    s["borders"] = _lengths(L, c["nseq"], seed) if c["nseq"] else torch.arange(B + 1) * L
    s["cu"] = s["borders"].to(dev, torch.int32) if c["nseq"] else None
    n = c["nseq"] or B
    s["init"] = normal(n, H, P, N, dtype=torch.float32) if c["state"] else None
    if op == "attn_bwd":
        s["do"] = normal(B, L, H, P)
        s["dfinal"] = normal(n, H, P, N, dtype=torch.float32) if c["state"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _own_attn_fwd(s):
    import state_space_model_ssd_gb300 as ssd
    o, final = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                            cu_seqlens=s["cu"], initial_state=s["init"],
                                            final_state=s["case"]["state"])
    return {"o": o, "final": final}


def _own_attn_bwd(s):
    import state_space_model_ssd_gb300 as ssd
    return ssd.linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                         cu_seqlens=s["cu"], initial_state=s["init"],
                                         d_final_state=s["dfinal"], d_initial_state=s["case"]["state"])


def _own_attn_step(s):
    import state_space_model_ssd_gb300 as ssd
    o = ssd.linear_attention_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                  slots=s["slots"])
    return {"o": o, "state": s["state"]}


def _own_select(s):
    import state_space_model_ssd_gb300 as ssd
    scores, parents, tokens = ssd.beam_select(s["logits"], s["scores"], s["case"]["keep"],
                                              finished=s["finished"], pad_token=0)
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _own_reorder(s):
    import state_space_model_ssd_gb300 as ssd
    slots = ssd.beam_reorder(s["caches"], s["slots"], s["parents"])
    return {"slots": slots, "caches": s["caches"]}


def _chunks(s):
    """The tokens of every sequence in rows of CHUNK (the last one of a sequence filled up): each
    row's sequence, its first token's position there, its length, and the tokens' indices."""
    cu, dev = s["borders"], s["q"].device
    lens = torch.diff(cu)
    per = (lens + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lens)), per)
    pos = (torch.arange(len(seq)) - (torch.cumsum(per, 0) - per)[seq]) * CHUNK
    n = torch.clamp(lens[seq] - pos, max=CHUNK)
    at = (cu[seq] + pos)[:, None] + torch.arange(CHUNK)
    live = torch.arange(CHUNK) < n[:, None]
    at = torch.where(live, at, 0)
    return seq.to(dev), pos.to(dev), n.to(dev), at.to(dev), live.to(dev), lens.to(dev)


def _rows(t, at, live, heads):
    """[rows, heads, CHUNK, channels] in float32, zero where a row is filled up; shared heads repeated."""
    t = t.flatten(0, 1)
    t = t[at].float() * live[:, :, None, None]
    return t.permute(0, 2, 1, 3).repeat_interleave(heads // t.shape[2], 1)


def _powers(ld, e):
    """exp(ld e) for each head, a power's exponent taken in float64; zero where e is negative."""
    p = torch.exp(ld.double().view(-1, *[1] * e.dim()) * e.clamp(min=0).double()).float()
    return torch.where(e < 0, torch.zeros((), device=p.device), p)


def _entering(s, ld, seq, pos, n, local):
    """The states before each row from the rows' own, and the carried ones."""
    between = pos[:, None] - (pos + n)[None, :]
    between = torch.where(seq[:, None] == seq[None, :], between, -1)
    enter = torch.matmul(_powers(ld, between), local.flatten(2).transpose(0, 1))
    enter = enter.transpose(0, 1).view(local.shape)
    if s["init"] is not None:
        enter = enter + _powers(ld, pos).t()[..., None, None] * s["init"][seq]
    return enter


def _plain_attn_fwd(s):
    c, dt, ld = s["case"], DT[s["case"]["dtype"]], s["log_decay"]
    H = c["heads"]
    seq, pos, n, at, live, lens = _chunks(s)
    q, k, v = (_rows(s[x], at, live, H) for x in "qkv")
    i = torch.arange(CHUNK, device=q.device)
    o = ((q @ k.transpose(-1, -2)) * _powers(ld, i[:, None] - i[None, :])) @ v
    to_end = _powers(ld, n[:, None] - 1 - i[None, :]).transpose(0, 1)
    local = (v * to_end[..., None]).transpose(-1, -2) @ k
    enter = _entering(s, ld, seq, pos, n, local)
    o = o + _powers(ld, i + 1)[None, ..., None] * (q @ enter.transpose(-1, -2))
    o = (o * s["scale"]).permute(0, 2, 1, 3)
    out = torch.empty(c["batch"] * c["seqlen"], H, c["headdim"], dtype=dt, device=q.device)
    out[at[live]] = o[live].to(dt)
    final = None
    if c["state"]:
        last = pos + n == lens[seq]
        final = s["init"].clone()
        final[seq[last]] = (_powers(ld, n).t()[..., None, None] * enter + local)[last]
    return {"o": out.view(c["batch"], c["seqlen"], H, c["headdim"]), "final": final}


def _plain_attn_bwd(s):
    c, dt, ld, sc = s["case"], DT[s["case"]["dtype"]], s["log_decay"], s["scale"]
    H, G = c["heads"], c["groups"]
    seq, pos, n, at, live, lens = _chunks(s)
    q, k, v = (_rows(s[x], at, live, H) for x in "qkv")
    do = _rows(s["do"], at, live, H) * sc
    i = torch.arange(CHUNK, device=q.device)
    decay = _powers(ld, i[:, None] - i[None, :])
    to_end = _powers(ld, n[:, None] - 1 - i[None, :]).transpose(0, 1)[..., None]
    from_start = _powers(ld, i + 1)[None, ..., None]
    a = (q @ k.transpose(-1, -2)) * decay
    da = (do @ v.transpose(-1, -2)) * decay
    enter = _entering(s, ld, seq, pos, n, (v * to_end).transpose(-1, -2) @ k)
    # adjoints of the states after each row
    local = (do * from_start).transpose(-1, -2) @ q
    between = torch.where(seq[:, None] == seq[None, :], pos[None, :] - (pos + n)[:, None], -1)
    leave = torch.matmul(_powers(ld, between), local.flatten(2).transpose(0, 1)).transpose(0, 1).view(local.shape)
    if c["state"]:
        leave = leave + _powers(ld, lens[seq] - pos - n).t()[..., None, None] * s["dfinal"][seq]
    dq = da @ k + from_start * (do @ enter)
    dk = da.transpose(-1, -2) @ q + to_end * (v @ leave)
    dv = a.transpose(-1, -2) @ do + to_end * (k @ leave.transpose(-1, -2))
    out = {}
    for name, d, heads in (("dq", dq, H), ("dk", dk, G), ("dv", dv, G)):
        d = d.unflatten(1, (heads, H // heads)).sum(2).permute(0, 2, 1, 3)
        t = torch.empty(c["batch"] * c["seqlen"], heads, d.shape[-1], dtype=dt, device=d.device)
        t[at[live]] = d[live].to(dt)
        out[name] = t.view(c["batch"], c["seqlen"], heads, -1)
    if c["state"]:
        first = pos == 0
        d0 = s["dfinal"].clone()
        d0[seq[first]] = (_powers(ld, n).t()[..., None, None] * leave + local)[first]
        out["d_initial_state"] = d0
    return out


def _plain_attn_step(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    H, G = c["heads"], c["groups"]
    # a padding row repeats row 0 (which is never one), so that no write of its own is needed
    live = s["slots"] >= 0
    row = torch.where(live, torch.arange(c["batch"], device=live.device), 0)
    slot = s["slots"].long()[row]
    q = s["q"].float()[row]
    k = s["k"].float()[row].repeat_interleave(H // G, 1)
    v = s["v"].float()[row].repeat_interleave(H // G, 1)
    S = torch.exp(s["log_decay"])[:, None, None] * s["state"][slot] + v[..., None] * k[..., None, :]
    s["state"][slot] = S
    o = (S * q[..., None, :]).sum(-1) * s["scale"]
    return {"o": torch.where(live[:, None, None], o, torch.zeros((), device=o.device)).to(dt), "state": s["state"]}


def _plain_select(s):
    c = s["case"]
    B, V = c["batch"], c["vocab"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    x = x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    # a beam that has ended goes on with the padding token alone, at no cost
    pad = torch.arange(V, device=x.device) == 0
    low = torch.full((), -torch.inf, dtype=x.dtype, device=x.device)
    x = torch.where(s["finished"][..., None], torch.where(pad, 0.0, low), x)
    x = (x + s["scores"].double()[..., None]).view(B, -1)
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    at = order.indices[:, :c["keep"]]
    return {"scores": order.values[:, :c["keep"]].float(), "parents": (at // V).int(), "tokens": (at % V).int()}


def _plain_reorder(s):
    slots, parents = s["slots"].long(), s["parents"].long()
    K = slots.shape[1]
    i = torch.arange(K, device=slots.device)
    again = ((parents[:, :, None] == parents[:, None, :]) & (i[:, None] > i[None, :])).any(-1)
    goes_on = (parents[:, None, :] == i[None, :, None]).any(-1)
    free = torch.sort(goes_on.int(), dim=-1, stable=True).indices
    rank = (torch.cumsum(again.int(), -1) - 1).clamp(min=0)
    src = slots.gather(1, parents)
    new = torch.where(again, slots.gather(1, free.gather(1, rank)), src)
    to, frm = new[again], src[again]
    for t in s["caches"]:
        t[to] = t[frm]
    return {"slots": new.int(), "caches": s["caches"]}


_own = {"attn_fwd": _own_attn_fwd, "attn_bwd": _own_attn_bwd, "attn_step": _own_attn_step, "select": _own_select,
        "reorder": _own_reorder}
_plain = {"attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step,
          "select": _plain_select, "reorder": _plain_reorder}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn_fwd": _exact_attn, "attn_bwd": _exact_attn, "attn_step": _exact_step, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](s)


def _exact_attn(s):
    """The recurrence in blocks of 64 tokens, one sequence after the other; the gradients by its
    reverse, from the states that the forward left at the blocks' borders."""
    c = s["case"]
    H, G, P, N, Q = c["heads"], c["groups"], c["headdim"], c["dstate"], 64
    bwd, r = c["op"] == "attn_bwd", H // G
    T = c["batch"] * c["seqlen"]
    q, k, v = (s[x].reshape(T, -1, s[x].shape[-1]) for x in "qkv")
    do = s["do"].reshape(T, H, P) if bwd else None
    dev = q.device
    a = s["log_decay"].double()
    f64 = dict(dtype=torch.float64, device=dev)
    outs = {x: torch.empty(T, H, d, **f64) for x, d in ((("dq", N), ("dk", N), ("dv", P)) if bwd else (("o", P),))}
    cuts = s["borders"].tolist()
    state = torch.zeros(len(cuts) - 1, H, P, N, **f64)

    def heads(t, lo, hi):
        return t[lo:hi].double().transpose(0, 1).repeat_interleave(H // t.shape[1], 0)

    for b in range(len(cuts) - 1):
        S = s["init"][b].double() if c["state"] else torch.zeros(H, P, N, **f64)
        starts, kept = list(range(cuts[b], cuts[b + 1], Q)), []
        for lo in starts:
            hi = min(lo + Q, cuts[b + 1])
            m = hi - lo
            t = torch.arange(m, **f64)
            if bwd:
                kept.append(S)
            kk, vv = heads(k, lo, hi), heads(v, lo, hi)
            if not bwd:
                qq = heads(q, lo, hi) * s["scale"]
                gap = (t[:, None] - t[None, :]) * a[:, None, None]
                w = torch.exp(torch.where(t[:, None] >= t[None, :], gap, -torch.inf))
                o = torch.bmm(torch.bmm(qq, kk.transpose(1, 2)) * w, vv)
                o += torch.exp(a[:, None] * (t + 1))[..., None] * torch.bmm(qq, S.transpose(1, 2))
                outs["o"][lo:hi] = o.transpose(0, 1)
            kk = kk * torch.exp(a[:, None] * (m - 1 - t))[..., None]
            S = S * torch.exp(a * m)[:, None, None] + torch.bmm(vv.transpose(1, 2), kk)
        if not bwd:
            state[b] = S
            continue
        R = s["dfinal"][b].double() if c["state"] else torch.zeros(H, P, N, **f64)
        for lo, S in zip(reversed(starts), reversed(kept)):
            hi = min(lo + Q, cuts[b + 1])
            m = hi - lo
            t = torch.arange(m, **f64)
            qq, kk, vv = heads(q, lo, hi), heads(k, lo, hi), heads(v, lo, hi)
            dd = heads(do, lo, hi) * s["scale"]
            gap = (t[:, None] - t[None, :]) * a[:, None, None]
            w = torch.exp(torch.where(t[:, None] >= t[None, :], gap, -torch.inf))
            up = torch.exp(a[:, None] * (t + 1))[..., None]
            down = torch.exp(a[:, None] * (m - 1 - t))[..., None]
            A, dA = torch.bmm(qq, kk.transpose(1, 2)) * w, torch.bmm(dd, vv.transpose(1, 2)) * w
            outs["dq"][lo:hi] = (torch.bmm(dA, kk) + torch.bmm(dd * up, S)).transpose(0, 1)
            outs["dk"][lo:hi] = (torch.bmm(dA.transpose(1, 2), qq) + torch.bmm(vv * down, R)).transpose(0, 1)
            dv = torch.bmm(A.transpose(1, 2), dd) + torch.bmm(kk * down, R.transpose(1, 2))
            outs["dv"][lo:hi] = dv.transpose(0, 1)
            R = R * torch.exp(a * m)[:, None, None] + torch.bmm((dd * up).transpose(1, 2), qq)
        state[b] = R
    shape = (c["batch"], c["seqlen"])
    if not bwd:
        return {"o": outs["o"].view(*shape, H, P), "final": state if c["state"] else None}
    got = {"dq": outs["dq"].view(*shape, H, N)}
    for x, d in (("dk", N), ("dv", P)):
        got[x] = outs[x].view(*shape, G, r, d).sum(3)
    if c["state"]:
        got["d_initial_state"] = state
    return got


def _exact_step(s):
    c = s["case"]
    r = c["heads"] // c["groups"]
    state = s["state"].double()
    o = torch.zeros(c["batch"], c["heads"], c["headdim"], dtype=torch.float64, device=state.device)
    a = torch.exp(s["log_decay"].double())
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        k, v = s["k"][i].double(), s["v"][i].double()
        kv = torch.einsum("gp,gn->gpn", v, k).repeat_interleave(r, 0)
        state[slot] = a[:, None, None] * state[slot] + kv
        o[i] = torch.einsum("hpn,hn->hp", state[slot], s["q"][i].double()) * s["scale"]
    return {"o": o, "state": state}


def _exact_select(s):
    """One user at a time: the best by repeatedly taking the largest that is left."""
    c = s["case"]
    V, scores = c["vocab"], []
    for b in range(c["batch"]):
        x = s["logits"][b].double()
        x = x - torch.logsumexp(x, -1, keepdim=True)
        done = s["finished"][b]
        x[done] = -torch.inf
        x[done, 0] = 0.0
        x = (x + s["scores"][b].double()[:, None]).flatten()
        scores.append(torch.topk(x, c["keep"]).values)
    return {"scores": torch.stack(scores), "parents": None, "tokens": None}


def _exact_reorder(s):
    """Beam by beam on the host; the states in the type they have, which is exact."""
    caches = [t.double() for t in s["caches"]]
    new = s["slots"].tolist()
    for b, (slots, parents) in enumerate(zip(s["slots"].tolist(), s["parents"].tolist())):
        free = [x for i, x in enumerate(slots) if i not in parents]
        seen = set()
        for j, p in enumerate(parents):
            new[b][j] = slots[p]
            if p in seen:
                new[b][j] = free.pop(0)
                for t in caches:
                    t[new[b][j]] = t[slots[p]]
            seen.add(p)
    return {"slots": torch.tensor(new, dtype=torch.int32), "caches": caches}
