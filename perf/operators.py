"""The cases that the cache's rotary write and its eviction are measured on.

A case is a dict of plain values: `op` names the operator, the rest its sizes.

  rope     rotary positions applied to new queries and keys, and the write of
           keys and values into their slots of the paged cache
  weights  decode attention over the paged cache that also adds each cached
           token's attention weight to its running total
  select   which tokens of each sequence an eviction keeps
  compact  the kept tokens' keys, values and totals moved together into
           other pages

With `own` false `run` computes an operator in plain tensor operations; with
`own` true it makes the calls that a user of the package makes.
"""
import math

import torch

own = False

BLOCK = 16
FP8_MAX = 448.0
K_SCALE, V_SCALE = 0.0125, 0.015  # per-tensor scales of the FP8 pools (amax of N(0, 1) over 448)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: one new token each, 32 / 8 heads
        {"name": "rope_step_bf16", "op": "rope", "kv": "bf16", "T": 64, "Hq": 32, "H": 8, "D": 128,
         "rot": 128, "layout": "half", "scaling": "none", "far": 4096, "fused": True, "chunk": 1},
        # an 8192-token prefill packet at far positions, 64 / 8 heads, FP8 pages
        {"name": "rope_packet_fp8", "op": "rope", "kv": "fp8_e4m3", "T": 8192, "Hq": 64, "H": 8, "D": 128,
         "rot": 128, "layout": "half", "scaling": "yarn", "far": 131072, "fused": True, "chunk": 2048},
        # prompts of ragged length written with a scale per tile
        {"name": "rope_prompts_block", "op": "rope", "kv": "fp8_e4m3_block", "T": 2037, "Hq": 32, "H": 8, "D": 128,
         "rot": 128, "layout": "interleaved", "scaling": "bands", "far": 131072, "fused": False, "chunk": 509},
        # an odd number of tokens, small heads of which half is rotated
        {"name": "rope_part_fp16", "op": "rope", "kv": "fp16", "T": 1021, "Hq": 4, "H": 2, "D": 64,
         "rot": 32, "layout": "interleaved", "scaling": "linear", "far": 30000, "fused": False, "chunk": 100},
        # four short sequences: latency of the call
        {"name": "weights_tiny_fp16", "op": "weights", "kv": "fp16", "S": 4, "Hq": 4, "H": 2, "D": 64,
         "shortest": 17, "longest": 100},
        # an ordinary ragged decode batch
        {"name": "weights_ragged_bf16", "op": "weights", "kv": "bf16", "S": 64, "Hq": 32, "H": 8, "D": 128,
         "shortest": 512, "longest": 4096},
        # a full decode batch of FP8 pages, eight queries per key head
        {"name": "weights_many_fp8", "op": "weights", "kv": "fp8_e4m3", "S": 256, "Hq": 64, "H": 8, "D": 128,
         "shortest": 4096, "longest": 4096},
        # few sequences of the longest context
        {"name": "weights_long_fp8", "op": "weights", "kv": "fp8_e4m3", "S": 4, "Hq": 64, "H": 8, "D": 128,
         "shortest": 131072, "longest": 131072},
        # half of each ragged sequence is to go
        {"name": "select_ragged", "op": "select", "S": 64, "H": 8, "shortest": 512, "longest": 4096,
         "budget": 1024, "sinks": 4, "recent": 256},
        # long contexts cut to an eighth
        {"name": "select_long", "op": "select", "S": 4, "H": 8, "shortest": 131072, "longest": 131072,
         "budget": 16384, "sinks": 4, "recent": 1024},
        # the move that follows the ragged selection
        {"name": "compact_ragged_bf16", "op": "compact", "kv": "bf16", "S": 64, "H": 8, "D": 128,
         "shortest": 512, "longest": 4096, "budget": 1024},
        # long FP8 contexts with a scale per tile: tiles are scaled anew
        {"name": "compact_long_block", "op": "compact", "kv": "fp8_e4m3_block", "S": 4, "H": 8, "D": 128,
         "shortest": 131072, "longest": 131072, "budget": 32768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "weights", "select", "compact"])
    kv = rng.choice(["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        H = rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, 8192)
        rot = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
        return {"op": op, "kv": kv, "T": T, "Hq": H * rng.randint(1, 8), "H": H, "D": D, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                "far": _log(rng, 4096, 1 << 20), "fused": rng.random() < 0.5, "chunk": rng.randint(1, max(1, T))}
    H = rng.choice([1, 2, 4, 8])
    longest = _log(rng, 1, 131072)
    S = _log(rng, 1, max(1, min(256, (4 * 131072) // longest)))
    case = {"op": op, "S": S, "H": H, "shortest": rng.randint(0, longest), "longest": longest}
    if op == "weights":
        return {**case, "kv": kv, "Hq": H * rng.randint(1, 8), "D": D}
    budget = max(1, int(longest * rng.uniform(0.05, 0.9)))
    if op == "compact":
        return {**case, "kv": kv, "D": D, "budget": min(budget, 32768)}
    sinks = min(rng.randint(0, 8), budget)
    return {**case, "budget": budget, "sinks": sinks, "recent": int((budget - sinks) * rng.random())}


def _scaling(case):
    """The rotary parameters of a case; scaled ones stretch an 8192-token model 16 times."""
    p = {"theta": 500000.0 if case["D"] == 128 else 10000.0, "scaling": case["scaling"], "factor": 1.0, "original": 8192,
         "low": 1.0, "high": 4.0, "gain": 1.0}
    if case["scaling"] != "none":
        p["factor"] = 16.0
    if case["scaling"] == "yarn":
        p["high"] = 32.0
        p["gain"] = 0.1 * math.log(p["factor"]) + 1.0
    if case["scaling"] == "ntk" and case["rot"] == 2:
        p["scaling"], p["factor"] = "none", 1.0  # the raised base is not defined for a single pair
    return p


# ------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Context lengths, uniform over the case's range, the longest one among them."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    n = torch.randint(case["shortest"], case["longest"] + 1, (case["S"],), generator=g)
    n[int(torch.randint(0, case["S"], (1,), generator=g))] = case["longest"]
    return [int(x) for x in n]


def _dtype(kv):
    return torch.float16 if kv == "fp16" else torch.bfloat16


def _elem(kv):
    return 1 if kv.startswith("fp8") else 2


def _region(kv, blocks, H, D, gen, scale, spread=1.0):
    """One layer's K or V region as bytes: N(0, spread) values in every slot."""
    n = blocks * H * BLOCK * D
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    x.normal_(0.0, spread, generator=gen)
    if kv == "fp16":
        return x.to(torch.float16).view(torch.uint8)
    if kv == "bf16":
        return x.view(torch.uint8)
    out = torch.empty(n + (-(-blocks * H * 4 // 16) * 16 if kv == "fp8_e4m3_block" else 0), dtype=torch.uint8, device="cuda")
    if kv == "fp8_e4m3":
        s = torch.full((1, 1), scale, device="cuda")
    else:
        s = (x.view(-1, BLOCK * D).abs().amax(1, keepdim=True).float() / FP8_MAX).contiguous()
        out[n:].zero_()
        out[n:n + blocks * H * 4] = s.view(-1).view(torch.uint8)
    rows = x.view(s.shape[0], -1)
    step = max(1, (1 << 28) // rows.shape[1]) if rows.shape[0] > 1 else 1
    done = out[:n].view(s.shape[0], -1)
    for lo in range(0, rows.shape[0], step):  # in parts: the fp32 copy would not fit thrice
        q = (rows[lo:lo + step].float() / s[lo:lo + step]).clamp(-FP8_MAX, FP8_MAX)
        done[lo:lo + step] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _tables(lengths, first, ids, width):
    """Block table [S, width]: sequence s gets the next ids; entries behind its pages are -1."""
    t = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = first
    for s, n in enumerate(lengths):
        k = -(-n // BLOCK)
        t[s, :k] = ids[at:at + k]
        at += k
    return t.cuda(), at


def _inputs(case, seed):
    """Everything a user's program holds before the call, but for the pool's handle."""
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed * 7 + 2)
    st = {"case": dict(case)}
    if op == "rope":
        T, Hq, H, D, kv = (case[k] for k in ("T", "Hq", "H", "D", "kv"))
        dt = _dtype(kv)
        chunks = [case["chunk"]] * (T // case["chunk"]) + ([T % case["chunk"]] if T % case["chunk"] else [])
        need = [-(-c // BLOCK) for c in chunks]
        st["blocks"] = sum(need) + sum(need) // 8 + 1
        ids = torch.randperm(st["blocks"], generator=cpu)
        starts = torch.randint(0, case["far"], (len(chunks),), generator=cpu)
        slot, pos, at = [], [], 0
        for c, k, p in zip(chunks, need, starts):
            i = torch.arange(c)
            slot.append(ids[at + i // BLOCK] * BLOCK + i % BLOCK)
            pos.append(p + i)
            at += k
        slot, pos = torch.cat(slot), torch.cat(pos)
        if kv != "fp8_e4m3_block" and T > 8:
            slot[T // 2] = -1  # a token that is only padding
        st["slots"], st["positions"] = slot.cuda(), pos.to(torch.int32).cuda()
        if case["fused"]:  # one product gave q, k and v side by side
            x = torch.empty(T, Hq + 2 * H, D, dtype=dt, device="cuda").normal_(generator=gen)
            st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        else:
            st["q"], st["k"], st["v"] = (torch.empty(T, h, D, dtype=dt, device="cuda").normal_(generator=gen) for h in (Hq, H, H))
        st["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
        st["k_cache"], st["v_cache"] = (_region(kv, st["blocks"], H, D, gen, s) for s in (K_SCALE, V_SCALE))
        st["rope"] = _scaling(case)
        st["freq"] = _frequencies(case["rot"], st["rope"])
        return st
    S, H = case["S"], case["H"]
    lengths = _lengths(case, seed)
    st["lengths"] = lengths
    pages = -(-case["longest"] // BLOCK)
    width = pages * BLOCK
    st["ctx"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    # running totals: few tokens hold most of the weight, many hold none at all
    w = torch.empty(S, H, width, device="cuda").normal_(0.0, 2.5, generator=gen).exp_()
    w *= torch.empty(S, H, width, device="cuda").uniform_(generator=gen) > 0.2
    w.masked_fill_(torch.arange(width, device="cuda") >= st["ctx"].view(S, 1, 1), 0.0)
    st["weights"] = w
    if op == "select":
        return st
    kv, D = case["kv"], case["D"]
    kept = [min(n, case["budget"]) for n in lengths] if op == "compact" else []
    st["blocks"] = S * pages + (S * -(-min(case["budget"], case["longest"]) // BLOCK) if kept else 0) + S + 1
    ids = torch.randperm(st["blocks"], generator=cpu).to(torch.int32)
    st["tables"], at = _tables(lengths, 0, ids, pages)
    st["k_cache"], st["v_cache"] = (_region(kv, st["blocks"], H, D, gen, s) for s in (K_SCALE, V_SCALE))
    if op == "weights":
        st["q"] = torch.empty(S, case["Hq"], D, dtype=_dtype(kv), device="cuda").normal_(0.0, 1.5, generator=gen)
        st["scale"] = 1.0 / math.sqrt(D)
        st["decay"] = 0.95
        st["weights_out"] = torch.zeros_like(w)
        return st
    B = case["budget"]
    st["dst_tables"], _ = _tables(kept, at, ids, -(-min(B, case["longest"]) // BLOCK))
    st["kept"] = torch.tensor(kept, dtype=torch.int32, device="cuda")
    # a sorted random choice of `kept` tokens of each sequence, another one for each head
    order = torch.empty(S, H, width, device="cuda").uniform_(generator=gen)
    order.masked_fill_(torch.arange(width, device="cuda") >= st["ctx"].view(S, 1, 1), 2.0)
    order = order.argsort(-1)[..., :B]
    order.masked_fill_(torch.arange(order.shape[-1], device="cuda") >= st["kept"].view(S, 1, 1), width)
    order = order.sort(-1).values.to(torch.int32)
    order.masked_fill_(order == width, -1)
    keep = torch.full((S, H, B), -1, dtype=torch.int32, device="cuda")
    keep[..., :order.shape[-1]] = order
    st["keep"] = keep
    st["weights_out"] = torch.ones_like(w)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] == "select":
        from paged_kv_cache_270_gb300.pool import KVPool

        st["pool"] = KVPool(1, 1, case["H"], 128, "bf16")
    elif own:
        from paged_kv_cache_270_gb300.pool import KVPool, make_rope

        pool = KVPool(1, st["blocks"], case["H"], case["D"], case["kv"], K_SCALE, V_SCALE)
        pool.k_cache.copy_(st["k_cache"])
        pool.v_cache.copy_(st["v_cache"])
        st["pool"], st["k_cache"], st["v_cache"] = pool, pool.k_cache, pool.v_cache
        if case["op"] == "rope":
            p = st["rope"]
            st["rope"] = make_rope(case["rot"], layout=case["layout"], theta=p["theta"], scaling=p["scaling"], factor=p["factor"],
                                   original_len=p["original"], low=p["low"], high=p["high"], gain=p["gain"])
        if case["op"] == "weights":
            n = pool.weights_workspace_bytes(case["S"], case["Hq"], st["tables"].shape[1])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            st["out"] = torch.empty_like(st["q"])
    return st


# --------------------------------------------------------------- the plain forms
def _values(case, st, which):
    """The region as the elements it stands for, [blocks, H, 16, D], without their scales."""
    n = st["blocks"] * case["H"] * BLOCK * case["D"] * _elem(case["kv"])
    t = st[which][:n].view(torch.float8_e4m3fn if case["kv"].startswith("fp8") else _dtype(case["kv"]))
    return t.view(st["blocks"], case["H"], BLOCK, case["D"])


def _tile_scales(case, st, which):
    n = st["blocks"] * case["H"] * BLOCK * case["D"]
    return st[which][n:n + st["blocks"] * case["H"] * 4].view(torch.float32).view(st["blocks"], case["H"])


def _caches(case, st):
    """The written regions, and a block-scaled pool's scales."""
    out = [_values(case, st, "k_cache"), _values(case, st, "v_cache")]
    if case["kv"] == "fp8_e4m3_block":
        out += [_tile_scales(case, st, "k_cache"), _tile_scales(case, st, "v_cache")]
    return out


def _frequencies(rot, p):
    """Angle per position of each pair, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta, s, L = p["theta"], p["factor"], p["original"]
    if p["scaling"] == "ntk":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if p["scaling"] == "linear":
        f = f / s
    if p["scaling"] == "bands":
        g = ((L * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * g + f / s * (1 - g)
    if p["scaling"] == "yarn":
        dim = lambda turns: rot * math.log(L / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(dim(p["high"])), 0), min(math.ceil(dim(p["low"])), rot - 1)
        g = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * g + f / s * (1 - g)
    return f


def _rotate(x, cos, sin, rot, layout):
    """x [T, H, D] in 32 bits, its first `rot` dims turned."""
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _put(case, st, which, x, scale):
    """x [T, H, D] in 32 bits into the slots of a region."""
    region, slots, kv = _values(case, st, which), st["slots"], case["kv"]
    blk, off = slots // BLOCK, slots % BLOCK
    if kv == "fp8_e4m3_block":
        # every run starts its tile afresh; the tile's scale is that of its written rows
        tile = torch.zeros(st["blocks"], BLOCK, case["H"], case["D"], device="cuda")
        tile[blk, off] = x
        m = tile.abs().amax((1, 3))
        s = m / FP8_MAX
        scales = _tile_scales(case, st, which)
        scales[blk] = s[blk]
        sx = s[blk].unsqueeze(-1)
        q = torch.where(sx > 0, x / sx, torch.zeros_like(x)).clamp(-FP8_MAX, FP8_MAX)
        region.view(torch.uint8)[blk, :, off] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        return
    keep = (slots >= 0).nonzero().squeeze(1)
    x = x[keep]
    if kv == "fp8_e4m3":
        q = (x / torch.tensor(scale, dtype=torch.float32, device="cuda")).clamp(-FP8_MAX, FP8_MAX)
        region.view(torch.uint8)[blk[keep], :, off[keep]] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        region[blk[keep], :, off[keep]] = x.to(region.dtype)


def _plain_rope(case, st):
    angle = st["positions"].double().unsqueeze(1) * st["freq"]
    gain = st["rope"]["gain"]
    cos, sin = (gain * angle.cos()).float().unsqueeze(1), (gain * angle.sin()).float().unsqueeze(1)
    q = _rotate(st["q"].float(), cos, sin, case["rot"], case["layout"])
    k = _rotate(st["k"].float(), cos, sin, case["rot"], case["layout"])
    _put(case, st, "k_cache", k, K_SCALE)
    _put(case, st, "v_cache", st["v"].float(), V_SCALE)
    return [q.to(st["q"].dtype)] + _caches(case, st)


def _gather(case, st, which, scale):
    """Every sequence's keys or values in 32 bits, [S, H, tokens, D]."""
    t = st["tables"].long().clamp_min(0)
    S, P = t.shape
    x = _values(case, st, which)
    x = (x.view(torch.uint8)[t].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[t]).float()  # [S, P, H, 16, D]
    if case["kv"] == "fp8_e4m3_block":
        x *= _tile_scales(case, st, which)[t].view(S, P, case["H"], 1, 1)
    elif case["kv"] == "fp8_e4m3":
        x *= torch.tensor(scale, dtype=torch.float32, device="cuda")
    return x.permute(0, 2, 1, 3, 4).reshape(S, case["H"], P * BLOCK, case["D"])


def _plain_weights(case, st):
    S, H, D = case["S"], case["H"], case["D"]
    there = torch.arange(st["weights"].shape[-1], device="cuda") < st["ctx"].view(S, 1, 1)
    q = st["q"].float().view(S, H, -1, D) * st["scale"]
    x = q @ _gather(case, st, "k_cache", K_SCALE).transpose(2, 3)
    x = x.masked_fill(~there.unsqueeze(2), -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = (x - m).exp()
    l = e.sum(-1, keepdim=True)
    p = torch.where(l > 0, e / l, torch.zeros_like(e))
    v = _gather(case, st, "v_cache", V_SCALE).masked_fill(~there.unsqueeze(3), 0.0)
    out = (p @ v).view(S, -1, D).to(st["q"].dtype)
    w = torch.where(there, st["decay"] * st["weights"] + p.sum(2), st["weights_out"])
    return [out, w]


def _plain_select(case, st):
    S, H, B = case["S"], case["H"], case["budget"]
    w, n = st["weights"], st["ctx"].view(S, 1, 1)
    W = w.shape[-1]
    at = torch.arange(W, device="cuda").expand(S, H, W)
    must = (at < case["sinks"]) | (at >= n - case["recent"])
    key = torch.where(must, torch.full_like(w, math.inf), w).masked_fill(at >= n, -math.inf)
    first = key.sort(dim=-1, descending=True, stable=True).indices[..., :B]
    chosen = torch.zeros(S, H, W, dtype=torch.bool, device="cuda").scatter_(-1, first, True) & (at < n)
    place = torch.where(chosen, at, torch.full_like(at, W)).sort(-1).values[..., :B]
    keep = torch.full((S, H, B), -1, dtype=torch.int32, device="cuda")
    keep[..., :place.shape[-1]] = torch.where(place < W, place, torch.full_like(place, -1)).to(torch.int32)
    return [keep, st["ctx"].clamp_max(B)]


def _plain_compact(case, st):
    S, H, D, kv = case["S"], case["H"], case["D"], case["kv"]
    P = st["dst_tables"].shape[1]
    n = P * BLOCK
    keep = st["keep"][..., :n].long()
    if keep.shape[-1] < n:
        keep = torch.cat([keep, keep.new_full((S, H, n - keep.shape[-1]), -1)], -1)
    live = torch.arange(n, device="cuda") < st["kept"].view(S, 1, 1)
    live = live.expand(S, H, n)
    src = keep.clamp_min(0)
    sblk = st["tables"].long().view(S, 1, -1).expand(S, H, -1).gather(2, src // BLOCK).clamp_min(0)
    head = torch.arange(H, device="cuda").view(1, H, 1).expand(S, H, n)
    dblk = st["dst_tables"].long().repeat_interleave(BLOCK, 1).view(S, 1, n).expand(S, H, n)
    doff = torch.arange(n, device="cuda").remainder(BLOCK).expand(S, H, n)
    for which in ("k_cache", "v_cache"):
        region = _values(case, st, which)
        raw = region.view(torch.uint8) if region.dtype == torch.float8_e4m3fn else region
        rows = raw[sblk, head, src % BLOCK]  # [S, H, n, D]
        if kv == "fp8_e4m3_block":
            scales = _tile_scales(case, st, which)
            x = rows.view(torch.float8_e4m3fn).float() * scales[sblk, head].unsqueeze(-1)
            x = x.masked_fill(~live.unsqueeze(-1), 0.0).view(S, H, P, BLOCK, D)
            s = x.abs().amax((3, 4), keepdim=True) / FP8_MAX
            q = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-FP8_MAX, FP8_MAX)
            rows = q.to(torch.float8_e4m3fn).view(torch.uint8).view(S, H, n, D)
            full = live[:, :, ::BLOCK]
            scales[dblk[:, :, ::BLOCK][full], head[:, :, ::BLOCK][full]] = s.view(S, H, P)[full]
        raw[dblk[live], head[live], doff[live]] = rows[live]
    w = torch.zeros_like(st["weights_out"])
    w[..., :n] = torch.where(live, st["weights"].gather(2, src), torch.zeros_like(w[..., :n]))
    return _caches(case, st) + [w]


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        plain = {"rope": _plain_rope, "weights": _plain_weights, "select": _plain_select, "compact": _plain_compact}
        return plain[op](case, st)
    pool = st["pool"]
    if op == "rope":
        q = pool.rope_and_cache(st["rope"], st["q"], st["k"], st["v"], st["positions"], st["slots"], q_out=st["q_out"])
        return [q] + _caches(case, st)
    if op == "weights":
        return list(pool.decode_weights(st["q"], st["tables"], st["ctx"], st["weights"], weights_out=st["weights_out"], decay=st["decay"],
                                        softmax_scale=st["scale"], out=st["out"], workspace=st["workspace"]))
    if op == "select":
        return list(pool.evict_select(st["weights"], st["ctx"], case["budget"], sinks=case["sinks"], recent=case["recent"]))
    pool.evict_compact(st["keep"], st["kept"], st["tables"], st["dst_tables"], weights=st["weights"], weights_out=st["weights_out"])
    return _caches(case, st) + [st["weights_out"]]


def work(case):
    op, H = case["op"], case["H"]
    if op == "rope":
        T, Hq, D = case["T"], case["Hq"], case["D"]
        return {"bytes": T * (4 * Hq * D + 4 * H * D + 2 * H * D * _elem(case["kv"]) + 12), "flops": 3 * T * (Hq + H) * case["rot"]}
    # the mean length of the sequences that a seed draws
    S = case["S"]
    tokens = (S - 1) * (case["shortest"] + case["longest"]) / 2 + case["longest"]
    kept = min(case.get("budget", 0), tokens / S) * S
    if op == "weights":
        D, Hq = case["D"], case["Hq"]
        return {"bytes": tokens * H * (2 * D * _elem(case["kv"]) + 8) + 4 * S * Hq * D + tokens / 4, "flops": 4 * tokens * Hq * D}
    if op == "select":
        return {"bytes": 4 * H * tokens + 4 * H * S * case["budget"], "flops": H * tokens}
    width = -(-case["longest"] // BLOCK) * BLOCK
    return {"bytes": kept * H * (4 * case["D"] * _elem(case["kv"]) + 8) + 4 * S * H * width, "flops": 0}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """What `run` returns, from the definitions, in 64 bits; None where codes or whole numbers are held."""
    op = case["op"]
    if op == "select":
        return None
    st = _inputs(case, seed)
    coded = case["kv"].startswith("fp8")
    if op == "rope":
        return _exact_rope(case, st, coded)
    if op == "compact":
        return _exact_compact(case, st, coded)
    S, H, D, kv = case["S"], case["H"], case["D"], case["kv"]
    G = case["Hq"] // H
    out = torch.zeros(S, case["Hq"], D, dtype=torch.float64, device="cuda")
    w = st["weights_out"].double()
    size = BLOCK * D * _elem(kv)
    for s, n in enumerate(st["lengths"]):
        if n == 0:
            continue
        rows = {}
        for which, scale in (("k_cache", K_SCALE), ("v_cache", V_SCALE)):
            ids = st["tables"][s, :-(-n // BLOCK)].long()
            raw = st[which][:st["blocks"] * H * size].view(st["blocks"], H * size)[ids]
            x = raw.view(torch.float8_e4m3fn if coded else _dtype(kv)).double().view(-1, H, BLOCK, D)
            if kv == "fp8_e4m3":
                x = x * float(torch.tensor(scale, dtype=torch.float32))
            if kv == "fp8_e4m3_block":
                at = st["blocks"] * H * size
                sc = st[which][at:at + st["blocks"] * H * 4].view(torch.float32).view(-1, H)[ids]
                x = x * sc.double()[:, :, None, None]
            rows[which] = x.transpose(0, 1).reshape(H, -1, D)[:, :n]
        for h in range(H):
            z = st["q"][s, h * G:(h + 1) * G].double() @ rows["k_cache"][h].T * st["scale"]
            p = torch.softmax(z, -1)
            out[s, h * G:(h + 1) * G] = p @ rows["v_cache"][h]
            w[s, h, :n] = st["decay"] * st["weights"][s, h, :n].double() + p.sum(0)
    return [out, w]


def _exact_compact(case, st, coded):
    H, D = case["H"], case["D"]
    w = torch.zeros(st["weights_out"].shape, dtype=torch.float64, device="cuda")
    flat = [] if coded else [st[c].view(_dtype(case["kv"])).double().view(-1, H, BLOCK, D) for c in ("k_cache", "v_cache")]
    for s, n in enumerate(min(n, case["budget"]) for n in st["lengths"]):
        i = torch.arange(n, device="cuda")
        for h in range(H):
            src = st["keep"][s, h, :n].long()
            w[s, h, :n] = st["weights"][s, h, src].double()
            for pages in flat:
                rows = pages[st["tables"][s, src // BLOCK].long(), h, src % BLOCK]
                pages[st["dst_tables"][s, i // BLOCK].long(), h, i % BLOCK] = rows
    return (flat or [None, None]) + ([None, None] if case["kv"] == "fp8_e4m3_block" else []) + [w]


def _exact_rope(case, st, coded):
    T, H, D, R = case["T"], case["H"], case["D"], case["rot"]
    p = st["rope"]
    speed = []
    for i in range(R // 2):
        base = p["theta"] * (p["factor"] ** (R / (R - 2)) if p["scaling"] == "ntk" else 1.0)
        f = base ** (-2.0 * i / R)
        share = 1.0  # of the unscaled speed
        if p["scaling"] == "linear":
            share = 0.0
        elif p["scaling"] == "bands":
            share = min(1.0, max(0.0, (p["original"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])))
        elif p["scaling"] == "yarn":
            index = [R * math.log(p["original"] / (2 * math.pi * t)) / (2 * math.log(base)) for t in (p["high"], p["low"])]
            lo, hi = max(math.floor(index[0]), 0), min(math.ceil(index[1]), R - 1)
            share = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        speed.append(share * f + (1.0 - share) * f / p["factor"])
    turn = torch.outer(st["positions"].double(), torch.tensor(speed, dtype=torch.float64, device="cuda"))
    spin = torch.polar(torch.full_like(turn, p["gain"]), turn).unsqueeze(1)

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) if case["layout"] == "half" else torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], R // 2, 2).contiguous())
        z = z * spin
        y = torch.cat([z.real, z.imag], -1) if case["layout"] == "half" else torch.view_as_real(z).reshape(*x.shape[:2], R)
        return torch.cat([y, x[..., R:]], -1)

    q = turned(st["q"])
    if coded:
        return [q, None, None] + ([None, None] if case["kv"] == "fp8_e4m3_block" else [])
    got = [q]
    use = st["slots"] >= 0
    flat = st["slots"][use]
    for which, x in (("k_cache", turned(st["k"])), ("v_cache", st["v"].double())):
        pages = st[which].view(_dtype(case["kv"])).double().view(st["blocks"], H, BLOCK, D).transpose(1, 2).reshape(-1, H, D)
        pages[flat] = x[use]
        got.append(pages.view(st["blocks"], BLOCK, H, D).transpose(1, 2).contiguous())
    return got
