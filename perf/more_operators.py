"""The cases that speculative decoding over the paged cache, and its head norms, are measured on.

A case is a dict of plain values: `op` names the operator, the rest its sizes.

  norm     every head's queries and keys normalised by their root mean square,
           rotated at positions of one or three axes, and keys and values
           written into their slots of the paged cache
  tree     attention of the drafted tokens of each sequence, a tree, over the
           sequence's pages and over their own ancestors in the tree
  accept   the accepted path of each tree moved together behind the sequence's
           history, in every layer of the pool

With `own` false `run` computes an operator in plain tensor operations; with
`own` true it makes the calls that a user of the package makes.
"""
import math

import torch

own = False

BLOCK = 16
FP8_MAX = 448.0
K_SCALE, V_SCALE = 0.0125, 0.015  # per-tensor scales of the FP8 pools (amax of N(0, 1) over 448)
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: one new token each, 32 / 8 heads
        {"name": "norm_step_bf16", "op": "norm", "kv": "bf16", "T": 64, "Hq": 32, "H": 8, "D": 128, "rot": 128,
         "layout": "half", "axes": "one", "far": 4096, "fused": True, "chunk": 1, "per_head": False, "offset": 0.0},
        # an 8192-token prefill packet of text and images, 64 / 8 heads, FP8 pages
        {"name": "norm_packet_fp8", "op": "norm", "kv": "fp8_e4m3", "T": 8192, "Hq": 64, "H": 8, "D": 128, "rot": 128,
         "layout": "half", "axes": "sections", "far": 131072, "fused": True, "chunk": 2048, "per_head": False, "offset": 0.0},
        # prompts of ragged length written with a scale per tile, axes in turn
        {"name": "norm_prompts_block", "op": "norm", "kv": "fp8_e4m3_block", "T": 2037, "Hq": 32, "H": 8, "D": 128,
         "rot": 128, "layout": "half", "axes": "turns", "far": 131072, "fused": False, "chunk": 509, "per_head": False, "offset": 0.0},
        # an odd number of tokens, small heads of which half is rotated, a weight of its own for each head
        {"name": "norm_part_fp16", "op": "norm", "kv": "fp16", "T": 1021, "Hq": 4, "H": 2, "D": 64, "rot": 32,
         "layout": "interleaved", "axes": "one", "far": 30000, "fused": False, "chunk": 100, "per_head": True, "offset": 1.0},
        # four short sequences with a few drafted tokens: latency of the call
        {"name": "tree_tiny_fp16", "op": "tree", "kv": "fp16", "S": 4, "Hq": 4, "H": 2, "D": 64, "shortest": 17, "longest": 100,
         "few": 3, "nodes": 7},
        # an ordinary ragged batch, 16 drafted tokens each
        {"name": "tree_step_bf16", "op": "tree", "kv": "bf16", "S": 64, "Hq": 32, "H": 8, "D": 128, "shortest": 512,
         "longest": 4096, "few": 16, "nodes": 16},
        # a large batch of FP8 pages, eight queries per key head, trees of different sizes
        {"name": "tree_many_fp8", "op": "tree", "kv": "fp8_e4m3", "S": 128, "Hq": 64, "H": 8, "D": 128, "shortest": 4096,
         "longest": 4096, "few": 8, "nodes": 16},
        # few sequences of the longest context, wider trees
        {"name": "tree_long_fp8", "op": "tree", "kv": "fp8_e4m3", "S": 4, "Hq": 64, "H": 8, "D": 128, "shortest": 131072,
         "longest": 131072, "few": 32, "nodes": 32},
        # an odd number of queries per key head, large trees of odd size, a scale per tile
        {"name": "tree_wide_block", "op": "tree", "kv": "fp8_e4m3_block", "S": 24, "Hq": 40, "H": 8, "D": 128, "shortest": 1000,
         "longest": 9001, "few": 25, "nodes": 61},
        # one layer after an ordinary step: latency of the call
        {"name": "accept_step_bf16", "op": "accept", "kv": "bf16", "layers": 1, "S": 64, "H": 8, "D": 128, "shortest": 16,
         "longest": 120, "few": 16, "nodes": 16, "path": 5},
        # all layers of a model at once, FP8 pages
        {"name": "accept_layers_fp8", "op": "accept", "kv": "fp8_e4m3", "layers": 32, "S": 64, "H": 8, "D": 128, "shortest": 20,
         "longest": 100, "few": 8, "nodes": 16, "path": 6},
        # all layers, odd sizes, large trees, a scale per tile
        {"name": "accept_layers_block", "op": "accept", "kv": "fp8_e4m3_block", "layers": 32, "S": 33, "H": 8, "D": 128,
         "shortest": 61, "longest": 150, "few": 25, "nodes": 61, "path": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "tree", "accept"])
    kv = rng.choice(["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"])
    D = rng.choice([64, 128, 128])
    H = rng.choice([1, 2, 4, 8])
    if op == "norm":
        T = _log(rng, 1, 8192)
        rot = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
        axes = rng.choice(["one", "sections", "turns"]) if rot >= 6 else "one"
        return {"op": op, "kv": kv, "T": T, "Hq": H * rng.randint(1, 8), "H": H, "D": D, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "axes": axes, "far": _log(rng, 4096, 1 << 20),
                "fused": rng.random() < 0.5, "chunk": rng.randint(1, max(1, T)), "per_head": rng.random() < 0.3,
                "offset": rng.choice([0.0, 0.0, 1.0])}
    nodes = _log(rng, 1, 256)
    few = rng.randint(1, nodes)
    if op == "accept":
        layers = rng.choice([1, 2, 5, 16, 32])
        return {"op": op, "kv": kv, "layers": layers, "S": _log(rng, 1, 64), "H": H, "D": D, "shortest": rng.randint(0, 100),
                "longest": 100 + nodes, "few": few, "nodes": nodes, "path": rng.randint(1, nodes)}
    G = rng.randint(1, 8)
    longest = _log(rng, nodes, 131072)
    # no more products than four sequences of the longest context, 64 heads and 32 tokens have
    most = (4 * 131072 * 64 * 32) // (longest * H * G * nodes)
    S = _log(rng, 1, max(1, min(128, most, (4 * 131072) // longest)))
    return {"op": op, "kv": kv, "S": S, "Hq": H * G, "H": H, "D": D, "shortest": rng.randint(0, longest), "longest": longest,
            "few": few, "nodes": nodes}


def _sections(case):
    """How many pairs turn with each of the three axes (time, height, width)."""
    pairs = case["rot"] // 2
    side = 3 * pairs // 8 if case["axes"] == "sections" else pairs * 5 // 16
    return [pairs - 2 * side, side, side]


def _axis_of(case):
    """The axis that each pair turns with."""
    pairs = case["rot"] // 2
    if case["axes"] == "one":
        return [0] * pairs
    n = _sections(case)
    if case["axes"] == "sections":
        return [0] * n[0] + [1] * n[1] + [2] * n[2]
    return [i % 3 if i < 3 * n[i % 3] else 0 for i in range(pairs)]


# ------------------------------------------------------------------ inputs
def _dtype(kv):
    return torch.float16 if kv == "fp16" else torch.bfloat16


def _elem(kv):
    return 1 if kv.startswith("fp8") else 2


def _region(kv, layers, blocks, H, D, gen, scale):
    """A K or V region of all layers as bytes: N(0, 1) values in every slot."""
    n = layers * blocks * H * BLOCK * D
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    x.normal_(0.0, 1.0, generator=gen)
    if kv == "fp16":
        return x.to(torch.float16).view(torch.uint8)
    if kv == "bf16":
        return x.view(torch.uint8)
    tiles = layers * blocks * H
    out = torch.empty(n + (-(-tiles * 4 // 16) * 16 if kv == "fp8_e4m3_block" else 0), dtype=torch.uint8, device="cuda")
    if kv == "fp8_e4m3":
        s = torch.full((1, 1), scale, device="cuda")
    else:
        # tiles of different magnitude, as tokens have
        rows = x.view(tiles, BLOCK * D)
        rows *= torch.empty(tiles, 1, device="cuda").uniform_(0.5, 2.0, generator=gen).to(torch.bfloat16)
        s = (rows.abs().amax(1, keepdim=True).float() / FP8_MAX).contiguous()
        out[n:].zero_()
        out[n:n + tiles * 4] = s.view(-1).view(torch.uint8)
    rows = x.view(s.shape[0], -1)
    step = max(1, (1 << 28) // rows.shape[1]) if rows.shape[0] > 1 else 1
    done = out[:n].view(s.shape[0], -1)
    for lo in range(0, rows.shape[0], step):  # in parts: the fp32 copy would not fit thrice
        q = (rows[lo:lo + step].float() / s[lo:lo + step]).clamp(-FP8_MAX, FP8_MAX)
        done[lo:lo + step] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _tables(lengths, ids, width):
    """Block table [S, width]: sequence s gets the next ids; entries behind its pages are -1."""
    t = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lengths):
        k = -(-n // BLOCK)
        t[s, :k] = ids[at:at + k]
        at += k
    return t.cuda()


def _norm_inputs(case, st, gen, cpu):
    T, Hq, H, D, kv = (case[k] for k in ("T", "Hq", "H", "D", "kv"))
    dt = _dtype(kv)
    chunks = [case["chunk"]] * (T // case["chunk"]) + ([T % case["chunk"]] if T % case["chunk"] else [])
    need = [-(-c // BLOCK) for c in chunks]
    st["blocks"] = sum(need) + sum(need) // 8 + 1
    ids = torch.randperm(st["blocks"], generator=cpu)
    starts = torch.randint(0, case["far"], (len(chunks),), generator=cpu)
    slot, pos, at = [], [], 0
    for j, (c, k, p) in enumerate(zip(chunks, need, starts)):
        i = torch.arange(c)
        slot.append(ids[at + i // BLOCK] * BLOCK + i % BLOCK)
        if case["axes"] == "one":
            pos.append((p + i).unsqueeze(0))
        elif j % 2 == 0 and len(chunks) > 1:  # text: all axes go on together
            pos.append((p + i).expand(3, c))
        else:  # frames of 24 x 32 patches
            pos.append(torch.stack([p + i // 768, p + i // 32 % 24, p + i % 32]))
        at += k
    slot, pos = torch.cat(slot), torch.cat(pos, 1)
    if kv != "fp8_e4m3_block" and T > 8:
        slot[T // 2] = -1  # a token that is only padding
    st["slots"], st["positions"] = slot.cuda(), pos.to(torch.int32).contiguous().cuda()
    if case["fused"]:  # one product gave q, k and v side by side
        x = torch.empty(T, Hq + 2 * H, D, dtype=dt, device="cuda").normal_(0.0, 1.5, generator=gen)
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        st["q"], st["k"], st["v"] = (torch.empty(T, h, D, dtype=dt, device="cuda").normal_(0.0, 1.5, generator=gen) for h in (Hq, H, H))
    for name, h in (("q_weight", Hq), ("k_weight", H)):
        shape = (h, D) if case["per_head"] else (D,)
        st[name] = torch.empty(shape, dtype=dt, device="cuda").normal_(1.0 - case["offset"], 0.2, generator=gen)
    st["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    st["k_cache"], st["v_cache"] = (_region(kv, 1, st["blocks"], H, D, gen, s) for s in (K_SCALE, V_SCALE))
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    st["speed"] = _theta(case) ** (-2.0 * i / case["rot"])
    st["axis"] = torch.tensor(_axis_of(case), device="cuda")
    return st


def _theta(case):
    return 1000000.0 if case["D"] == 128 else 10000.0


def _trees(case, st, cpu):
    """Sizes of the trees, lengths of the histories in front of them, and who sees whom."""
    S, N = case["S"], case["nodes"]
    sizes = torch.randint(case["few"], N + 1, (S,), generator=cpu)
    sizes[int(torch.randint(0, S, (1,), generator=cpu))] = N
    total = torch.randint(case["shortest"], case["longest"] + 1, (S,), generator=cpu)
    total[int(torch.randint(0, S, (1,), generator=cpu))] = case["longest"]
    ctx = torch.maximum(total, sizes)  # a sequence holds its tree at least
    st["sizes"], st["lengths"] = sizes.tolist(), ctx.tolist()
    q_start = torch.zeros(S + 1, dtype=torch.int32)
    q_start[1:] = sizes.cumsum(0)
    st["q_start"], st["ctx"] = q_start.cuda(), ctx.to(torch.int32).cuda()
    # a node's parent is one of the eight nodes before it, or the history
    sees = torch.zeros(S, N, N, dtype=torch.bool)
    back = torch.randint(1, 9, (S, N), generator=cpu)
    every = torch.arange(S)
    for i in range(N):
        parent = i - back[:, i]
        sees[:, i] = sees[every, parent.clamp_min(0)] & (parent >= 0).unsqueeze(1)
        sees[:, i, i] = True
    hole = torch.randint(0, 32, (S, N), generator=cpu) == 0  # places of a tree that hold no token
    sees[hole] = False
    st["sees"] = sees
    here = torch.arange(N) < sizes.unsqueeze(1)
    words = -(-N // 64)
    bits = torch.zeros(S, N, words * 64, dtype=torch.int64)
    bits[..., :N] = sees
    packed = (bits.view(S, N, words, 64) << torch.arange(64)).sum(-1)  # (bit 63 is the sign)
    # rows as many as the batch may need: those behind the last tree are padding
    st["mask"] = torch.zeros(S * N, words, dtype=torch.int64)
    st["mask"][:sum(st["sizes"])] = packed[here]
    st["mask"] = st["mask"].cuda()
    return ctx.tolist()


def _tree_inputs(case, st, gen, cpu):
    S, H, D, kv = case["S"], case["H"], case["D"], case["kv"]
    lengths = _trees(case, st, cpu)
    pages = -(-max(case["longest"], case["nodes"]) // BLOCK)
    st["blocks"] = S * pages + 1
    st["tables"] = _tables(lengths, torch.randperm(st["blocks"], generator=cpu).to(torch.int32), pages)
    st["k_cache"], st["v_cache"] = (_region(kv, 1, st["blocks"], H, D, gen, s) for s in (K_SCALE, V_SCALE))
    st["q"] = torch.empty(S * case["nodes"], case["Hq"], D, dtype=_dtype(kv), device="cuda").normal_(0.0, 1.5, generator=gen)
    st["scale"] = 1.0 / math.sqrt(D)
    st["out"] = torch.zeros_like(st["q"])
    return st


def _accept_inputs(case, st, gen, cpu):
    S, H, D, kv = case["S"], case["H"], case["D"], case["kv"]
    lengths = _trees(case, st, cpu)
    pages = -(-max(case["longest"], case["nodes"]) // BLOCK)
    st["blocks"] = S * pages + 1
    st["tables"] = _tables(lengths, torch.randperm(st["blocks"], generator=cpu).to(torch.int32), pages)
    st["k_cache"], st["v_cache"] = (_region(kv, case["layers"], st["blocks"], H, D, gen, s) for s in (K_SCALE, V_SCALE))
    # An accepted path starts along the first nodes and goes on in nodes behind its own places (with
    # a scale per tile: in pages behind them), so that a pass leaves what the next one reads as it is.
    paths = torch.full((S, case["path"]), -1, dtype=torch.int32)
    lens = []
    for s, n in enumerate(st["sizes"]):
        k = int(torch.randint(0, min(n, case["path"]) + 1, (1,), generator=cpu))
        base = lengths[s] - n
        first = k if kv != "fp8_e4m3_block" else -(-(base + k) // BLOCK) * BLOCK - base
        moved = min(int(torch.randint(0, k + 1, (1,), generator=cpu)), max(0, n - first))
        paths[s, :k - moved] = torch.arange(k - moved)
        if moved:
            paths[s, k - moved:k] = (first + torch.randperm(n - first, generator=cpu)[:moved].sort().values).to(torch.int32)
        lens.append(k)
    st["paths"], st["path_lens"] = paths.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["new_lens"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    return st


def _inputs(case, seed):
    """Everything a user's program holds before the call, but for the pool's handle."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed * 7 + 2)
    make = {"norm": _norm_inputs, "tree": _tree_inputs, "accept": _accept_inputs}
    return make[case["op"]](case, {"case": dict(case)}, gen, cpu)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from paged_kv_cache_270_gb300.pool import KVPool, make_rope, make_rope_axes

        pool = KVPool(case.get("layers", 1), st["blocks"], case["H"], case["D"], case["kv"], K_SCALE, V_SCALE)
        pool.k_cache.copy_(st["k_cache"])
        pool.v_cache.copy_(st["v_cache"])
        st["pool"], st["k_cache"], st["v_cache"] = pool, pool.k_cache, pool.v_cache
        if case["op"] == "norm":
            st["rope"] = make_rope(case["rot"], layout=case["layout"], theta=_theta(case))
            if case["axes"] == "one":
                st["axes"] = None
            else:
                st["axes"] = make_rope_axes(_sections(case), order=case["axes"])
        if case["op"] == "tree":
            n = pool.tree_workspace_bytes(case["Hq"], case["nodes"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------- the plain forms
def _values(case, st, which):
    """The region as the elements it stands for, [layers, blocks, H, 16, D], without their scales."""
    L = case.get("layers", 1)
    n = L * st["blocks"] * case["H"] * BLOCK * case["D"] * _elem(case["kv"])
    t = st[which][:n].view(torch.float8_e4m3fn if case["kv"].startswith("fp8") else _dtype(case["kv"]))
    return t.view(L, st["blocks"], case["H"], BLOCK, case["D"])


def _tile_scales(case, st, which):
    tiles = case.get("layers", 1) * st["blocks"] * case["H"]
    n = tiles * BLOCK * case["D"]
    return st[which][n:n + tiles * 4].view(torch.float32).view(-1, st["blocks"], case["H"])


def _caches(case, st):
    """The written regions, and a block-scaled pool's scales."""
    out = [_values(case, st, "k_cache"), _values(case, st, "v_cache")]
    if case["kv"] == "fp8_e4m3_block":
        out += [_tile_scales(case, st, "k_cache"), _tile_scales(case, st, "v_cache")]
    return out


def _codes(x):
    return x.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _put(case, st, which, x, scale):
    """x [T, H, D] in 32 bits into the slots of a region."""
    region, slots, kv = _values(case, st, which)[0], st["slots"], case["kv"]
    blk, off = slots // BLOCK, slots % BLOCK
    if kv == "fp8_e4m3_block":
        # every run starts its tile afresh; the tile's scale is that of its written rows
        tile = torch.zeros(st["blocks"], BLOCK, case["H"], case["D"], device="cuda")
        tile[blk, off] = x
        s = tile.abs().amax((1, 3)) / FP8_MAX
        _tile_scales(case, st, which)[0][blk] = s[blk]
        sx = s[blk].unsqueeze(-1)
        q = _codes(torch.where(sx > 0, x / sx, torch.zeros_like(x)))
        region.view(torch.uint8)[blk, :, off] = q.view(torch.uint8)
        return
    keep = (slots >= 0).nonzero().squeeze(1)
    x = x[keep]
    if kv == "fp8_e4m3":
        q = _codes(x / torch.tensor(scale, dtype=torch.float32, device="cuda"))
        region.view(torch.uint8)[blk[keep], :, off[keep]] = q.view(torch.uint8)
    else:
        region[blk[keep], :, off[keep]] = x.to(region.dtype)


def _normed(case, x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + case["offset"])


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


def _plain_norm(case, st):
    angle = st["positions"][st["axis"]].T.double() * st["speed"]  # [T, pairs], in 64 bits: far positions
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    q = _rotate(_normed(case, st["q"], st["q_weight"]), cos, sin, case["rot"], case["layout"])
    k = _rotate(_normed(case, st["k"], st["k_weight"]), cos, sin, case["rot"], case["layout"])
    _put(case, st, "k_cache", k, K_SCALE)
    _put(case, st, "v_cache", st["v"].float(), V_SCALE)
    return [q.to(st["q"].dtype)] + _caches(case, st)


def _gather(case, st, which, scale):
    """Every sequence's keys or values in 32 bits, [S, H, tokens, D]."""
    t = st["tables"].long().clamp_min(0)
    S, P = t.shape
    x = _values(case, st, which)[0]
    x = (x.view(torch.uint8)[t].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[t]).float()  # [S, P, H, 16, D]
    if case["kv"] == "fp8_e4m3_block":
        x *= _tile_scales(case, st, which)[0][t].view(S, P, case["H"], 1, 1)
    elif case["kv"] == "fp8_e4m3":
        x *= torch.tensor(scale, dtype=torch.float32, device="cuda")
    return x.permute(0, 2, 1, 3, 4).reshape(S, case["H"], P * BLOCK, case["D"])


def _plain_tree(case, st):
    S, H, D, N = case["S"], case["H"], case["D"], case["nodes"]
    G = case["Hq"] // H
    start = st["q_start"].long()
    size = start[1:] - start[:-1]
    node = torch.arange(N, device="cuda")
    here = node < size.unsqueeze(1)  # [S, N]
    row = (start[:-1].unsqueeze(1) + node).clamp_max(st["q"].shape[0] - 1)
    W = st["tables"].shape[1] * BLOCK
    at = torch.arange(W, device="cuda") - (st["ctx"].long() - size).unsqueeze(1)  # [S, W]: its place in the tree
    word = st["mask"][row]  # [S, N, words]
    of = at.clamp(0, N - 1).unsqueeze(1).expand(S, N, W)
    bit = (word.gather(2, of // 64) >> (of % 64)) & 1
    sees = ((at < 0).unsqueeze(1) | ((bit == 1) & (at < size.unsqueeze(1)).unsqueeze(1))).unsqueeze(1).unsqueeze(3)  # [S, 1, N, 1, W]
    q = (st["q"].float()[row] * st["scale"]).view(S, N, H, G, D).transpose(1, 2).reshape(S, H, N * G, D)
    x = (q @ _gather(case, st, "k_cache", K_SCALE).transpose(2, 3)).view(S, H, N, G, W)
    x = x.masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = (x - m).exp()
    l = e.sum(-1, keepdim=True)
    p = torch.where(l > 0, e / l, torch.zeros_like(e)).view(S, H, N * G, W)
    v = _gather(case, st, "v_cache", V_SCALE).masked_fill((torch.arange(W, device="cuda") >= st["ctx"].unsqueeze(1)).view(S, 1, W, 1), 0.0)
    out = (p @ v).view(S, H, N, G, D).transpose(1, 2).reshape(S, N, H * G, D)
    got = torch.zeros_like(st["q"])
    got[(torch.arange(S * N, device="cuda") < start[-1])] = out[here].to(st["q"].dtype)
    return got


def _plain_accept(case, st):
    S, H, P = case["S"], case["H"], case["path"]
    lens = st["path_lens"].long()
    start = st["q_start"].long()
    base = st["ctx"].long() - (start[1:] - start[:-1])
    i = torch.arange(P, device="cuda")
    path = st["paths"].long()
    live = (i < lens.unsqueeze(1)) & (path != i)  # [S, P]: the rows that move
    tables = st["tables"].long()
    src = base.unsqueeze(1) + path.clamp_min(0)
    dst = base.unsqueeze(1) + i
    last = tables.shape[1] - 1
    sblk, dblk = (tables.gather(1, (x // BLOCK).clamp_max(last))[live] for x in (src, dst))
    soff, doff = (src % BLOCK)[live], (dst % BLOCK)[live]
    _moves(case, st, "k_cache", sblk, soff, dblk, doff)
    _moves(case, st, "v_cache", sblk, soff, dblk, doff)
    return _caches(case, st) + [(base + lens).to(torch.int32)]


def _moves(case, st, which, sblk, soff, dblk, doff):
    region = _values(case, st, which)  # [L, B, H, 16, D]
    raw = region.view(torch.uint8) if region.dtype == torch.float8_e4m3fn else region
    rows = raw[:, sblk, :, soff]  # [moved, L, H, D]
    if case["kv"] == "fp8_e4m3_block":
        scales = _tile_scales(case, st, which)  # [L, B, H]
        x = rows.view(torch.float8_e4m3fn).float() * scales[:, sblk].permute(1, 0, 2).unsqueeze(-1)  # [moved, L, H, D]
        # a tile's scale grows to hold the rows that come from other tiles; its own codes follow
        need = (x.abs().amax(-1) / FP8_MAX).permute(1, 0, 2) * (sblk != dblk).view(1, -1, 1)  # [L, moved, H]
        new = scales.clone().scatter_reduce_(1, dblk.view(1, -1, 1).expand_as(need), need, "amax")
        grown = (new > scales).view(*new.shape, 1, 1)
        held = region.float() * scales.view(*new.shape, 1, 1) / torch.where(new > 0, new, torch.ones_like(new)).view(*new.shape, 1, 1)
        raw.copy_(torch.where(grown, _codes(held).view(torch.uint8), raw))
        scales.copy_(new)
        s = new[:, dblk].permute(1, 0, 2).unsqueeze(-1)
        rows = _codes(torch.where(s > 0, x / s, torch.zeros_like(x))).view(torch.uint8)
    raw[:, dblk, :, doff] = rows


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "tree": _plain_tree, "accept": _plain_accept}[op](case, st)
    pool = st["pool"]
    if op == "norm":
        positions = st["positions"] if st["axes"] is not None else st["positions"][0]
        q = pool.norm_rope_and_cache(st["rope"], st["q"], st["k"], st["v"], positions, st["slots"], q_weight=st["q_weight"],
                                     k_weight=st["k_weight"], eps=EPS, weight_offset=case["offset"], axes=st["axes"], q_out=st["q_out"])
        return [q] + _caches(case, st)
    if op == "tree":
        return pool.decode_tree(st["q"], st["q_start"], st["tables"], st["ctx"], case["nodes"], mask=st["mask"],
                                softmax_scale=st["scale"], out=st["out"], workspace=st["workspace"])
    lens = pool.tree_accept(st["paths"], st["path_lens"], st["q_start"], st["tables"], st["ctx"], new_lens=st["new_lens"])
    return _caches(case, st) + [lens]


def work(case):
    """With the mean lengths and sizes that a seed draws."""
    op, H, D = case["op"], case["H"], case["D"]
    if op == "norm":
        T, Hq = case["T"], case["Hq"]
        axes = 1 if case["axes"] == "one" else 3
        return {"bytes": T * (4 * Hq * D + 4 * H * D + 2 * H * D * _elem(case["kv"]) + 8 + 4 * axes),
                "flops": T * (Hq + H) * (3 * case["rot"] + 4 * D)}
    S = case["S"]
    nodes = (S - 1) * (case["few"] + case["nodes"]) / 2 + case["nodes"]
    if op == "accept":
        half = min(case["path"], nodes / S) / 4 if S > 1 else case["path"] / 4  # rows that move, on average
        moved = S * half * case["layers"]
        return {"bytes": moved * H * 4 * D * _elem(case["kv"]) + 4 * S * (case["path"] + 4), "flops": 0}
    mean = max((case["shortest"] + case["longest"]) / 2, nodes / S)
    tokens = (S - 1) * mean + case["longest"]
    return {"bytes": tokens * H * 2 * D * _elem(case["kv"]) + 4 * nodes * case["Hq"] * D + 8 * nodes * -(-case["nodes"] // 64) + tokens / 4,
            "flops": 4 * tokens / S * nodes * case["Hq"] * D}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """What `run` returns, from the definitions, in 64 bits; None where codes or whole numbers are held."""
    st = _inputs(case, seed)
    coded = case["kv"].startswith("fp8")
    return {"norm": _exact_norm, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](case, st, coded)


def _exact_norm(case, st, coded):
    H, D, R = case["H"], case["D"], case["rot"]
    speed = [_theta(case) ** (-2.0 * i / R) for i in range(R // 2)]
    pos = torch.stack([st["positions"][a] for a in _axis_of(case)], 1).double()  # [T, pairs]
    turn = pos * torch.tensor(speed, dtype=torch.float64, device="cuda")
    spin = torch.polar(torch.ones_like(turn), turn).unsqueeze(1)

    def turned(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * (case["offset"] + w.double())
        if case["layout"] == "half":
            z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * spin
            y = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], R // 2, 2).contiguous()) * spin
            y = torch.view_as_real(z).reshape(*x.shape[:2], R)
        return torch.cat([y, x[..., R:]], -1)

    q = turned(st["q"], st["q_weight"])
    if coded:
        return [q, None, None] + ([None, None] if case["kv"] == "fp8_e4m3_block" else [])
    got = [q]
    use = st["slots"] >= 0
    flat = st["slots"][use]
    for which, x in (("k_cache", turned(st["k"], st["k_weight"])), ("v_cache", st["v"].double())):
        pages = st[which].view(_dtype(case["kv"])).double().view(st["blocks"], H, BLOCK, D).transpose(1, 2).reshape(-1, H, D)
        pages[flat] = x[use]
        got.append(pages.view(st["blocks"], BLOCK, H, D).transpose(1, 2).unsqueeze(0).contiguous())
    return got


def _exact_tree(case, st, coded):
    H, D, kv = case["H"], case["D"], case["kv"]
    G = case["Hq"] // H
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    size = BLOCK * D * _elem(kv)
    at = 0
    for s, (n, k) in enumerate(zip(st["lengths"], st["sizes"])):
        ids = st["tables"][s, :-(-n // BLOCK)].long()
        rows = {}
        for which, scale in (("k_cache", K_SCALE), ("v_cache", V_SCALE)):
            raw = st[which][:st["blocks"] * H * size].view(st["blocks"], H * size)[ids]
            x = raw.view(torch.float8_e4m3fn if coded else _dtype(kv)).double().view(-1, H, BLOCK, D)
            if kv == "fp8_e4m3":
                x = x * float(torch.tensor(scale, dtype=torch.float32))
            if kv == "fp8_e4m3_block":
                end = st["blocks"] * H * size
                sc = st[which][end:end + st["blocks"] * H * 4].view(torch.float32).view(-1, H)[ids]
                x = x * sc.double()[:, :, None, None]
            rows[which] = x.transpose(0, 1).reshape(H, -1, D)[:, :n]
        hidden = torch.zeros(k, n, dtype=torch.bool)
        hidden[:, n - k:] = ~st["sees"][s, :k, :k]
        hidden = hidden.cuda().unsqueeze(1)
        for h in range(H):
            q = st["q"][at:at + k, h * G:(h + 1) * G].double()
            z = (q.reshape(k * G, D) @ rows["k_cache"][h].T * st["scale"]).view(k, G, n).masked_fill(hidden, -math.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)  # (a row that sees nothing)
            out[at:at + k, h * G:(h + 1) * G] = (p.view(k * G, n) @ rows["v_cache"][h]).view(k, G, D)
        at += k
    return out


def _exact_accept(case, st, coded):
    if coded:
        return None
    L, H, D = case["layers"], case["H"], case["D"]
    got = []
    paths, lens = st["paths"].cpu(), st["path_lens"].tolist()
    for which in ("k_cache", "v_cache"):
        old = st[which].view(_dtype(case["kv"])).double().view(L, st["blocks"], H, BLOCK, D)
        new = old.clone()
        for s, k in enumerate(lens):
            base = st["lengths"][s] - st["sizes"][s]
            for i in range(k):
                a, b = base + int(paths[s, i]), base + i
                new[:, st["tables"][s, b // BLOCK].long(), :, b % BLOCK] = old[:, st["tables"][s, a // BLOCK].long(), :, a % BLOCK]
        got.append(new)
    return got + [None]
