"""pa_evict_select and pa_evict_compact against plain numpy / torch on the CPU
(exact: the selection is a ranking, the move a copy or a rounding that IEEE
arithmetic fixes), and the whole path that an eviction takes."""
import math

import numpy as np
import pytest
import torch

from gpu_harness import bits_to_torch
from paged_kv_cache_270_gb300 import _native as N
from paged_kv_cache_270_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _pool(kv="bf16", H=2, D=64, blocks=4, layers=1):
    from paged_kv_cache_270_gb300.pool import KVPool
    return KVPool(layers, blocks, H, D, kv, 0.02, 0.03)


# ------------------------------------------------------------------ selection
def _choose(w, n, budget, sinks, recent):
    """One row: the definition, by a stable sort."""
    if n <= budget:
        return np.concatenate([np.arange(n), np.full(budget - n, -1)])
    mid = w[sinks:n - recent].astype(np.float64)
    rank = np.where(np.isnan(mid), -np.inf, mid)
    # NaN below every number, -inf among them; lower tokens first
    order = np.lexsort((np.arange(len(mid)), -rank, np.isnan(mid)))
    took = np.sort(order[:budget - sinks - recent]) + sinks
    return np.concatenate([np.arange(sinks), took, np.arange(n - recent, n)])


def _check_select(w, ctx, budget, sinks, recent):
    pool = _pool()
    t = torch.from_numpy(w).cuda()
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    keep, kept = pool.evict_select(t, c, budget, sinks=sinks, recent=recent)
    assert pool.device_error() == N.PA_OK
    assert kept.tolist() == [min(n, budget) for n in ctx]
    got = keep.cpu().numpy()
    for s, n in enumerate(ctx):
        for h in range(w.shape[1]):
            assert np.array_equal(got[s, h], _choose(w[s, h], n, budget, sinks, recent)), (s, h)
    pool.close()


def _totals(kind, shape, rng):
    if kind == "heavy":  # a few tokens hold most, some hold exactly nothing
        return (np.exp(2.5 * rng.standard_normal(shape)) * (rng.random(shape) > 0.3)).astype(np.float32)
    if kind == "zero":
        return np.zeros(shape, np.float32)
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "close":  # neighbours in the last place
        return (np.uint32(0x3F800000) + rng.integers(0, 40, shape).astype(np.uint32)).view(np.float32)
    x = rng.standard_normal(shape).astype(np.float32)  # any bits: signs, infinities, NaN, both zeros
    for value in (np.inf, -np.inf, np.nan, 0.0, -0.0, -np.nan, 1e-45, -1e-45, 3.4e38):
        x[rng.random(shape) < 0.04] = value
    return x


@pytest.mark.parametrize("kind", ["heavy", "zero", "ties", "close", "any"])
@pytest.mark.parametrize("tokens, ctx, heads, budget, sinks, recent", [
    (64, [64, 0, 1, 33, 63, 32], 3, 32, 4, 8), (7, [7], 1, 1, 0, 0), (100, [100, 51], 2, 50, 25, 25),
    (100, [100, 99], 1, 99, 0, 0), (100, [100, 3], 2, 1, 1, 0), (100, [100], 1, 1, 0, 1), (50, [50, 20], 2, 400, 5, 5),
    (4001, [4001, 513, 2000], 2, 511, 4, 100), (8193, [8193, 8192, 100], 1, 1000, 3, 17),
    (30000, [30000, 29999], 1, 4000, 1, 31), (65535, [65535, 1025], 2, 1024, 0, 500)])
def test_select(kind, tokens, ctx, heads, budget, sinks, recent):
    rng = np.random.default_rng([tokens, budget])
    w = _totals(kind, (len(ctx), heads, tokens), rng)
    for s, n in enumerate(ctx):
        w[s, :, n:] = np.nan  # behind the context: not read
    _check_select(w, ctx, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["heavy", "zero", "any"])
def test_select_long(kind):
    """Eight CTAs per row; shares beyond what they keep in shared memory."""
    rng = np.random.default_rng(5)
    _check_select(_totals(kind, (1, 2, 131072), rng), [131072], 16384, 4, 1024)
    _check_select(_totals(kind, (2, 1, 420001), rng), [420001, 394000], 100000, 0, 3)


def test_select_many_rows():
    rng = np.random.default_rng(6)
    ctx = [int(x) for x in rng.integers(0, 700, 300)]
    _check_select(_totals("heavy", (300, 8, 700), rng), ctx, 200, 4, 64)


def test_select_bounds_and_wrapper():
    pool = _pool()
    w = torch.arange(32, dtype=torch.float32, device="cuda").view(1, 1, 32)
    keep, kept = pool.evict_select(w, torch.tensor([40], dtype=torch.int32, device="cuda"), 4)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    assert keep.flatten().tolist() == [28, 29, 30, 31] and kept.tolist() == [4]
    keep, kept = pool.evict_select(w, torch.tensor([-3], dtype=torch.int32, device="cuda"), 4)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    assert keep.flatten().tolist() == [-1] * 4 and kept.tolist() == [0]
    c = torch.tensor([32], dtype=torch.int32, device="cuda")
    for bad in (dict(weights=w.double()), dict(weights=w[0]), dict(ctx=c.long()), dict(ctx=torch.cat([c, c])),
                dict(weights=torch.zeros(1, 32, 2, device="cuda").transpose(1, 2)), dict(keep=c)):
        a = dict(weights=w, ctx=c, keep=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            pool.evict_select(a["weights"], a["ctx"], 4, keep=a["keep"])
    with pytest.raises(N.PAError):
        pool.evict_select(w, c, 4, sinks=3, recent=2)
    for budget in (0, -1):
        with pytest.raises(N.PAError):
            pool.evict_select(w, c, budget)
    pool.close()


# ----------------------------------------------------------------- compaction
def _fill(pool, seed):
    """Random finite cache bytes (and tile scales)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for which in ("k", "v"):
        for layer in range(pool.n_layers):
            v = pool.layer_view(which, layer)
            x = torch.randn(v.shape[:3] + (pool.head_dim,), device="cuda", generator=g)
            if pool.elem_bytes == 1:
                v.copy_((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            else:
                v.copy_(x.to(pool.in_dtype).view(torch.uint8))
            if pool.block_scaled:
                pool.scale_view(which, layer).copy_(
                    torch.rand(pool.num_blocks, pool.n_kv_heads, device="cuda", generator=g) * 0.1)


def _expect(pool, which, keep, kept, src, dst, layer=0):
    """The layer after the move, from its bytes before it, on the CPU."""
    tiles = pool.layer_view(which, layer).cpu().clone()
    scales = pool.scale_view(which, layer).cpu().clone() if pool.block_scaled else None
    before, sbefore = tiles.clone(), scales.clone() if scales is not None else None
    for s, n in enumerate(kept):
        for h in range(pool.n_kv_heads):
            row = keep[s, h if keep.shape[1] > 1 else 0]
            for p in range(-(-n // 16)):
                toks = row[16 * p:min(n, 16 * p + 16)]
                blk, off = src[s, toks // 16].astype(np.int64), toks % 16
                rows = before[blk, h, off]
                d = int(dst[s, p])
                if pool.block_scaled:
                    v = rows.view(torch.float8_e4m3fn).float() * sbefore[blk, h].view(-1, 1)
                    scale = v.abs().max() / torch.tensor(448.0)
                    ratio = sbefore[blk, h].view(-1, 1) / scale if scale > 0 else torch.zeros(len(blk), 1)
                    rows = (rows.view(torch.float8_e4m3fn).float() * ratio).clamp(-448, 448)
                    rows = rows.to(torch.float8_e4m3fn).view(torch.uint8)
                    scales[d, h] = scale
                tiles[d, h, :len(toks)] = rows
    return tiles, scales


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("D, H, heads, ctx, budget", [
    (64, 2, 2, [100, 5, 0, 33], 40), (128, 1, 1, [257, 17], 31), (128, 4, 1, [64, 300], 64), (64, 3, 3, [1, 16, 500], 16),
    (128, 8, 8, [900, 48, 1000], 333)])
def test_compact(kv, D, H, heads, ctx, budget):
    rng = np.random.default_rng([D, budget])
    S = len(ctx)
    kept = [min(n, budget) for n in ctx]
    src_n, dst_n = -(-max(ctx) // 16) + 1, -(-budget // 16) + 1
    need = [-(-n // 16) for n in ctx] + [-(-n // 16) for n in kept]
    pool = _pool(kv, H, D, sum(need) + 2, layers=2)
    _fill(pool, budget)
    ids = rng.permutation(pool.num_blocks).astype(np.int32)
    src, dst = np.full((S, src_n), -9, np.int32), np.full((S, dst_n), 10 ** 8, np.int32)
    at = 0
    for s in range(S):
        for t, n in ((src, ctx[s]), (dst, kept[s])):
            t[s, :-(-n // 16)] = ids[at:at + -(-n // 16)]
            at += -(-n // 16)
    keep = np.full((S, heads, budget), -1, np.int32)
    for s in range(S):
        for h in range(heads):
            keep[s, h, :kept[s]] = np.sort(rng.permutation(ctx[s])[:kept[s]])
    w = rng.random((S, heads, max(ctx))).astype(np.float32)
    want = {x: _expect(pool, x, keep, kept, src, dst, layer=1) for x in ("k", "v")}
    layer0 = {x: pool.layer_view(x, 0).clone() for x in ("k", "v")}
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    wout = torch.full((S, heads, max(ctx) + 77), 5.0, device="cuda")
    got = pool.evict_compact(dev(keep), torch.tensor(kept, dtype=torch.int32, device="cuda"), dev(src), dev(dst),
                             weights=dev(w), weights_out=wout, layer=1)
    assert pool.device_error() == N.PA_OK
    for x in ("k", "v"):
        assert torch.equal(pool.layer_view(x, 1).cpu(), want[x][0]), x
        assert torch.equal(pool.layer_view(x, 0), layer0[x])
        if pool.block_scaled:
            assert torch.equal(pool.scale_view(x, 1).cpu(), want[x][1])
    ref = np.zeros(wout.shape, np.float32)
    for s in range(S):
        for h in range(heads):
            ref[s, h, :kept[s]] = w[s, h, keep[s, h, :kept[s]]]
    assert np.array_equal(got.cpu().numpy(), ref)
    # without totals the caches end the same
    pool.evict_compact(dev(keep), torch.tensor(kept, dtype=torch.int32, device="cuda"), dev(src), dev(dst), layer=1)
    assert torch.equal(pool.layer_view("k", 1).cpu(), want["k"][0])
    pool.close()


def test_compact_bad_input_is_skipped():
    """Tokens outside the table, ids outside the pool and lengths past the budget are
    reported; their rows stay, the others move."""
    pool = _pool("bf16", 1, 64, 6)
    _fill(pool, 1)
    before = pool.layer_view("k").clone()
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    src, dst = dev([0, 1, 99]), dev([4, -1])
    keep = dev([[3, 48, -7, 40, 17]])  # 48 and -7 outside the table, 40 in a bad block

    def move(keep, kept, dst):
        pool.evict_compact(keep, dev(kept), src, dst)
        return pool.device_error()

    assert move(keep, 5, dst) == N.PA_ERR_BOUNDS
    now = pool.layer_view("k")
    assert torch.equal(now[4, 0, 0], before[0, 0, 3]) and torch.equal(now[4, 0, 4], before[1, 0, 1])
    assert torch.equal(now[4, 0, 1:4], before[4, 0, 1:4]) and torch.equal(now[[0, 1, 2, 3, 5]], before[[0, 1, 2, 3, 5]])
    twenty = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 1, 20)
    assert move(twenty, 20, dst) == N.PA_ERR_BOUNDS  # the second page's id is bad
    assert torch.equal(pool.layer_view("k")[4, 0], before[0, 0]) and torch.equal(pool.layer_view("k")[5], before[5])
    assert move(twenty, 21, dev([4, 5])) == N.PA_ERR_BOUNDS
    assert move(twenty, -1, dev([4, 5])) == N.PA_ERR_BOUNDS
    assert move(twenty, 20, dev([4])) == N.PA_ERR_BOUNDS  # more than the table's blocks hold
    assert move(twenty, 20, dev([4, 5])) == N.PA_OK
    w = torch.ones(1, 1, 10, device="cuda")
    pool.evict_compact(twenty, dev(20), src, dev([4, 5]), weights=w)  # totals shorter than the tokens
    assert pool.device_error() == N.PA_ERR_BOUNDS
    with pytest.raises(N.PAError):
        pool.evict_compact(twenty, dev(20), src, src)
    for bad in (dict(weights=w.double()), dict(weights=w[0]), dict(weights_out=w), dict(keep=keep[0, 0]), dict(src=src[0])):
        a = dict(keep=keep, src=src, weights=None, weights_out=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            pool.evict_compact(a["keep"], dev(5), a["src"], dst, weights=a["weights"], weights_out=a["weights_out"])
    pool.close()


# ------------------------------------------------------------- the whole path
@pytest.mark.parametrize("kv", ["fp16", "fp8_e4m3_block"])
def test_generation_under_a_budget(kv):
    """A prompt and 40 decode steps with the cache held to a budget: rotary write, decode
    with totals, selection and move together, positions running on past the evictions.
    A model in fp64 follows with the bytes of the pool: it checks every output and every
    total, and evicts the tokens that the totals say."""
    from paged_kv_cache_270_gb300.pool import make_rope
    S, H, G, D, budget, sinks, recent, prompt, steps = 3, 2, 4, 64, 48, 4, 12, [70, 50, 9], 40
    Hq, width = H * G, 6
    pool = _pool(kv, H, D, 64)
    pool.k_cache.fill_(0xFF)
    pool.v_cache.fill_(0xFF)
    if pool.block_scaled:
        pool.scale_view("k").fill_(math.nan)
        pool.scale_view("v").fill_(math.nan)
    dtype = pool.in_dtype
    rope = make_rope(D, "interleaved", scaling="bands", factor=4.0, original_len=64)
    g = torch.Generator(device="cuda").manual_seed(1)
    tables = np.zeros((S, width), np.int32)
    owned = [list(pool.alloc(-(-n // 16))) for n in prompt]
    for s in range(S):
        tables[s, :len(owned[s])] = owned[s]
    ctx, pos = np.array(prompt, np.int32), np.array(prompt)
    weights = torch.zeros(S, H, width * 16, device="cuda")
    model_w = np.zeros((S, H, width * 16))

    def rand(T):
        x = torch.randn(T, Hq + 2 * H, D, device="cuda", generator=g).to(dtype)
        return x[:, :Hq] * 2, x[:, Hq:Hq + H], x[:, Hq + H:]

    def write(T, positions, slots):
        q, k, v = rand(T)
        return pool.rope_and_cache(rope, q, k, v, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                                   torch.tensor(slots, device="cuda"))

    def values(which):  # what the pool holds, in fp64
        x = pool.layer_view(which).cpu()
        if pool.elem_bytes == 1:
            return x.view(torch.float8_e4m3fn).double().numpy() * pool.scale_view(which).cpu().double().numpy()[:, :, None, None]
        return x.view(dtype).double().numpy()

    for s in range(S):
        write(prompt[s], list(range(prompt[s])), [int(tables[s, i // 16]) * 16 + i % 16 for i in range(prompt[s])])
    evictions = 0
    for step in range(steps):
        slots = []
        for s in range(S):
            if ctx[s] % 16 == 0:
                owned[s] += list(pool.alloc(1))
                tables[s, ctx[s] // 16] = owned[s][-1]
            slots.append(int(tables[s, ctx[s] // 16]) * 16 + int(ctx[s]) % 16)
        q = write(S, pos.tolist(), slots)
        ctx += 1
        pos += 1
        dt, dc = torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()
        out, _ = pool.decode_weights(q, dt, dc, weights, decay=0.9, out_dtype=torch.float32)
        k, v = values("k"), values("v")
        qd = q.double().cpu().numpy().reshape(S, H, G, D)
        model_w *= 0.9
        for s in range(S):
            n = int(ctx[s])
            i = np.arange(n)
            for h in range(H):
                ks, vs = (x[tables[s, i // 16], h, i % 16] for x in (k, v))
                z = qd[s, h] @ ks.T / math.sqrt(D)
                p = np.exp(z - z.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                ref = p @ vs
                o = out[s, h * G:(h + 1) * G].double().cpu().numpy()
                assert np.abs(o - ref).max() <= 1e-4 * np.abs(ref).max()
                model_w[s, h, :n] += p.sum(0)
        got = weights.double().cpu().numpy()
        # each step adds a weight off by at most 7e-4 (the bound of pa_decode_weights, with
        # |q| |k| scale log2(e) < 60 here) and two roundings
        assert np.all(np.abs(got - model_w) <= 1e-3 * model_w + 1e-30)
        if step % 13 == 12:
            keep, kept = pool.evict_select(weights, dc, budget, sinks=sinks, recent=recent)
            kh, nh = keep.cpu().numpy(), kept.cpu().numpy()
            dst, fresh = np.zeros_like(tables), []
            for s in range(S):
                fresh.append(list(pool.alloc(-(-int(nh[s]) // 16))))
                dst[s, :len(fresh[s])] = fresh[s]
            new_w = pool.evict_compact(keep, kept, dt, torch.from_numpy(dst).cuda(), weights=weights)
            for s in range(S):
                pool.free(owned[s])
                evictions += int(nh[s] < ctx[s])
                for h in range(H):
                    assert np.array_equal(kh[s, h], _choose(weights[s, h].cpu().numpy(), int(ctx[s]), budget, sinks, recent))
                    took = model_w[s, h, kh[s, h, :nh[s]]]
                    model_w[s, h] = 0
                    model_w[s, h, :nh[s]] = took
            weights, owned, tables, ctx = new_w, fresh, dst, nh.astype(np.int32)
            assert pool.stats()[0] == sum(len(x) for x in owned)
    assert pool.device_error() == N.PA_OK
    assert evictions >= 5 and int(pos.max()) > int(ctx.max())
    pool.close()


def test_path_in_one_graph():
    """Rotary write, decode with totals, selection and move captured as one graph and
    replayed: the same bits as the calls one by one."""
    from paged_kv_cache_270_gb300.pool import make_rope
    S, H, Hq, D, n, budget = 4, 2, 8, 128, 100, 40
    pool = _pool("fp8_e4m3", H, D, 64)
    _fill(pool, 3)
    rope = make_rope(D)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(S, Hq + 2 * H, D, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randperm(64, device="cuda", generator=g).to(torch.int32)
    tables, dst = ids[:28].view(S, 7).contiguous(), ids[28:40].view(S, 3).contiguous()
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    slots = tables[:, (n - 1) // 16].long() * 16 + (n - 1) % 16
    positions = torch.full((S,), 5000, dtype=torch.int32, device="cuda")
    start = torch.rand(S, H, 112, device="cuda", generator=g)
    start[..., n:] = 0
    w, w2 = start.clone(), torch.empty_like(start)
    q, out = torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda")
    keep, kept = torch.empty(S, H, budget, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    ws = torch.empty(pool.weights_workspace_bytes(S, Hq, 7), dtype=torch.uint8, device="cuda")

    def path():
        pool.rope_and_cache(rope, x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], positions, slots, q_out=q)
        pool.decode_weights(q, tables, ctx, w, out=out, workspace=ws)
        pool.evict_select(w, ctx, budget, sinks=2, recent=10, keep=keep, kept_lens=kept)
        pool.evict_compact(keep, kept, tables, dst, weights=w, weights_out=w2)

    path()
    torch.cuda.synchronize()
    want = [t.clone() for t in (q, out, keep, kept, w, w2, pool.k_cache, pool.v_cache)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path()
    for t in (q, out, keep, kept, w2):
        t.zero_()
    w.copy_(start)
    _fill(pool, 3)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (q, out, keep, kept, w, w2, pool.k_cache, pool.v_cache)):
        assert torch.equal(a, b)
    assert pool.device_error() == N.PA_OK
    pool.close()
