"""Edges of the rotary write and the eviction path: byte offsets past 32 bits in the
cache, the totals and the workspace, other streams, score scales, infinities in the
cache, two captured graphs that share a workspace."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _pool(kv, H, D, blocks, layers=1):
    from paged_kv_cache_270_gb300.pool import KVPool
    return KVPool(layers, blocks, H, D, kv, 0.02, 0.03)


def _path(pool, tables, dst, seed=0, n=77, budget=30):
    """Writes n tokens per sequence, decodes with totals, selects and compacts; what each
    step left, in the order of the sequences' tokens."""
    from paged_kv_cache_270_gb300.pool import make_rope
    S, H, D, Hq = tables.shape[0], pool.n_kv_heads, pool.head_dim, 4 * pool.n_kv_heads
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(S * n, Hq + 2 * H, D, device="cuda", generator=g).to(pool.in_dtype)
    at = torch.arange(n, device="cuda")
    slots = (tables[:, at // 16].long() * 16 + at % 16).flatten().contiguous()
    pos = at.repeat(S).to(torch.int32)
    q = pool.rope_and_cache(make_rope(D), x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], pos, slots)
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    last = q.view(S, n, Hq, D)[:, -1].contiguous()
    w = torch.zeros(S, H, n, device="cuda")
    out, w = pool.decode_weights(last, tables, ctx, w)
    keep, kept = pool.evict_select(w, ctx, budget, sinks=2, recent=8)
    w2 = pool.evict_compact(keep, kept, tables, dst, weights=w)
    assert pool.device_error() == N.PA_OK
    pages = [pool.layer_view(c)[t.long()] for c in "kv" for t in (tables, dst[:, :-(-budget // 16)])]
    return [q, out, w, keep, kept, w2, pool.decode(last, dst, kept, num_splits=1)] + [p.clone() for p in pages]


@pytest.mark.parametrize("kv, H, blocks", [("bf16", 8, 140000), ("fp8_e4m3", 16, 140000)])
def test_cache_offsets_past_32_bits(kv, H, blocks):
    """The last blocks of a layer of more than 2^32 bytes give the bits that the first
    blocks of a small pool give."""
    big, small = _pool(kv, H, 128, blocks), _pool(kv, H, 128, 40)
    assert big.layer_bytes > 2 ** 32
    ids = torch.randperm(40, device="cuda").to(torch.int32)
    t, d = ids[:20].view(4, 5).contiguous(), ids[20:28].view(4, 2).contiguous()
    # rows of a page that no token was written to hold anything: the same in both
    small.k_cache.zero_()
    small.v_cache.zero_()
    for c in "kv":
        big.layer_view(c)[blocks - 40:].zero_()
    for a, b in zip(_path(small, t, d), _path(big, t + (blocks - 40), d + (blocks - 40))):
        assert torch.equal(a, b)
    big.close()
    small.close()


def test_totals_and_scores_past_32_bits():
    """A workspace of more than 2^32 bytes of scores (a very wide table), and totals' rows
    more than 2^32 bytes apart."""
    pool = _pool("bf16", 8, 64, 600)
    S, Hq, n = 64, 64, 100
    tables = torch.randperm(600, device="cuda")[:S * 7].to(torch.int32).view(S, 7)
    wide = torch.full((S, 40000), -1, dtype=torch.int32, device="cuda")
    wide[:, :7] = tables
    pool.k_cache.view(torch.bfloat16).normal_()
    pool.v_cache.view(torch.bfloat16).normal_()
    q = torch.randn(S, Hq, 64, device="cuda").to(torch.bfloat16)
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    assert pool.weights_workspace_bytes(S, Hq, 40000) > 10 ** 10
    out, w = pool.decode_weights(q, tables.contiguous(), ctx, None, weights_out=torch.zeros(S, 8, n, device="cuda"))
    out2, w2 = pool.decode_weights(q, wide, ctx, None, weights_out=torch.zeros(S, 8, n, device="cuda"))
    # (another schedule: the sums are taken in another order, 100 terms at most)
    assert torch.allclose(w, w2, rtol=110 * 2.0 ** -23, atol=0) and torch.allclose(out.float(), out2.float(), rtol=2.0 ** -7, atol=1e-3)
    assert pool.device_error() == N.PA_OK
    far = torch.zeros(4, 8, 40_000_000, device="cuda")  # 5 GB
    far[..., :n] = w[:4]
    far[..., n:2 * n] = 9.0
    near, kept = pool.evict_select(w[:4].contiguous(), ctx[:4], 33, sinks=1, recent=7)
    keep, kept2 = pool.evict_select(far, ctx[:4].contiguous(), 33, sinks=1, recent=7)
    assert torch.equal(keep, near) and torch.equal(kept, kept2)
    dst = torch.arange(S * 7, S * 7 + 12, device="cuda").to(torch.int32).view(4, 3)
    moved = pool.evict_compact(keep, kept, tables[:4].contiguous(), dst, weights=far)
    assert torch.equal(moved[..., :33], w[:4].gather(2, keep.long())) and not moved[..., 33:].any()
    assert pool.device_error() == N.PA_OK
    pool.close()


def test_other_stream():
    """Calls given a stream order their temporaries there, whatever the current stream does."""
    pool = _pool("fp16", 2, 64, 64)
    ids = torch.arange(28, device="cuda").to(torch.int32)
    t, d = ids[:20].view(4, 5).contiguous(), ids[20:].view(4, 2).contiguous()
    want = _path(pool, t, d)
    q, ctx = want[0].view(4, 77, 8, 64)[:, -1].contiguous(), torch.full((4,), 77, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        out, w = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(4, 2, 77, device="cuda"), stream=None)
        side.wait_stream(torch.cuda.current_stream())
        out, w = pool.decode_weights(q, t, ctx, None, weights_out=w, stream=side)
        keep, kept = pool.evict_select(w, ctx, 30, sinks=2, recent=8, stream=side)
        w2 = pool.evict_compact(keep, kept, t, d, weights=w, stream=side)
        junk = [torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(8)]  # reuses what is free
        side.synchronize()
        assert torch.equal(out, want[1]) and torch.equal(w, want[2])
        assert torch.equal(keep, want[3]) and torch.equal(w2, want[5])
        del junk
    pool.close()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_score_scales(scale):
    """Any finite scale: zero weighs all tokens the same, a negative one turns the ranking."""
    pool = _pool("fp16", 2, 64, 16)
    pool.k_cache.view(torch.float16).normal_()
    pool.v_cache.view(torch.float16).normal_()
    t = torch.arange(10, device="cuda").to(torch.int32).view(2, 5)
    ctx = torch.tensor([70, 16], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 6, 64, device="cuda").to(torch.float16)
    out, w = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(2, 2, 80, device="cuda"),
                                 softmax_scale=scale, out_dtype=torch.float32)
    k, v = (pool.layer_view(c).view(torch.float16).double()[t.long()].permute(0, 2, 1, 3, 4).reshape(2, 2, 80, 64) for c in "kv")
    there = torch.arange(80, device="cuda") < ctx.view(2, 1, 1)
    z = (q.double().view(2, 2, 3, 64) @ k.transpose(2, 3) * scale).masked_fill(~there.unsqueeze(2), -math.inf)
    p = z.softmax(-1)
    # scores off by 64 2^-23 |q| |k| |scale| log2(e) at most, twice that relative in a weight
    d = 64 * 2.0 ** -23 * float(q.double().norm(dim=-1).max() * k.norm(dim=-1).max()) * abs(scale) * math.log2(math.e)
    tol = 2 * math.log(2) * d + 100 * 2.0 ** -23
    ref = p.sum(2)
    assert bool(((w.double() - ref).abs() <= tol * ref + 1e-37).all())
    if scale == 0.0:
        assert torch.allclose(w[0, :, :70], torch.full((2, 70), 3 / 70, device="cuda"), rtol=1e-5)
    err = (out.double().view(2, 2, 3, 64) - p @ v).abs().amax(-1) / (p @ v).abs().amax(-1)
    assert float(err.max()) <= 1e-4
    pool.close()


def test_infinities_and_nan():
    """A NaN key makes its own row's weights NaN and no other's; bytes behind the context never count."""
    pool = _pool("bf16", 2, 64, 8)
    k = pool.layer_view("k").view(torch.bfloat16)
    pool.k_cache.view(torch.bfloat16).normal_()
    pool.v_cache.view(torch.bfloat16).normal_()
    t = torch.arange(6, device="cuda").to(torch.int32).view(2, 3)
    ctx = torch.tensor([40, 33], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    clean_out, clean = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(2, 2, 48, device="cuda"))
    k[2, :, 9:] = math.nan  # sequence 0, behind its 40 tokens
    pool.layer_view("v").view(torch.bfloat16)[2, :, 9:] = math.inf
    k[5, 1, 0] = math.nan   # sequence 1, head 1, its last token
    out, w = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(2, 2, 48, device="cuda"))
    assert torch.equal(w[0], clean[0]) and torch.equal(out[0], clean_out[0])
    assert torch.equal(w[1, 0], clean[1, 0]) and torch.equal(out[1, :2], clean_out[1, :2])
    assert bool(w[1, 1, :33].isnan().any()) and not w[1, 1, 33:].any()
    # the selection ranks them last and goes on
    keep, _ = pool.evict_select(w, ctx, 10, sinks=1, recent=2)
    assert keep[1, 1].tolist()[0] == 0 and keep[1, 1].tolist()[-2:] == [31, 32]
    assert pool.device_error() == N.PA_OK
    pool.close()


def test_a_nan_key_in_a_row_of_many_ctas():
    """A row that many CTAs share ends as pa_decode's does: zeros out, NaN weights, and the
    other rows untouched."""
    pool = _pool("bf16", 2, 128, 900)
    pool.k_cache.view(torch.bfloat16).normal_()
    pool.v_cache.view(torch.bfloat16).normal_()
    t = torch.randperm(900, device="cuda")[:800].to(torch.int32).view(1, 800)
    ctx = torch.tensor([12800], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, 128, device="cuda").to(torch.bfloat16)
    clean, w0 = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(1, 2, 12800, device="cuda"))
    pool.layer_view("k").view(torch.bfloat16)[int(t[0, 333]), 1, 7] = math.nan
    out, w1 = pool.decode_weights(q, t, ctx, None, weights_out=torch.zeros(1, 2, 12800, device="cuda"))
    want = pool.decode(q, t, ctx)
    assert torch.equal(out[:, :8], clean[:, :8]) and torch.equal(w1[:, 0], w0[:, 0])
    assert bool((want[:, 8:] == 0).all()) and bool((out[:, 8:] == 0).all()) and bool(w1[:, 1].isnan().all())
    pool.close()


def test_two_graphs_share_a_workspace():
    """Nothing in the workspace outlives a call: two captured decodes with one workspace,
    replayed in turn, keep giving their own results."""
    pool = _pool("fp8_e4m3", 4, 128, 600)
    pool.k_cache.random_(0, 120)
    pool.v_cache.random_(0, 120)
    cases = []
    for S, n in ((3, 1500), (20, 130)):
        t = torch.randperm(600, device="cuda")[:S * -(-n // 16)].to(torch.int32).view(S, -1).contiguous()
        ctx = torch.randint(1, n + 1, (S,), device="cuda").to(torch.int32)
        q = torch.randn(S, 32, 128, device="cuda").to(torch.bfloat16)
        cases.append((q, t, ctx, torch.zeros(S, 4, n, device="cuda"), torch.empty_like(q)))
    ws = torch.empty(max(pool.weights_workspace_bytes(q.shape[0], 32, t.shape[1]) for q, t, *_ in cases),
                     dtype=torch.uint8, device="cuda")
    wants, graphs = [], []
    for q, t, ctx, w, out in cases:
        o, ww = pool.decode_weights(q, t, ctx, None, weights_out=w.clone())
        wants.append((o, ww))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pool.decode_weights(q, t, ctx, None, weights_out=w, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(5):
        for g, (q, t, ctx, w, out), (o, ww) in zip(graphs, cases, wants):
            w.zero_()
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(w, ww)
    pool.close()


@pytest.mark.parametrize("T", [1, 2, 9, 300])
def test_rope_any_number_of_tokens_and_heads(T):
    """One query head to many, one key head to many: each token's warps cover all of them."""
    from paged_kv_cache_270_gb300.pool import make_rope
    for kv, Hq, H, D in (("bf16", 1, 1, 64), ("fp16", 96, 12, 128), ("fp8_e4m3", 9, 9, 64), ("fp8_e4m3_block", 17, 17, 128)):
        pool = _pool(kv, H, D, 40)
        x = torch.randn(T, Hq + 2 * H, D, device="cuda").to(pool.in_dtype)
        slots, pos = torch.randperm(640, device="cuda")[:T], torch.randint(0, 1 << 30, (T,), device="cuda").to(torch.int32)
        if kv == "fp8_e4m3_block":  # runs of one call may not share a block
            slots = torch.arange(T, device="cuda")
        q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        rope = make_rope(D, "interleaved")
        out = pool.rope_and_cache(rope, q, k, v, pos, slots)
        # head by head through a pool of one head, whose rows must be the same bits
        one = _pool(kv, 1, D, 40)
        for h in range(H):
            hq = min(h, Hq - 1)
            got = one.rope_and_cache(rope, q[:, hq:hq + 1].contiguous(), k[:, h:h + 1].contiguous(), v[:, h:h + 1].contiguous(), pos, slots)
            assert torch.equal(got[:, 0], out[:, hq])
            for c in "kv":
                assert torch.equal(one.layer_view(c)[slots // 16, 0, slots % 16], pool.layer_view(c)[slots // 16, h, slots % 16])
        assert pool.device_error() == N.PA_OK
        pool.close()
        one.close()
