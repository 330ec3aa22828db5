"""pa_decode_weights against the fp64 oracle: the outputs within pa_decode's
tolerances, the totals within a bound on fp32 arithmetic.

Bound on a weight p = 2^(x - M) / L of a row of n tokens.  The products of q
and k are exact in fp32; adding D of them, each step at worst truncated, leaves
the score off by at most D 2^-23 |q| |k| scale log2(e) = d (Cauchy-Schwarz on
the absolute values; |k| of FP8 rows is within 1 + 2^-4 of the bfloat16 row's).
An error d in every score moves p by at most 2 d ln 2, relative (numerator and
denominator).  ex2.approx is off by 2^-22, a handful of other roundings by
2^-24 each, L's n additions by n 2^-24: together below (16 + n) 2^-23.  The total
adds at most 8 such weights and decay * w_in, one rounding each."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_harness import bits_to_torch, check_fp32, check_half, fill_both, new_pool, oracle_pools, vmax_of
from paged_kv_cache_270_gb300 import _native as N
from paged_kv_cache_270_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DTYPES = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    oracle.build()


def _workload(kv, G, Hkv, D, ctx, seed, extra=0):
    rng = np.random.default_rng([seed, 41])
    ctx = np.array(ctx, np.int32)
    pages = -(-ctx // 16)
    nb = int(pages.sum()) + 3
    width = max(int(pages.max()), 1) + extra
    perm = rng.permutation(nb).astype(np.int32)
    tables = rng.integers(-7, 10 ** 6, (len(ctx), width)).astype(np.int32)  # behind the pages: never read
    at = 0
    for s, k in enumerate(pages):
        tables[s, :k] = perm[at:at + k]
        at += k
    w = W.Workload(name=f"weights{seed}", index=70 + seed, kv_dtype=kv, n_q_heads=Hkv * G, n_kv_heads=Hkv,
                   head_dim=D, ctx_lens=ctx, num_blocks=nb, block_tables=tables, kv_seed=seed)
    if int(ctx.max()) > 0:
        w.compute_fp8_scales()
    return w


def _bound(w, p, q_bits, w_in, decay):
    """The totals in fp64 and how far off fp32 may be, [S][Hkv][tokens]."""
    S, G, D = w.S, w.n_q_heads // w.n_kv_heads, w.head_dim
    q = W.bits_to_f32(q_bits, w.in_dtype).astype(np.float64)
    want = np.where(np.arange(w_in.shape[2]) < w.ctx_lens[:, None, None], decay * w_in, w_in)
    tol = np.abs(want) * 2.0 ** -23
    for s in range(S):
        n = int(w.ctx_lens[s])
        if n == 0:
            continue
        k = W.bits_to_f32(w.kv_bits(s, 0, n)[0], w.in_dtype).astype(np.float64)
        k = np.sqrt((k * k).sum(-1).max(0)) * (1 + 2.0 ** -4)  # [Hkv], the longest row
        d = D * 2.0 ** -23 * np.sqrt((q[s] ** 2).sum(-1)) * np.repeat(k, G) * abs(w.softmax_scale) * math.log2(math.e)
        each = p[s, :, :n]
        err = each * (2 * math.log(2) * d[:, None] + (16 + n) * 2.0 ** -23) + 2.0 ** -126
        want[s, :, :n] += each.reshape(-1, G, n).sum(1)
        tol[s, :, :n] += err.reshape(-1, G, n).sum(1) + 8 * 2.0 ** -24 * np.abs(want[s, :, :n])
    return want, tol


def _run(w, pool, q_bits, w_in, decay=1.0, out_dtype=None, in_place=False, stride=None):
    q = bits_to_torch(q_bits, w.in_dtype)
    t, c = torch.from_numpy(w.block_tables).cuda(), torch.from_numpy(w.ctx_lens).cuda()
    win = torch.from_numpy(w_in.astype(np.float32)).cuda()
    out, wout = pool.decode_weights(q, t, c, win, weights_out=None if in_place else win.clone(), decay=decay,
                                    out_dtype=out_dtype, softmax_scale=w.softmax_scale)
    torch.cuda.synchronize()
    assert (wout.data_ptr() == win.data_ptr()) == in_place
    return out, wout


def _check(w, decay=1.0, in_place=False, stride_extra=0, seed=0):
    pool = new_pool(w, 0xFF)  # NaN in every slot that no token was written to
    ops = oracle_pools(w, 0xFF)
    fill_both(w, pool, ops)
    q = w.q_bits()
    rng = np.random.default_rng(seed)
    tokens = max(int(w.ctx_lens.max()), 1) + stride_extra
    w_in = (rng.random((w.S, w.n_kv_heads, tokens)) * 3).astype(np.float32).astype(np.float64)
    ref, p = oracle.paged_attention(w.kv_dtype, w.in_dtype, w.num_blocks, 16, w.n_kv_heads, w.head_dim, *ops,
                                    w.k_scale, w.v_scale, q, w.block_tables, w.ctx_lens, w.softmax_scale,
                                    want_probs=True)
    want, tol = _bound(w, p, q, w_in, float(np.float32(decay)))
    for out_dtype in (None, torch.float32):
        out, got = _run(w, pool, q, w_in, decay, out_dtype, in_place)
        assert pool.device_error() == N.PA_OK
        if out_dtype or not w.ctx_lens.any():  # (no value, no largest one: the rows are zero)
            check_fp32(out.float(), ref)
        else:
            check_half(out, ref, vmax_of(w, ops))
        got = got.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))
        behind = np.arange(tokens) >= w.ctx_lens[:, None, None]
        assert np.array_equal(np.where(behind, got, 0), np.where(behind, w_in, 0))  # left as they were
    pool.close()


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("G, Hkv, D, ctx, extra", [
    (2, 2, 64, [17, 33, 64, 100], 0), (8, 2, 128, [1, 0, 16, 15, 700, 0, 31], 2), (1, 3, 128, [0, 257, 5], 0),
    (3, 1, 64, [129, 1], 1), (4, 8, 128, [1000, 3, 420], 0), (7, 2, 128, [48], 5), (5, 1, 128, [333, 32, 1], 0)])
def test_against_oracle(kv, G, Hkv, D, ctx, extra):
    _check(_workload(kv, G, Hkv, D, ctx, seed=len(ctx) + G, extra=extra), stride_extra=3 * extra)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "bf16"])
def test_long_rows_span_many_ctas(kv):
    """One sequence over every CTA (hundreds of pieces), and long next to short ones."""
    _check(_workload(kv, 8, 1, 128, [21001], seed=1))
    _check(_workload(kv, 2, 2, 64, [9000, 1, 40, 0, 5000], seed=2))


@pytest.mark.parametrize("decay", [0.0, 0.5, -1.0])
def test_decay_in_place(decay):
    _check(_workload("bf16", 4, 2, 128, [100, 33], seed=3), decay=decay, in_place=True)


def test_no_sequence_has_context():
    w = _workload("fp16", 2, 2, 64, [0, 0, 0], seed=4)
    _check(w, stride_extra=9)


def test_totals_from_nothing_add_up():
    """With no totals before, a row's weights sum to the heads of its group; a second
    call doubles them."""
    w = _workload("fp8_e4m3", 4, 2, 128, [3000, 17, 512], seed=5)
    pool = new_pool(w, 0xFF)
    fill_both(w, pool, None)
    q = bits_to_torch(w.q_bits(), "bf16")
    t, c = torch.from_numpy(w.block_tables).cuda(), torch.from_numpy(w.ctx_lens).cuda()
    tot = torch.full((3, 2, 3000), 7.0, device="cuda")
    pool.decode_weights(q, t, c, None, weights_out=tot)
    there = torch.arange(3000, device="cuda") < c.view(3, 1, 1)
    assert bool((tot[~there.expand_as(tot)] == 7.0).all())
    sums = tot.double().masked_fill(~there, 0).sum(-1)
    assert float((sums - 4).abs().max()) <= 4 * (16 + 3000) * 2.0 ** -23
    once = tot.clone()
    pool.decode_weights(q, t, c, tot)
    assert torch.allclose(tot.masked_fill(~there, 0), 2 * once.masked_fill(~there, 0), rtol=2.0 ** -22, atol=0)
    pool.close()


def test_more_sequences_than_one_schedule():
    """4099 sequences: two schedules, each with its own contexts."""
    S = 4099
    ctx = [(s * 7) % 23 for s in range(S)]
    w = _workload("fp16", 2, 1, 64, ctx, seed=6)
    _check(w)


def test_repeats_bit_for_bit_and_in_a_graph():
    w = _workload("fp8_e4m3_block", 8, 4, 128, [4000, 100, 0, 2500], seed=7)
    pool = new_pool(w, 0xFF)
    fill_both(w, pool, None)
    q = bits_to_torch(w.q_bits(), "bf16")
    t, c = torch.from_numpy(w.block_tables).cuda(), torch.from_numpy(w.ctx_lens).cuda()
    tot = torch.rand(4, 4, 4000, device="cuda")
    ws = torch.empty(pool.weights_workspace_bytes(4, 32, t.shape[1]), dtype=torch.uint8, device="cuda")
    out, first = pool.decode_weights(q, t, c, tot, weights_out=torch.zeros_like(tot), workspace=ws)
    for junk in (0x00, 0xFF):  # nothing of the workspace is read before it is written
        ws.fill_(junk)
        o, again = pool.decode_weights(q, t, c, tot, weights_out=torch.zeros_like(tot), workspace=ws)
        assert torch.equal(o, out) and torch.equal(again, first)
    gout, gw = torch.empty_like(out), torch.zeros_like(tot)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.decode_weights(q, t, c, tot, weights_out=gw, out=gout, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, out) and torch.equal(gw, first)
    # shorter contexts, replayed: rows behind them stay
    c -= 60
    c.clamp_(min=0)
    gw.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    behind = torch.arange(4000, device="cuda") >= c.view(4, 1, 1)
    assert bool((gw[behind.expand_as(gw)] == 5.0).all())
    o, short = pool.decode_weights(q, t, c, tot, weights_out=torch.full_like(tot, 5.0))
    assert torch.equal(gw, short) and torch.equal(gout, o)
    assert pool.device_error() == N.PA_OK
    pool.close()


def test_bad_lengths_are_reported():
    """A context longer than its table, or than the totals' rows, sets PA_ERR_BOUNDS; what
    lies outside both stays untouched."""
    w = _workload("bf16", 2, 2, 64, [64, 40], seed=8)
    pool = new_pool(w, 0)
    fill_both(w, pool, None)
    q = bits_to_torch(w.q_bits(), "bf16")
    t = torch.from_numpy(w.block_tables).cuda()
    c = torch.tensor([64, 40], dtype=torch.int32, device="cuda")
    buf = torch.full((2, 2, 50), 9.0, device="cuda")
    pool.decode_weights(q, t, c, None, weights_out=buf)  # rows of 50 for 64 tokens
    assert pool.device_error() == N.PA_ERR_BOUNDS
    assert bool((buf[0] != 9.0).all()) and bool((buf[1, :, 40:] == 9.0).all())
    full = torch.full((2, 2, 64), 9.0, device="cuda")
    pool.decode_weights(q, t, c, None, weights_out=full)
    assert pool.device_error() == N.PA_OK
    assert torch.equal(full[:, :, :50][0], buf[0])
    c[0] = 65
    pool.decode_weights(q, t, c, None, weights_out=full)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    t[1, 0] = w.num_blocks
    c[0] = 64
    pool.decode_weights(q, t, c, None, weights_out=full)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    with pytest.raises(N.PAError) as e:
        pool.decode_weights(q, t, c, None, weights_out=full,
                            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == N.PA_ERR_INVALID
    for bad in (full.half(), full[:1], full.transpose(1, 2), full[:, 0]):
        with pytest.raises((TypeError, ValueError)):
            pool.decode_weights(q, t, c, bad)
    pool.close()


def test_timeout_leaves_the_context_usable():
    """Waits that run out are reported; the next call is right.  A wait outlasts the
    hardware's own brief first test only now and then, so the GPU is kept busy (256
    sequences of 4096 tokens) and the call repeated until one does."""
    from paged_kv_cache_270_gb300.pool import KVPool
    S, n = 256, 4096
    pool = KVPool(1, S * n // 16, 8, 128, "fp8_e4m3", 0.01, 0.01)
    pool.k_cache.random_(0, 120)
    pool.v_cache.random_(0, 120)
    q = torch.randn(S, 64, 128, device="cuda").to(torch.bfloat16)
    t = torch.randperm(S * n // 16, device="cuda").to(torch.int32).view(S, -1)
    c = torch.full((S,), n, dtype=torch.int32, device="cuda")
    tot = torch.zeros(S, 8, n, device="cuda")
    want, first = pool.decode_weights(q, t, c, None, weights_out=tot.clone())
    torch.cuda.synchronize()
    assert pool.device_error() == N.PA_OK
    seen = []
    try:
        N.pa_set_pipeline_wait_limit_ns(1)
        while len(seen) < 200 and N.PA_ERR_TIMEOUT not in seen:
            pool.decode_weights(q, t, c, None, weights_out=tot)
            seen.append(pool.device_error())
    finally:
        torch.cuda.synchronize()
        N.pa_set_pipeline_wait_limit_ns(0)
    assert set(seen) <= {N.PA_OK, N.PA_ERR_TIMEOUT} and seen[-1] == N.PA_ERR_TIMEOUT
    out, again = pool.decode_weights(q, t, c, None, weights_out=tot)
    assert pool.device_error() == N.PA_OK
    assert torch.equal(out, want) and torch.equal(again, first)
    pool.close()
