"""Edges of pa_decode_weights: the precision of its 16-bit outputs."""
import math

import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu

DTYPES = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _filled(kv, H, D, ctx, seed=0):
    """A pool of random values, tables of random pages, and what they hold in 64 bits:
    (pool, tables, ctx, k, v) with k, v [S, H, tokens, D]."""
    from paged_kv_cache_270_gb300.pool import KVPool
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, pages = len(ctx), max(1, -(-max(ctx) // 16))
    pool = KVPool(1, S * pages + 3, H, D, kv, 0.02, 0.03)
    held = []
    for which, scale in (("k", 0.02), ("v", 0.03)):
        x = torch.randn(pool.num_blocks, H, 16, D, device="cuda", generator=g)
        if pool.elem_bytes == 2:
            x = x.to(pool.in_dtype)
            held.append(x.double())
        else:
            x = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            s = torch.full((pool.num_blocks, H), scale, device="cuda")
            if pool.block_scaled:
                s = torch.rand(pool.num_blocks, H, device="cuda", generator=g) * 0.03 + 0.005
                pool.scale_view(which).copy_(s)
            held.append(x.double() * s.double()[:, :, None, None])
        pool.layer_view(which).copy_(x.view(torch.uint8))
    t = torch.randperm(pool.num_blocks, device="cuda", generator=g)[:S * pages].to(torch.int32).view(S, pages).contiguous()
    k, v = (x[t.long()].permute(0, 2, 1, 3, 4).reshape(S, H, pages * 16, D) for x in held)
    return pool, t, torch.tensor(ctx, dtype=torch.int32, device="cuda"), k, v


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("G, H, D, ctx", [(4, 2, 64, [5, 17, 2, 33]), (8, 4, 128, [3, 40, 16, 1, 9]), (3, 1, 128, [25, 6]),
                                          (8, 1, 128, [420])])
def test_a_16_bit_output_is_rounded_once(kv, G, H, D, ctx):
    """The probabilities keep their precision up to the product with V, whatever the pool's
    type, so that a 16-bit output is an fp32 result rounded once.

    Bound.  A score is off by at most d = (D + 8) 2^-23 |q| |k| scale log2(e) (D truncated
    additions and a few roundings, by Cauchy-Schwarz); a weight then by 2 d ln 2, by 2^-22 of
    ex2 and the n additions of its sum.  A weight is held as two numbers of the pool's product type: the
    second one's rounding leaves 2^-22 (binary16; below its normal range 2^-25, against a largest weight of
    one) or 2^-17 (bfloat16).  The n products are added in fp32, 2^-23 each, the sum rescaled
    once a page, 2^-22.  Small scores (q of 0.05) keep d from hiding a rounding of the weights."""
    S = len(ctx)
    pool, t, c, k, v = _filled(kv, H, D, ctx, seed=G)
    g = torch.Generator(device="cuda").manual_seed(9)
    q = (torch.randn(S, H * G, D, device="cuda", generator=g) * 0.05).to(pool.in_dtype)
    scale = 1 / math.sqrt(D)
    tokens = k.shape[2]
    out, _ = pool.decode_weights(q, t, c, None, weights_out=torch.zeros(S, H, tokens, device="cuda"))
    there = torch.arange(tokens, device="cuda") < c.view(S, 1, 1)
    qd = q.double().view(S, H, G, D)
    p = (qd @ k.transpose(2, 3) * scale).masked_fill(~there.unsqueeze(2), -math.inf).softmax(-1)
    v = v.masked_fill(~there.unsqueeze(3), 0)
    ref, size = p @ v, p @ v.abs()
    n = c.double().view(S, 1, 1, 1)
    d = (D + 8) * 2.0 ** -23 * qd.norm(dim=-1, keepdim=True) * k.norm(dim=-1).masked_fill(~there, 0).amax(-1).view(S, H, 1, 1) * scale * math.log2(math.e)
    split = 2.0 ** -17 if kv == "bf16" else 2.0 ** -22
    err = size * (2 * math.log(2) * d + split + (32 + 4 * n) * 2.0 ** -23) + v.abs().sum(2, keepdim=True) * 2.0 ** -25
    eps = torch.finfo(out.dtype).eps / 2
    tol = err + eps * (ref.abs() + err) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
    off = (out.double().view_as(ref) - ref).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    assert pool.device_error() == N.PA_OK
    pool.close()
