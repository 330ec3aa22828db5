"""Rows of pa_decode_weights without a finite score, and keys of infinite size, whether one
CTA holds the row whole or several share it."""
import math

import pytest
import torch

from test_gpu_weights_edges import _filled
from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("kv", ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"])
@pytest.mark.parametrize("n", [40, 12800])
def test_a_row_without_a_finite_score_ends_in_zeros(kv, n):
    """A NaN query leaves its row no score at all: its output is zeros, as pa_decode's is with the
    same schedule, the totals of its KV head are NaN, and no other row changes."""
    pool, t, c, _, _ = _filled(kv, 2, 128, [n], seed=3)
    q = torch.randn(1, 16, 128, device="cuda").to(pool.in_dtype)
    clean, w0 = pool.decode_weights(q, t, c, None, weights_out=torch.zeros(1, 2, n, device="cuda"))
    q[0, 3] = math.nan
    out, w1 = pool.decode_weights(q, t, c, None, weights_out=torch.zeros(1, 2, n, device="cuda"))
    plain = pool.decode(q, t, c, num_splits=N.PA_SPLITS_BALANCED)
    assert bool((plain[0, 3] == 0).all())
    assert bool((out[0, 3] == 0).all()), out[0, 3]
    others = [h for h in range(16) if h != 3]
    assert torch.equal(out[:, others], clean[:, others])
    assert bool(w1[0, 0].isnan().all()) and torch.equal(w1[0, 1], w0[0, 1])
    assert pool.device_error() == N.PA_OK
    pool.close()


@pytest.mark.parametrize("kv", ["fp16", "bf16"])
@pytest.mark.parametrize("G", [3, 5, 7])
@pytest.mark.parametrize("n", [40, 12800])
def test_a_key_of_infinite_size_in_an_odd_group(kv, G, n):
    """A key whose scores are all -inf weighs nothing: its total stays, and so does every
    other number finite, in a group of any size (an odd one keeps a place for one head more)."""
    pool, t, c, _, _ = _filled(kv, 2, 64, [n], seed=G)
    q = torch.randn(1, 2 * G, 64, device="cuda").abs().add(0.1).to(pool.in_dtype)
    at = n - 7
    pool.layer_view("k").view(pool.in_dtype)[int(t[0, at // 16]), 1, at % 16, 5] = -math.inf
    start = torch.rand(1, 2, n, device="cuda")
    out, w = pool.decode_weights(q, t, c, start, weights_out=torch.zeros_like(start), out_dtype=torch.float32)
    assert bool((w[0, 1, at] == start[0, 1, at])), w[0, 1, at]
    assert bool(w.isfinite().all()) and bool(out.isfinite().all())
    # the weights of a row add up to its heads: n additions and as many roundings as in the kernels' sum
    added = (w.double() - start.double()).sum(-1)
    assert float((added - G).abs().max()) <= G * (16 + n) * 2.0 ** -23 + n * 2.0 ** -24 * 2
    assert pool.device_error() == N.PA_OK
    pool.close()
