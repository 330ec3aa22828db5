"""Rows of pa_decode_weights without a finite score, whether one CTA holds the row whole or
several share it."""
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
