"""The timeout path of pa_decode_weights on the builds and schedules that another test's batch
does not run: units that one CTA streams whole, 16-bit and block-scaled pools, odd groups."""
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


@pytest.mark.parametrize("kv, G, H, D, S, n", [
    ("bf16", 4, 8, 128, 256, 1024), ("fp16", 3, 4, 64, 600, 700), ("fp8_e4m3_block", 8, 8, 128, 64, 2048),
    ("fp8_e4m3", 7, 2, 128, 300, 500), ("bf16", 1, 8, 64, 4, 20000)])
def test_waits_that_run_out_leave_the_next_call_right(kv, G, H, D, S, n):
    """With waits of 1 ns some give up while others go on. Whatever each warp saw, the call
    ends, reports the timeout if there was one, and the next one gives the bits of the first."""
    pool, t, c, _, _ = _filled(kv, H, D, [n] * S, seed=1)
    q = torch.randn(S, H * G, D, device="cuda").to(pool.in_dtype)
    start = torch.zeros(S, H, n, device="cuda")
    want, first = pool.decode_weights(q, t, c, None, weights_out=start.clone())
    torch.cuda.synchronize()
    assert pool.device_error() == N.PA_OK
    try:
        N.pa_set_pipeline_wait_limit_ns(1)
        for _ in range(40):
            pool.decode_weights(q, t, c, None, weights_out=start)
            assert pool.device_error() in (N.PA_OK, N.PA_ERR_TIMEOUT)
    finally:
        torch.cuda.synchronize()
        N.pa_set_pipeline_wait_limit_ns(0)
    out, again = pool.decode_weights(q, t, c, None, weights_out=start)
    assert pool.device_error() == N.PA_OK
    assert torch.equal(out, want) and torch.equal(again, first)
    pool.close()
