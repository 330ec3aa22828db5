"""The timeout path of pa_decode_tree: waits of 1 ns, of which some give up while others go on."""
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from tree_reference import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("kv, H, G, D, ctx, size", [
    ("bf16", 8, 4, 128, [2000] * 16, 16), ("fp8_e4m3", 8, 8, 128, [4000] * 8, 32), ("fp8_e4m3_block", 4, 5, 64, [900] * 30, 25),
    ("fp16", 2, 2, 64, [100] * 300, 7), ("fp8_e4m3", 1, 8, 128, [30000], 200)])
def test_waits_that_run_out_leave_the_next_call_right(kv, H, G, D, ctx, size):
    """Whatever each warp saw, the call ends, reports the timeout if there was one, and the next
    one gives the bits of the first."""
    b = Batch(kv, H, G, D, ctx, [size] * len(ctx), seed=1)
    want = b.run()
    torch.cuda.synchronize()
    assert b.pool.device_error() == N.PA_OK
    try:
        N.pa_set_pipeline_wait_limit_ns(1)
        for _ in range(40):
            b.run()
            assert b.pool.device_error() in (N.PA_OK, N.PA_ERR_TIMEOUT)
    finally:
        torch.cuda.synchronize()
        N.pa_set_pipeline_wait_limit_ns(0)
    assert torch.equal(b.run(), want)
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
