"""pa_decode_tree's waits do run out under a limit of 1 ns: the limit reaches the tree kernel, and what its roles do
then is run."""
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
    ("bf16", 8, 4, 128, [4000] * 32, 16), ("fp8_e4m3", 8, 8, 128, [8000] * 16, 32), ("fp8_e4m3_block", 8, 5, 64, [6000] * 16, 25)])
def test_waits_run_out(kv, H, G, D, ctx, size):
    b = Batch(kv, H, G, D, ctx, [size] * len(ctx), seed=2, mask="chain")
    want = b.run()
    torch.cuda.synchronize()
    assert b.pool.device_error() == N.PA_OK
    codes = []
    try:
        N.pa_set_pipeline_wait_limit_ns(1)
        for _ in range(40):
            b.run()
            codes.append(b.pool.device_error())
    finally:
        torch.cuda.synchronize()
        N.pa_set_pipeline_wait_limit_ns(0)
    assert set(codes) <= {N.PA_OK, N.PA_ERR_TIMEOUT}
    assert N.PA_ERR_TIMEOUT in codes
    assert torch.equal(b.run(), want)
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
