"""pa_decode_tree with queries at the low end of bfloat16's range: rows of zeros but for one element, rows of
subnormals, and small ones that meet large keys (tolerances: tree_reference)."""
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


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp8_e4m3_block"])
def test_small_queries(kv, D, out_dtype):
    """A row whose largest element is 2^-112 to 2^-133: nearly every key has the same weight."""
    b = Batch(kv, 2, 4, D, [300, 40, 5000], [9, 20, 4], seed=21)
    b.q[0] = 0.0
    b.q[0, 1, 5] = 2.0 ** -125
    b.q[1, 0] = 0.0
    b.q[1, 0, D - 1] = -2.0 ** -133  # the smallest bfloat16
    for i, e in enumerate(range(112, 130)):
        b.q[2 + i, 3] = (b.q[2 + i, 3].double() * 2.0 ** -e).bfloat16()
    b.q[30, :] = (b.q[30].double() * 2.0 ** -129).bfloat16()
    out = b.run(out_dtype=out_dtype)
    assert b.pool.device_error() == N.PA_OK
    b.check(out)
    b.pool.close()


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_small_queries_of_large_keys(out_dtype):
    """Elements near 2^-120 and tiles whose keys lie near 2^120: scores of ordinary size, whose factor
    (of the row's power of two and the softmax scale) is no normal number by itself."""
    b = Batch("fp8_e4m3_block", 2, 4, 128, [300, 40, 5000], [9, 20, 4], seed=22)
    b.q.copy_((b.q.double() * 2.0 ** -120).bfloat16())
    b.pool.scale_view("k").mul_(2.0 ** 120)
    out = b.run(out_dtype=out_dtype)
    assert b.pool.device_error() == N.PA_OK
    b.check(out)
    b.pool.close()
