"""pa_decode_tree where a history is split over the GPU: an infinity or a NaN that a node sees reaches its result
from a piece of next to no weight as well."""
import math

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


def _batch(kv):
    """30000 tokens of one kv head, cut into pieces; page 3 (in the first piece) has nearly all of the weight."""
    b = Batch(kv, 1, 1, 128, [30000], [3], mask="chain", seed=31)
    blk = int(b.tables_np[0, 3])
    k = (8.0 * b.q[:1].view(1, 1, 128)).expand(16, 1, 128).contiguous()  # scores near 200 for row 0
    b.q[1:] = b.q[0]
    b.pool.reshape_and_cache(k, torch.ones_like(k), torch.arange(16, device="cuda") + 16 * blk)
    return b


@pytest.mark.parametrize("kv", ["fp16", "bf16"])
def test_infinite_value_of_little_weight(kv):
    """Node 1's value is infinite in one dimension: rows 1 and 2, which see it, are infinite there and
    nowhere else; row 0 keeps its bits."""
    b = _batch(kv)
    want = b.run()
    assert bool((want - 1.0).abs().max() < 0.01)
    t = b.ctx[0] - 2
    b.pool.layer_view("v")[int(b.tables_np[0, t // 16]), 0, t % 16].view(b.pool.in_dtype)[70] = -math.inf
    out = b.run()
    assert torch.equal(out[0], want[0])
    assert bool((out[1:, 0, 70] == -math.inf).all())
    rest = torch.arange(128, device="cuda") != 70
    assert torch.equal(out[1:, :, rest], want[1:, :, rest])
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp8_e4m3_block"])
def test_page_of_nan_of_little_weight(kv):
    """A page of the history whose values are NaN."""
    b = _batch(kv)
    blk = int(b.tables_np[0, 1500])
    if b.pool.block_scaled:
        b.pool.scale_view("v")[blk] = math.nan
    else:
        b.pool.layer_view("v")[blk] = 0x7F if b.pool.elem_bytes == 1 else 0xFF
    assert b.run().isnan().all()
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
