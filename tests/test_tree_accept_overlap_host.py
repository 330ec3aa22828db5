"""pa_tree_accept refuses lengths written into the block tables, which every warp reads (CPU, fake addresses)."""
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

FAKE_K, FAKE_V, A = 0x7F0000000000, 0x7F8000000000, 0x7E0000000000


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")
@pytest.mark.parametrize("kv", [N.PA_FP16, N.PA_FP8_E4M3_BLOCK])
def test_new_lens_inside_the_tables(kv):
    from paged_kv_cache_270_gb300 import build
    build.build()
    S, width, tables = 3, 5, A + (1 << 20)
    h = N.pa_pool_create(N.make_desc(2, 64, 2, 64, kv), FAKE_K, FAKE_V)
    try:
        for new in (tables, tables + 4 * S * width - 4, tables - 4 * S + 4, tables + 20):
            with pytest.raises(N.PAError) as e:
                N.pa_tree_accept(h, 0, 2, A, 4, A + 4096, A + 8192, tables, width, A + 12288, S, new, 0)
            assert e.value.code == N.PA_ERR_INVALID and "new_lens" in str(e.value), hex(new)
    finally:
        N.pa_pool_destroy(h)
