"""pa_evict_select with the largest budget it takes, 2^31 - 1025: the rows that keep all their
tokens are filled to their end and no further."""
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("tokens", [100, 20000, 40000, 70000])  # one, two, four and eight CTAs for the row
def test_the_largest_budget(tokens):
    from paged_kv_cache_270_gb300.pool import KVPool
    budget, guard = 2 ** 31 - 1025, 1 << 16
    pool = KVPool(1, 4, 1, 64, "bf16")
    whole = torch.full((guard + budget + guard,), -77, dtype=torch.int32, device="cuda")  # 8.6 GB
    keep = whole[guard:guard + budget].view(1, 1, budget)
    n = tokens - 3
    w = torch.rand(1, 1, tokens, device="cuda")
    got, kept = pool.evict_select(w, torch.tensor([n], dtype=torch.int32, device="cuda"), budget, sinks=5, recent=9, keep=keep)
    assert pool.device_error() == N.PA_OK and kept.tolist() == [n]
    assert torch.equal(keep[0, 0, :n], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert int(keep[0, 0, n:].max()) == -1 and int(keep[0, 0, n:].min()) == -1
    assert bool((whole[:guard] == -77).all()) and bool((whole[guard + budget:] == -77).all())
    pool.close()
    del whole, keep, got
    torch.cuda.empty_cache()
