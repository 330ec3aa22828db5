"""Block tables so wide that pa_decode_weights could not count their tokens in 32 bits are
refused, before any CUDA call (fake addresses)."""
import pytest
import torch

N = pytest.importorskip("paged_kv_cache_270_gb300._native")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")

A = 1 << 44


@pytest.fixture(scope="module")
def pool():
    from paged_kv_cache_270_gb300 import build
    build.build()
    h = N.pa_pool_create(N.make_desc(1, 64, 1, 64, N.PA_FP16), 1 << 40, 1 << 41)
    yield h
    N.pa_pool_destroy(h)


@pytest.mark.parametrize("columns", [2 ** 27 - 255, 2 ** 27, 2 ** 28, 2 ** 31 - 1])
def test_too_wide(pool, columns):
    with pytest.raises(N.PAError) as e:
        N.pa_decode_weights(pool, 0, A, N.PA_FP16, A, A, columns, A, 1, 1, 0.125, A, A, 64, 1.0, A, 1 << 60, 0)
    assert e.value.code == N.PA_ERR_UNSUPPORTED
    with pytest.raises(N.PAError) as e:
        N.pa_decode_weights_workspace_bytes(pool, 1, 1, columns)
    assert e.value.code == N.PA_ERR_UNSUPPORTED


def test_the_widest(pool):
    """Not refused for its width: what fails here is the missing GPU."""
    for call in (lambda: N.pa_decode_weights_workspace_bytes(pool, 1, 1, 2 ** 27 - 256),
                 lambda: N.pa_decode_weights(pool, 0, A, N.PA_FP16, A, A, 2 ** 27 - 256, A, 1, 1, 0.125, A, A, 64, 1.0, A,
                                             1 << 60, 0)):
        with pytest.raises(N.PAError) as e:
            call()
        assert e.value.code == N.PA_ERR_CUDA
