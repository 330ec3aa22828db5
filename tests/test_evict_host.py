"""What pa_evict_select and pa_evict_compact refuse, before any CUDA call."""
import pytest
import torch

N = pytest.importorskip("paged_kv_cache_270_gb300._native")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")

FAKE_K, FAKE_V, A, B = 1 << 40, 1 << 41, 1 << 44, 1 << 45
INV, UNS = N.PA_ERR_INVALID, N.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def pool():
    from paged_kv_cache_270_gb300 import build
    build.build()
    h = N.pa_pool_create(N.make_desc(2, 64, 2, 64, N.PA_FP16), FAKE_K, FAKE_V)
    yield h
    N.pa_pool_destroy(h)


def _select(pool, **kw):
    a = dict(w=A, stride=64, ctx=A, S=3, H=2, budget=32, sinks=4, recent=8, keep=A, kept=A)
    a.update(kw)
    N.pa_evict_select(pool, *a.values(), 0)


def _compact(pool, **kw):
    a = dict(layer=0, keep=A, H=2, budget=32, kept=A, src=A, src_n=8, dst=B, dst_n=2, S=3, w_in=A, in_n=128,
             w_out=B, out_n=128)
    a.update(kw)
    N.pa_evict_compact(pool, *a.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(S=-1), INV), (dict(H=0), INV), (dict(budget=0), INV), (dict(sinks=-1), INV), (dict(recent=-1), INV),
    (dict(sinks=30), INV), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INV), (dict(stride=0), INV),
    (dict(stride=1 << 31), INV), (dict(budget=2 ** 31 - 1), INV), (dict(S=1 << 20, H=1 << 10), UNS), (dict(w=0), INV),
    (dict(ctx=0), INV), (dict(keep=0), INV), (dict(kept=0), INV), (dict(w=A + 4), INV)])
def test_select_refusals(pool, kw, code):
    with pytest.raises(N.PAError) as e:
        _select(pool, **kw)
    assert e.value.code == code


@pytest.mark.parametrize("kw, code", [
    (dict(layer=2), INV), (dict(layer=-1), INV), (dict(H=3), INV), (dict(H=0), INV), (dict(S=-1), INV),
    (dict(budget=0), INV), (dict(budget=2 ** 31 - 1), INV), (dict(src_n=0), INV), (dict(dst_n=0), INV), (dict(w_in=0), INV),
    (dict(w_out=0), INV), (dict(w_out=A), INV), (dict(in_n=0), INV), (dict(out_n=0), INV), (dict(out_n=1 << 31), INV),
    (dict(keep=0), INV), (dict(kept=0), INV), (dict(src=0), INV), (dict(dst=0), INV), (dict(dst=A), INV),
    (dict(w_in=A + 8), INV), (dict(w_out=B + 4), INV),
    (dict(S=2 ** 31 - 1, budget=2 ** 30, dst_n=2 ** 30), UNS)])
def test_compact_refusals(pool, kw, code):
    with pytest.raises(N.PAError) as e:
        _compact(pool, **kw)
    assert e.value.code == code


def test_no_sequences(pool):
    _select(pool, S=0, w=0, keep=0)
    _compact(pool, S=0, keep=0, src=0)


def test_null_pool():
    with pytest.raises(N.PAError):
        _select(0)
    with pytest.raises(N.PAError):
        _compact(0)
