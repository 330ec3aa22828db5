"""What pa_decode_weights refuses, before any CUDA call (fake addresses)."""
import math

import pytest
import torch

N = pytest.importorskip("paged_kv_cache_270_gb300._native")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")

FAKE_K, FAKE_V, A = 1 << 40, 1 << 41, 1 << 44
INV, UNS = N.PA_ERR_INVALID, N.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def pool():
    from paged_kv_cache_270_gb300 import build
    build.build()
    h = N.pa_pool_create(N.make_desc(2, 64, 2, 64, N.PA_FP16), FAKE_K, FAKE_V)
    yield h
    N.pa_pool_destroy(h)


def _call(pool, **kw):
    a = dict(layer=0, out=A, out_dtype=N.PA_FP16, q=A, tables=A, max_blocks=4, ctx=A, S=3, Hq=4, scale=0.125,
             w_in=A, w_out=A, stride=64, decay=1.0, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    N.pa_decode_weights(pool, *a.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(layer=2), INV), (dict(layer=-1), INV), (dict(Hq=3), INV), (dict(Hq=18), UNS), (dict(S=-1), INV),
    (dict(S=70000), UNS), (dict(max_blocks=0), INV), (dict(out_dtype=N.PA_BF16), INV), (dict(scale=math.nan), INV),
    (dict(decay=math.inf), INV), (dict(decay=math.nan), INV), (dict(stride=0), INV), (dict(stride=1 << 40), INV),
    (dict(out=0), INV), (dict(q=0), INV), (dict(q=A + 8), INV), (dict(tables=0), INV), (dict(ctx=0), INV),
    (dict(w_out=0), INV), (dict(w_out=A + 4), INV), (dict(w_in=A + 8), INV), (dict(ws=0), INV), (dict(ws=A + 8), INV)])
def test_refusals(pool, kw, code):
    with pytest.raises(N.PAError) as e:
        _call(pool, **kw)
    assert e.value.code == code


def test_no_sequences(pool):
    _call(pool, S=0, q=0, out=0, w_out=0, ws=0)


@pytest.mark.parametrize("ws", [torch.empty(1 << 20, dtype=torch.uint8, device="meta"),
                                torch.empty(1, dtype=torch.uint8).expand(1 << 20), b"bytes"])
def test_a_workspace_of_another_device_or_with_repeated_memory(ws):
    from paged_kv_cache_270_gb300.pool import KVPool
    p = KVPool(1, 8, 2, 64, "fp16", device="cpu")
    with pytest.raises((TypeError, ValueError), match="workspace"):
        p.decode_weights(torch.zeros(1, 4, 64, dtype=torch.float16), torch.zeros(1, 4, dtype=torch.int32),
                         torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64), workspace=ws)
    p.close()


def test_workspace_refusals(pool):
    for args, code in (((-1, 4, 4), INV), ((3, 5, 4), INV), ((3, 18, 4), UNS), ((3, 4, 0), INV)):
        with pytest.raises(N.PAError) as e:
            N.pa_decode_weights_workspace_bytes(pool, *args)
        assert e.value.code == code
