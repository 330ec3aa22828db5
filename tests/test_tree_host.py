"""What the entry points of speculative decoding and of the normalised rotary write refuse
before any CUDA call (so with fake addresses), and the axes' order (CPU)."""
import math

import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

FAKE_K, FAKE_V, A = 0x7F0000000000, 0x7F8000000000, 0x7E0000000000
INV, UNS = N.PA_ERR_INVALID, N.PA_ERR_UNSUPPORTED
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_270_gb300 import build
    build.build()
    return N.lib()


def _pool(**kw):
    a = dict(layers=2, blocks=64, heads=2, dim=64, kv=N.PA_FP16)
    a.update(kw)
    return N.pa_pool_create(N.make_desc(a["layers"], a["blocks"], a["heads"], a["dim"], a["kv"]), FAKE_K, FAKE_V)


def _refused(call, cases):
    for kw, code in cases:
        with pytest.raises(N.PAError) as e:
            call(**kw)
        assert e.value.code == code, kw


def test_axes(lib):
    from paged_kv_cache_270_gb300.pool import make_rope_axes
    a = make_rope_axes([3, 2, 1])
    assert a.n_axes == 3 and list(a.axis[:6]) == [0, 0, 0, 1, 1, 2] and not any(a.axis[6:])
    a = make_rope_axes([4, 3, 2], "turns")
    assert list(a.axis[:9]) == [0, 1, 2, 0, 1, 2, 0, 1, 0]
    a = make_rope_axes([24, 20, 20], "turns")  # axis 0 keeps the pairs behind the others' last
    assert [list(a.axis).count(i) for i in range(3)] == [24, 20, 20] and list(a.axis[60:]) == [0] * 4
    for bad in ([], [0], [65], [1] * 5, [3, -1], [40, 30]):
        with pytest.raises(ValueError):
            make_rope_axes(bad)
    for bad in ([1, 5, 1], [0, 2, 2]):
        with pytest.raises(ValueError):
            make_rope_axes(bad, "turns")
    with pytest.raises(ValueError):
        make_rope_axes([1], "rows")


@no_gpu
def test_norm_rope_refusals(lib):
    h = _pool()
    rope = N.pa_rope_init(N.pa_rope_desc(0, 64, 0, 1e4, 1.0, 8192.0, 1.0, 4.0, 1.0))

    def call(**kw):
        a = dict(layer=0, rope=rope, axes=None, qw=A, kw=A, per_head=0, eps=1e-6, offset=0.0, q=A, qs=256, q_out=A, Hq=4,
                 k=A, ks=128, v=A, vs=128, pos=A, slots=A, T=3)
        a.update(kw)
        N.pa_norm_rope_and_cache(h, *a.values(), 0)

    def axes(n, *of):
        x = N.pa_rope_axes(n)
        for i, v in enumerate(of):
            x.axis[i] = v
        return x

    try:
        call(T=0)
        call(T=0, qw=0, kw=0, axes=axes(4, 0, 1, 2, 3), eps=0.0)
        _refused(call, [(dict(eps=-1e-9), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
                        (dict(offset=math.nan), INV), (dict(offset=-math.inf), INV), (dict(per_head=2), INV),
                        (dict(per_head=-1), INV), (dict(qw=A + 8), INV), (dict(kw=A + 2), INV), (dict(axes=axes(0)), INV),
                        (dict(axes=axes(5)), INV), (dict(axes=axes(-1)), INV), (dict(axes=axes(2, 0, 1, 2)), INV),
                        (dict(axes=axes(1, 1)), INV), (dict(rope=None), INV), (dict(layer=2), INV), (dict(T=-1), INV),
                        (dict(Hq=0), INV), (dict(qs=248), INV), (dict(q=0), INV), (dict(q_out=A + 4), INV),
                        (dict(pos=0), INV), (dict(slots=0), INV), (dict(qs=264), INV), (dict(Hq=1 << 20, qs=1 << 27), UNS)])
    finally:
        N.pa_pool_destroy(h)


@no_gpu
def test_decode_tree_refusals(lib):
    h = _pool()

    def call(**kw):
        a = dict(layer=0, out=A + 8192, dt=N.PA_FP16, q=A, T=9, qs=A, tables=A, width=4, ctx=A, S=3, Hq=4, nodes=8, mask=A,
                 scale=0.1, ws=A, ws_bytes=1 << 40)
        a.update(kw)
        N.pa_decode_tree(h, *a.values(), 0)

    try:
        call(S=0)
        call(T=0)
        call(S=0, out=0, q=0, ws=0)
        _refused(call, [(dict(layer=2), INV), (dict(layer=-1), INV), (dict(dt=N.PA_BF16), INV), (dict(dt=N.PA_FP8_E4M3), INV),
                        (dict(T=-1), INV), (dict(S=-1), INV), (dict(S=65536), UNS), (dict(Hq=3), INV), (dict(Hq=0), INV),
                        (dict(Hq=18), UNS), (dict(nodes=0), INV), (dict(nodes=257), INV), (dict(nodes=-1), INV),
                        (dict(width=0), INV), (dict(width=1 << 27), UNS), (dict(scale=math.nan), INV),
                        (dict(scale=math.inf), INV), (dict(out=0), INV), (dict(q=0), INV), (dict(qs=0), INV),
                        (dict(tables=0), INV), (dict(ctx=0), INV), (dict(out=A + 8), INV), (dict(q=A + 2), INV),
                        (dict(mask=A + 4), INV), (dict(ws=0), INV), (dict(ws=A + 8), INV), (dict(out=A), INV),
                        (dict(out=A + 9 * 512 - 16), INV), (dict(q=A + 8192 + 9 * 512 - 16), INV),
                        (dict(dt=N.PA_FP32, q=A + 8192 + 9 * 1024 - 16), INV)])
        for bad in (dict(Hq=3), dict(nodes=0), dict(nodes=257)):
            a = dict(Hq=4, nodes=8)
            a.update(bad)
            with pytest.raises(N.PAError):
                N.pa_decode_tree_workspace_bytes(h, *a.values())
    finally:
        N.pa_pool_destroy(h)


@no_gpu
def test_tree_accept_refusals(lib):
    h = _pool()

    def call(**kw):
        a = dict(layer=0, n=2, paths=A, P=5, lens=A, qs=A, tables=A, width=4, ctx=A, S=3, new=A + 4096)
        a.update(kw)
        N.pa_tree_accept(h, *a.values(), 0)

    try:
        call(S=0)
        _refused(call, [(dict(layer=2), INV), (dict(layer=1), INV), (dict(n=0), INV), (dict(n=3), INV), (dict(n=-1), INV),
                        (dict(P=-1), INV), (dict(P=257), INV), (dict(S=-1), INV), (dict(width=0), INV),
                        (dict(width=1 << 27), UNS), (dict(paths=0), INV), (dict(lens=0), INV), (dict(qs=0), INV),
                        (dict(tables=0), INV), (dict(ctx=0), INV), (dict(new=0), INV), (dict(new=A), INV),
                        (dict(ctx=A + 4096 - 8), INV), (dict(ctx=A + 4096 + 8), INV), (dict(lens=A + 4096), INV),
                        (dict(qs=A + 4096 - 12), INV), (dict(paths=A + 4096 - 56), INV),
                        (dict(S=0x7FFFFFFF, n=2), UNS)])
    finally:
        N.pa_pool_destroy(h)
