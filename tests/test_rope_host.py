"""Rotary embeddings on the host: the speeds that pa_rope_init makes, and what
it and pa_rope_and_cache refuse (before any CUDA call, so with fake addresses)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

N = pytest.importorskip("paged_kv_cache_270_gb300._native")

FAKE_K, FAKE_V, A = 1 << 40, 1 << 41, 1 << 44
INV, UNS = N.PA_ERR_INVALID, N.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_270_gb300 import build
    build.build()
    return N.lib()


def _desc(**kw):
    a = dict(layout=N.PA_ROPE_HALF, rot_dim=64, scaling=N.PA_ROPE_SCALE_NONE, theta=10000.0, factor=8.0,
             original_len=4096.0, low=1.0, high=4.0, gain=1.0)
    a.update(kw)
    return N.pa_rope_desc(*a.values())


def _speeds(d):
    """The formulas of the header, pair by pair, in radians per position."""
    R, out = d.rot_dim, []
    base = d.theta
    if d.scaling == N.PA_ROPE_SCALE_NTK:
        base *= d.factor ** (R / (R - 2))
    at = lambda turns: R * math.log(d.original_len / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        if d.scaling == N.PA_ROPE_SCALE_LINEAR:
            f /= d.factor
        elif d.scaling == N.PA_ROPE_SCALE_BANDS:
            r = d.original_len * f / (2 * math.pi)
            g = 0.0 if r <= d.low else 1.0 if r >= d.high else (r - d.low) / (d.high - d.low)
            f = g * f + (1 - g) * f / d.factor
        elif d.scaling == N.PA_ROPE_SCALE_YARN:
            lo, hi = max(math.floor(at(d.high)), 0), min(math.ceil(at(d.low)), R - 1)
            g = 1.0 if i <= lo else 0.0 if i >= hi else (hi - i) / (hi - lo)
            f = g * f + (1 - g) * f / d.factor
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("kw", [
    {}, dict(rot_dim=2), dict(rot_dim=20), dict(rot_dim=128, theta=500000.0),
    dict(scaling=N.PA_ROPE_SCALE_LINEAR), dict(scaling=N.PA_ROPE_SCALE_NTK),
    dict(scaling=N.PA_ROPE_SCALE_BANDS), dict(scaling=N.PA_ROPE_SCALE_BANDS, rot_dim=128, original_len=8192.0),
    dict(scaling=N.PA_ROPE_SCALE_YARN, high=32.0), dict(scaling=N.PA_ROPE_SCALE_YARN, high=32.0, rot_dim=30),
    dict(scaling=N.PA_ROPE_SCALE_YARN, original_len=100.0),  # the edges clamp
    dict(scaling=N.PA_ROPE_SCALE_LINEAR, factor=0.01)])     # faster than a turn per position
def test_speeds(lib, kw):
    d = _desc(**kw)
    r = N.pa_rope_init(d)
    assert (r.layout, r.rot_dim, r.gain) == (d.layout, d.rot_dim, np.float32(d.gain))
    turns = _speeds(d) / (2 * math.pi)
    got = np.array([float(Fraction(r.step[i], 1 << 64)) for i in range(64)])
    assert np.all(got[d.rot_dim // 2:] == 0)
    off = got[:d.rot_dim // 2] - turns % 1.0
    off -= np.round(off)  # 0 and 1 are the same turn
    # a dozen double operations (pow, log: a few units in the last place each)
    assert np.all(np.abs(off) <= 64 * 2.0 ** -53 * np.maximum(turns, 2.0 ** -11))


def test_divisors(lib):
    d = _desc(rot_dim=16)
    div = np.linspace(1, 5, 8)
    plain, cut = N.pa_rope_init(d), N.pa_rope_init(d, div)
    for i in range(8):
        assert cut.step[i] == pytest.approx(plain.step[i] / div[i], rel=1e-14)
    with pytest.raises(ValueError):
        N.pa_rope_init(d, div[:7])


@pytest.mark.parametrize("kw", [
    dict(layout=2), dict(layout=-1), dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(rot_dim=-2),
    dict(scaling=5), dict(scaling=-1), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan),
    dict(gain=math.nan), dict(gain=1e39), dict(scaling=N.PA_ROPE_SCALE_LINEAR, factor=0.0),
    dict(scaling=N.PA_ROPE_SCALE_LINEAR, factor=math.nan), dict(scaling=N.PA_ROPE_SCALE_NTK, rot_dim=2),
    dict(scaling=N.PA_ROPE_SCALE_BANDS, low=4.0), dict(scaling=N.PA_ROPE_SCALE_BANDS, low=0.0),
    dict(scaling=N.PA_ROPE_SCALE_YARN, original_len=0.0), dict(scaling=N.PA_ROPE_SCALE_YARN, high=math.inf)])
def test_init_refusals(lib, kw):
    with pytest.raises(N.PAError) as e:
        N.pa_rope_init(_desc(**kw))
    assert e.value.code == INV


@pytest.mark.parametrize("bad", [0.0, -1.0, math.nan, math.inf])
def test_divisor_refusals(lib, bad):
    with pytest.raises(N.PAError) as e:
        N.pa_rope_init(_desc(rot_dim=4), [1.0, bad])
    assert e.value.code == INV


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses")
def test_call_refusals(lib):
    h = N.pa_pool_create(N.make_desc(2, 64, 2, 64, N.PA_FP16), FAKE_K, FAKE_V)
    rope = N.pa_rope_init(_desc())
    wide = N.pa_rope_init(_desc(rot_dim=66))

    def call(**kw):
        a = dict(layer=0, rope=rope, q=A, qs=256, q_out=A, Hq=4, k=A, ks=128, v=A, vs=128, pos=A, slots=A, T=3)
        a.update(kw)
        N.pa_rope_and_cache(h, *a.values(), 0)

    try:
        call(T=0)
        call(T=0, q=0)
        for kw, code in [(dict(layer=2), INV), (dict(layer=-1), INV), (dict(rope=wide), INV), (dict(rope=None), INV),
                         (dict(rope=N.pa_rope()), INV), (dict(T=-1), INV), (dict(Hq=0), INV),
                         (dict(Hq=1 << 20, qs=1 << 27), UNS), (dict(qs=248), INV), (dict(qs=257), INV),
                         (dict(qs=-256), INV), (dict(ks=120), INV), (dict(vs=132), INV), (dict(q=0), INV),
                         (dict(q_out=0), INV), (dict(k=0), INV), (dict(v=0), INV), (dict(pos=0), INV),
                         (dict(slots=0), INV), (dict(q=A + 8), INV), (dict(v=A + 2), INV), (dict(q_out=A + 4), INV),
                         (dict(qs=264), INV)]:  # rotating in place needs contiguous queries
            with pytest.raises(N.PAError) as e:
                call(**kw)
            assert e.value.code == code, kw
    finally:
        N.pa_pool_destroy(h)
