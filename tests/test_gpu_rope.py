"""pa_rope_and_cache against the rotation written out in fp64.

Tolerances.  The kernel's cos and sin carry the rounding of the angle's
fraction of half a turn to fp32 (pi 2^-25), sincospif's error and the product
with gain: below 4 units of 2^-24 in all, times gain.  The two products and
their sum add three roundings.  So a rotated value is within
8 2^-24 gain (|a| + |b|) of exact before its one rounding to the output type,
which adds half a step: eps / 2 of the value (and half the smallest step of a
binary16 number, or of an E4M3 code)."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu

KINDS = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _pool(kv, H, D, blocks, **kw):
    from paged_kv_cache_270_gb300.pool import KVPool
    p = KVPool(kw.pop("layers", 1), blocks, H, D, kv, 0.02, 0.03)
    p.k_cache.fill_(0xFF)
    p.v_cache.fill_(0xFF)
    return p


def _speeds(rope):
    return np.array([rope.step[i] / 2.0 ** 64 for i in range(rope.rot_dim // 2)])


def _exact(x, positions, rope):
    """Rotated x [T, H, D] in fp64, and the error the fp32 arithmetic may make."""
    x = x.double().cpu().numpy()
    R, gain = rope.rot_dim, float(rope.gain)
    # whole turns are dropped from the integer product, so the angle is exact
    steps = [int(rope.step[i]) for i in range(R // 2)]
    turns = np.array([[((s * int(p)) % (1 << 64)) / 2.0 ** 64 for s in steps] for p in positions.tolist()])
    c, s = (gain * f(2 * math.pi * turns)[:, None, :] for f in (np.cos, np.sin))
    ia = np.arange(R // 2) if rope.layout == N.PA_ROPE_HALF else 2 * np.arange(R // 2)
    ib = ia + (R // 2 if rope.layout == N.PA_ROPE_HALF else 1)
    a, b = x[..., ia], x[..., ib]
    y, err = x.copy(), np.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err[..., ia] = err[..., ib] = 8 * 2.0 ** -24 * abs(gain) * (np.abs(a) + np.abs(b))
    return y, err


def _check16(got, y, err, dtype):
    got = got.double().cpu().numpy()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = err + torch.finfo(dtype).eps / 2 * (np.abs(y) + err) + tiny
    assert np.all(np.abs(got - y) <= tol), float(np.max(np.abs(got - y) - tol))


def _check8(codes, scale, y, err):
    got = codes.view(torch.float8_e4m3fn).double().cpu().numpy() * scale
    y = np.clip(y, -448 * scale, 448 * scale)
    tol = err + 2.0 ** -4 * (np.abs(y) + err) * (1 + 2.0 ** -20) + 2.0 ** -10 * scale
    assert np.all(np.abs(got - y) <= tol), float(np.max(np.abs(got - y) - tol))


def _inputs(T, Hq, H, D, dtype, fused, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = torch.randn(T, Hq + 2 * H, D, device="cuda", generator=g).to(dtype)
        return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    return tuple(torch.randn(T, h, D, device="cuda", generator=g).to(dtype) for h in (Hq, H, H))


def _rows(pool, which, slots):
    """The cache rows of `slots` as uint8 [n, H, row bytes]."""
    v = pool.layer_view(which)
    return v[slots // 16, :, slots % 16]


def _rope(**kw):
    from paged_kv_cache_270_gb300.pool import make_rope
    return make_rope(**kw)


CASES = [  # kv, T, Hq, H, D, rope, fused
    ("bf16", 1, 4, 1, 128, dict(rot_dim=128), False),
    ("fp16", 37, 4, 2, 64, dict(rot_dim=64, layout="interleaved"), True),
    ("fp16", 5, 8, 8, 128, dict(rot_dim=6), False),
    ("bf16", 64, 32, 8, 128, dict(rot_dim=128, theta=5e5, scaling="bands", factor=8.0), True),
    ("bf16", 33, 3, 1, 64, dict(rot_dim=20), True),
    ("bf16", 9, 7, 7, 64, dict(rot_dim=62, layout="interleaved"), False),
    ("fp8_e4m3", 129, 64, 8, 128, dict(rot_dim=128, scaling="yarn", factor=16.0), True),
    ("fp8_e4m3", 17, 2, 2, 64, dict(rot_dim=16), False),
    ("fp8_e4m3", 3, 1, 1, 128, dict(rot_dim=100, gain=0.5), False),
    ("fp8_e4m3", 1000, 4, 2, 64, dict(rot_dim=2, layout="interleaved", scaling="linear", factor=4.0), True),
    ("fp8_e4m3_block", 70, 8, 1, 128, dict(rot_dim=128), True),
    ("fp8_e4m3_block", 41, 16, 5, 64, dict(rot_dim=32, layout="interleaved", scaling="ntk", factor=4.0), False),
    ("fp8_e4m3_block", 16, 2, 2, 128, dict(rot_dim=44), True),
]


@pytest.mark.parametrize("kv, T, Hq, H, D, rope, fused", CASES)
def test_against_fp64(kv, T, Hq, H, D, rope, fused):
    rope = _rope(**rope)
    blocks = -(-T // 16) + 3
    pool = _pool(kv, H, D, blocks)
    q, k, v = _inputs(T, Hq, H, D, pool.in_dtype, fused, T)
    rng = np.random.default_rng(T)
    ids = rng.permutation(blocks)
    slots = torch.from_numpy(np.array([ids[i // 16] * 16 + i % 16 for i in range(T)])).cuda()
    pos = torch.from_numpy(rng.integers(0, 2 ** 20, T).astype(np.int32)).cuda()
    pos[0], pos[-1] = 2 ** 31 - 1, -12345
    out = pool.rope_and_cache(rope, q, k, v, pos, slots)
    assert pool.device_error() == N.PA_OK
    _check16(out, *_exact(q, pos, rope), pool.in_dtype)
    for which, (y, err) in (("k", _exact(k, pos, rope)), ("v", (v.double().cpu().numpy(), 0.0))):
        rows = _rows(pool, which, slots)
        if not kv.startswith("fp8"):
            _check16(rows.contiguous().view(pool.in_dtype), y, err, pool.in_dtype)
        elif kv == "fp8_e4m3":
            _check8(rows.contiguous(), float(np.float32(0.02 if which == "k" else 0.03)), y, err)
        else:
            sc = pool.scale_view(which)
            for j in range(-(-T // 16)):
                t = slice(16 * j, min(T, 16 * j + 16))
                for h in range(H):
                    s = float(sc[int(ids[j]), h])
                    # one division of a value off by err: 2^-24 relative on top
                    want, e = np.abs(y[t, h]).max() / 448, np.max(err[t, h]) / 448 if which == "k" else 0.0
                    assert abs(s - want) <= e + 2.0 ** -23 * want
                    _check8(rows[t, h].contiguous(), s, y[t, h], err[t, h] if which == "k" else 0.0)
    pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_position_zero_is_the_plain_write(kv):
    """At position 0 nothing turns: the cache then holds, bit for bit, what
    pa_reshape_and_cache writes, run by run (appends with growing and with
    shrinking magnitudes among them), and q_out is q."""
    H, D, blocks = 3, 128, 9
    one, two = (_pool(kv, H, D, blocks) for _ in range(2))
    rope = _rope(rot_dim=128)
    at, ids = 0, [7, 2, 5, 0]
    for step, (n, mag) in enumerate([(5, 1.0), (3, 4.0), (1, 0.5), (20, 1.0), (1, 9.0), (18, 2.0)]):
        q, k, v = (x * mag for x in _inputs(n, 6, H, D, one.in_dtype, False, step))
        slots = torch.tensor([ids[i // 16] * 16 + i % 16 for i in range(at, at + n)], device="cuda")
        out = one.rope_and_cache(rope, q, k, v, torch.zeros(n, dtype=torch.int32, device="cuda"), slots)
        two.reshape_and_cache(k, v, slots)
        at += n
        assert torch.equal(out, q)
        assert torch.equal(one.k_cache, two.k_cache) and torch.equal(one.v_cache, two.v_cache), step
    assert one.device_error() == N.PA_OK
    one.close()
    two.close()


@pytest.mark.parametrize("kv", KINDS)
def test_skipped_and_bad_slots(kv):
    """Negative slots write nothing, a slot past the pool writes nothing and is
    reported; every token's query is rotated; nothing else is touched."""
    H, D, blocks, T = 2, 64, 4, 6
    pool = _pool(kv, H, D, blocks, layers=2)
    before = pool.k_cache.clone(), pool.v_cache.clone()
    q, k, v = _inputs(T, 4, H, D, pool.in_dtype, False, 3)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    rope = _rope(rot_dim=64)
    out = pool.rope_and_cache(rope, q, k, v, pos, torch.full((T,), -1, dtype=torch.int64, device="cuda"), layer=1)
    assert pool.device_error() == N.PA_OK
    _check16(out, *_exact(q, pos, rope), pool.in_dtype)
    assert torch.equal(pool.k_cache, before[0]) and torch.equal(pool.v_cache, before[1])
    slots = torch.tensor([-5, blocks * 16, 1 << 40, 16, 17, -1], device="cuda")
    pool.rope_and_cache(rope, q, k, v, pos, slots, layer=1)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    # layer 0 is as it was, and of layer 1 only rows 0 and 1 of block 1 changed
    for which in ("k", "v"):
        assert bool((pool.layer_view(which, 0) == 0xFF).all())
        changed = (pool.layer_view(which, 1) != 0xFF).flatten(3).any(3)  # [blocks, H, 16]
        assert changed[1, :, 0].all() and changed.sum() <= 2 * H
        assert not changed[[0, 2, 3]].any()
    pool.close()


@pytest.mark.parametrize("rot, layout", [(128, "half"), (128, "interleaved"), (42, "half"), (48, "half")])
def test_in_place(rot, layout):
    """q_out may be q."""
    pool = _pool("bf16", 8, 128, 16)
    rope = _rope(rot_dim=rot, layout=layout)
    q, k, v = _inputs(100, 40, 8, 128, torch.bfloat16, False, 1)
    slots = torch.arange(100, device="cuda")
    pos = torch.arange(100, dtype=torch.int32, device="cuda") + 70000
    apart = pool.rope_and_cache(rope, q, k, v, pos, slots)
    same = pool.rope_and_cache(rope, q, k, v, pos, slots, q_out=q)
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, apart)
    with pytest.raises(N.PAError):
        x = torch.zeros(4, 56, 128, dtype=torch.bfloat16, device="cuda")
        N.pa_rope_and_cache(pool.handle, 0, rope, x.data_ptr(), 56 * 128, x.data_ptr(), 40, x.data_ptr(), 56 * 128,
                            x.data_ptr(), 56 * 128, pos.data_ptr(), slots.data_ptr(), 4, 0)
    pool.close()


def test_unturned_dims_pass_through():
    """Infinities and NaN behind rot_dim stay where they are, in q and in the cache."""
    for layout, rot in (("half", 32), ("interleaved", 30), ("half", 14)):
        pool = _pool("bf16", 1, 64, 2)
        q, k, v = _inputs(2, 1, 1, 64, torch.bfloat16, False, 5)
        for x in (q, k):
            x[..., rot] = math.inf
            x[..., rot + 1] = math.nan
            x[..., 63] = -math.inf
        out = pool.rope_and_cache(_rope(rot_dim=rot, layout=layout), q, k, v,
                                  torch.tensor([3, 4], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], device="cuda"))
        kept = _rows(pool, "k", torch.tensor([0, 1], device="cuda")).contiguous().view(torch.bfloat16)
        for got, x in ((out, q), (kept, k)):
            assert torch.isfinite(got[..., :rot]).all()
            assert torch.equal(got[..., rot:].nan_to_num(7.0), x[..., rot:].nan_to_num(7.0))
            assert torch.equal(got[..., rot:].isnan(), x[..., rot:].isnan())
        pool.close()


def test_graph_and_other_stream():
    """A captured call replays on new inputs; a call on a side stream orders there."""
    pool = _pool("fp8_e4m3", 8, 128, 8)
    rope = _rope(rot_dim=128)
    q, k, v = _inputs(24, 16, 8, 128, torch.bfloat16, True, 0)
    pos = torch.arange(24, dtype=torch.int32, device="cuda")
    slots = torch.arange(24, device="cuda")
    out = torch.empty(24, 16, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = pool.rope_and_cache(rope, q, k, v, pos + 5, slots).clone()
    cache = pool.k_cache.clone()
    torch.cuda.synchronize()
    pool.k_cache.fill_(0xFF)  # as it was before the first call
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pool.rope_and_cache(rope, q, k, v, pos, slots, q_out=out)
        pos += 5
        g.replay()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pool.k_cache, cache)
    pool.close()


def test_many_tokens():
    """A packet of 8192 tokens, spot-checked against fp64."""
    T, Hq, H = 8192, 64, 8
    pool = _pool("fp8_e4m3", H, 128, T // 16)
    rope = _rope(rot_dim=128, scaling="yarn", factor=16.0)
    q, k, v = _inputs(T, Hq, H, 128, torch.bfloat16, True, 9)
    slots = torch.randperm(T, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 100000
    out = pool.rope_and_cache(rope, q, k, v, pos, slots)
    pick = torch.randint(0, T, (64,), device="cuda")
    _check16(out[pick], *_exact(q[pick], pos[pick], rope), torch.bfloat16)
    _check8(_rows(pool, "k", slots[pick]).contiguous(), float(np.float32(0.02)), *_exact(k[pick], pos[pick], rope))
    pool.close()


def test_wrapper_refusals():
    pool = _pool("bf16", 2, 64, 2)
    rope = _rope(rot_dim=64)
    q, k, v = _inputs(3, 4, 2, 64, torch.bfloat16, False, 0)
    pos, slots = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(k=k[:2]), dict(v=v[:, :1]), dict(pos=pos.long()),
                dict(slots=slots[:2]), dict(slots=slots.int()), dict(q=q.cpu()), dict(q=q[0]), dict(k=k[..., :32])):
        a = dict(q=q, k=k, v=v, pos=pos, slots=slots)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            pool.rope_and_cache(rope, a["q"], a["k"], a["v"], a["pos"], a["slots"])
    pool.rope_and_cache(rope, q[:0], k[:0], v[:0], pos[:0], slots[:0])
    pool.close()
