"""pa_norm_rope_and_cache against the norm and the rotation written out in fp64.

Tolerances, in units of 2^-24.  The sum of squares of a head passes at most 10
additions and a product: 12 with the mean and eps, half of it (6) under the root;
rsqrtf gives 2 steps of 2^-23 (4); weight_offset + w and the two products 3.  So
a normalised value is within 14 units of exact (relative), and the rotation adds 8 of
(|a| + |b|) gain, as for pa_rope_and_cache: 24 units of (|a| + |b|) |gain| where a pair
turns, 14 of the value where it does not, before the one rounding to the output type."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from test_gpu_rope import _check8, _check16, _inputs, _pool, _rope, _rows

pytestmark = pytest.mark.gpu

KINDS = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _axes(sections, order):
    from paged_kv_cache_270_gb300.pool import make_rope_axes
    return make_rope_axes(sections, order)


def _exact(x, positions, rope, axes, w, eps, offset):
    """x [T, H, D] normalised (w: None, [D] or [H, D]) and rotated in fp64, and its error bound."""
    x = x.double().cpu().numpy()
    u = 2.0 ** -24
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + w.double().cpu().numpy())
    R, gain = rope.rot_dim, float(rope.gain)
    pos = positions.cpu().numpy().reshape(-1, x.shape[0])
    steps = [int(rope.step[i]) for i in range(R // 2)]
    of = [axes.axis[i] if axes is not None else 0 for i in range(R // 2)]
    turns = np.array([[((s * int(pos[a, t])) % (1 << 64)) / 2.0 ** 64 for s, a in zip(steps, of)] for t in range(x.shape[0])])
    c, s = (gain * f(2 * math.pi * turns)[:, None, :] for f in (np.cos, np.sin))
    ia = np.arange(R // 2) if rope.layout == N.PA_ROPE_HALF else 2 * np.arange(R // 2)
    ib = ia + (R // 2 if rope.layout == N.PA_ROPE_HALF else 1)
    a, b = x[..., ia], x[..., ib]
    y, err = x.copy(), (14 * u * np.abs(x) if w is not None else np.zeros_like(x))
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err[..., ia] = err[..., ib] = (24 if w is not None else 8) * u * abs(gain) * (np.abs(a) + np.abs(b))
    return y, err


CASES = [  # kv, T, Hq, H, D, rope, sections (None: one axis), order, weights, offset, fused
    ("bf16", 1, 4, 1, 128, dict(rot_dim=128), None, "", "shared", 0.0, False),
    ("bf16", 64, 32, 8, 128, dict(rot_dim=128), [16, 24, 24], "sections", "shared", 0.0, True),
    ("fp16", 37, 4, 2, 64, dict(rot_dim=64, layout="interleaved"), [12, 10, 10], "turns", "head", 1.0, True),
    ("fp16", 5, 8, 8, 128, dict(rot_dim=6), [1, 1, 1], "turns", "shared", 1.0, False),
    ("bf16", 33, 3, 1, 64, dict(rot_dim=20), None, "", "head", 0.0, True),
    ("bf16", 9, 7, 7, 64, dict(rot_dim=62, layout="interleaved", gain=1.3), [31, 0], "sections", "q", 0.0, False),
    ("fp8_e4m3", 129, 64, 8, 128, dict(rot_dim=128, scaling="yarn", factor=16.0), [24, 20, 20], "turns", "shared", 0.0, True),
    ("fp8_e4m3", 17, 2, 2, 64, dict(rot_dim=16), [2, 2, 2, 2], "turns", "k", 0.0, False),
    ("fp8_e4m3", 3, 1, 1, 128, dict(rot_dim=100, gain=0.5), [50], "sections", "head", 0.0, False),
    ("fp8_e4m3", 1000, 4, 2, 64, dict(rot_dim=2, layout="interleaved"), [0, 1], "sections", "shared", 0.0, True),
    ("fp8_e4m3_block", 70, 8, 1, 128, dict(rot_dim=128), [16, 24, 24], "sections", "shared", 0.0, True),
    ("fp8_e4m3_block", 41, 16, 5, 64, dict(rot_dim=32, layout="interleaved"), None, "", "head", 1.0, False),
    ("fp8_e4m3_block", 16, 2, 2, 128, dict(rot_dim=44), [8, 7, 7], "turns", "shared", 0.0, True),
    ("fp8_e4m3_block", 35, 3, 3, 128, dict(rot_dim=128), [16, 24, 24], "sections", "none", 0.0, False),
    ("fp8_e4m3_block", 51, 11, 11, 128, dict(rot_dim=90), [15, 15, 15], "turns", "head", 1.0, True),
    ("fp8_e4m3_block", 30, 9, 9, 64, dict(rot_dim=62, gain=0.7), None, "", "k", 0.0, False),
    ("fp8_e4m3_block", 64, 5, 1, 64, dict(rot_dim=64), [12, 10, 10], "sections", "shared", 0.0, False),
    ("fp8_e4m3_block", 29, 2, 2, 128, dict(rot_dim=126, layout="interleaved"), None, "", "shared", 0.0, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_fp64(case):
    kv, T, Hq, H, D, rope, sections, order, weights, offset, fused = CASES[case]
    rope = _rope(**rope)
    axes = _axes(sections, order) if sections else None
    blocks = -(-T // 16) + 3
    pool = _pool(kv, H, D, blocks)
    q, k, v = _inputs(T, Hq, H, D, pool.in_dtype, fused, T)
    g = torch.Generator(device="cuda").manual_seed(T)
    qw, kw = ((torch.randn((h, D) if weights == "head" else (D,), device="cuda", generator=g) * 0.3 + 1 - offset).to(pool.in_dtype)
              for h in (Hq, H))
    qw = qw if weights in ("shared", "head", "q") else None
    kw = kw if weights in ("shared", "head", "k") else None
    rng = np.random.default_rng(T)
    ids = rng.permutation(blocks)
    slots = torch.from_numpy(np.array([ids[i // 16] * 16 + i % 16 for i in range(T)])).cuda()
    n = len(sections) if sections else 1
    pos = torch.from_numpy(rng.integers(0, 2 ** 20, (n, T)).astype(np.int32)).cuda()
    pos[0, 0], pos[-1, -1] = 2 ** 31 - 1, -12345
    eps = 1e-5
    out = pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=qw, k_weight=kw, eps=eps, weight_offset=offset, axes=axes)
    assert pool.device_error() == N.PA_OK
    e32 = float(np.float32(eps))
    _check16(out, *_exact(q, pos, rope, axes, qw, e32, offset), pool.in_dtype)
    for which, (y, err) in (("k", _exact(k, pos, rope, axes, kw, e32, offset)), ("v", (v.double().cpu().numpy(), 0.0))):
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
                    want, e = np.abs(y[t, h]).max() / 448, np.max(err[t, h]) / 448 if which == "k" else 0.0
                    assert abs(s - want) <= e + 2.0 ** -23 * want
                    _check8(rows[t, h].contiguous(), s, y[t, h], err[t, h] if which == "k" else 0.0)
    pool.close()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("rot, layout", [(128, "half"), (96, "interleaved"), (42, "half")])
def test_without_norm_it_is_the_rotary_write(kv, rot, layout):
    """No weights and equal positions on all axes: pa_rope_and_cache, bit for bit."""
    one, two = (_pool(kv, 3, 128, 9) for _ in range(2))
    rope = _rope(rot_dim=rot, layout=layout)
    axes = _axes([rot // 2 - 2 * (rot // 8), rot // 8, rot // 8], "sections")
    q, k, v = _inputs(77, 6, 3, 128, one.in_dtype, True, 1)
    slots = torch.arange(77, device="cuda") + 5
    pos = torch.arange(77, dtype=torch.int32, device="cuda") * 317
    a = one.norm_rope_and_cache(rope, q, k, v, pos.expand(3, 77).contiguous(), slots, axes=axes)
    b = two.rope_and_cache(rope, q, k, v, pos, slots)
    assert torch.equal(a, b) and torch.equal(one.k_cache, two.k_cache) and torch.equal(one.v_cache, two.v_cache)
    one.close()
    two.close()


@pytest.mark.parametrize("kv", KINDS)
def test_skipped_and_bad_slots(kv):
    pool = _pool(kv, 2, 64, 4)
    before = pool.k_cache.clone(), pool.v_cache.clone()
    q, k, v = _inputs(6, 4, 2, 64, pool.in_dtype, False, 3)
    pos = torch.arange(6, dtype=torch.int32, device="cuda") * 1000
    w = torch.rand(64, device="cuda").to(pool.in_dtype)
    rope = _rope(rot_dim=64)
    out = pool.norm_rope_and_cache(rope, q, k, v, pos, torch.full((6,), -1, device="cuda"), q_weight=w, k_weight=w)
    assert pool.device_error() == N.PA_OK
    _check16(out, *_exact(q, pos, rope, None, w, float(np.float32(1e-6)), 0.0), pool.in_dtype)
    assert torch.equal(pool.k_cache, before[0]) and torch.equal(pool.v_cache, before[1])
    pool.norm_rope_and_cache(rope, q, k, v, pos, torch.tensor([-5, 64, 1 << 40, 16, 17, -1], device="cuda"), q_weight=w, k_weight=w)
    assert pool.device_error() == N.PA_ERR_BOUNDS
    for which in ("k", "v"):
        changed = (pool.layer_view(which) != 0xFF).flatten(3).any(3)
        assert changed[1, :, 0].all() and changed.sum() <= 4 and not changed[[0, 2, 3]].any()
    pool.close()


@pytest.mark.parametrize("rot, layout", [(128, "half"), (128, "interleaved"), (42, "half"), (48, "half")])
def test_in_place(rot, layout):
    """q_out may be q."""
    pool = _pool("bf16", 8, 128, 16)
    rope = _rope(rot_dim=rot, layout=layout)
    q, k, v = _inputs(100, 40, 8, 128, torch.bfloat16, False, 1)
    w = (torch.rand(128, device="cuda") + 0.5).bfloat16()
    slots = torch.arange(100, device="cuda")
    pos = torch.arange(100, dtype=torch.int32, device="cuda") + 70000
    apart = pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=w, k_weight=w)
    same = pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=w, k_weight=w, q_out=q)
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, apart)
    pool.close()


def test_rows_of_zeros_and_infinities():
    """A head of zeros stays zero (eps > 0); an infinite or NaN element spoils its own head alone."""
    pool = _pool("bf16", 2, 64, 1)
    q, k, v = _inputs(3, 4, 2, 64, torch.bfloat16, False, 2)
    w = torch.ones(64, device="cuda").bfloat16()
    rope, slots, pos = _rope(rot_dim=64), torch.arange(3, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    clean = pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=w, k_weight=w).clone()
    q[0, 1] = 0.0
    q[1, 2, 5] = math.inf
    q[2, 3, 63] = math.nan
    out = pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=w, k_weight=w)
    assert bool((out[0, 1] == 0).all())
    assert out[1, 2].isnan().any() and out[2, 3].isnan().all()
    for t, h in ((0, 1), (1, 2), (2, 3)):
        out[t, h] = clean[t, h]
    assert torch.equal(out, clean)
    pool.close()


def test_graph_and_other_stream():
    pool = _pool("fp8_e4m3_block", 8, 128, 8)
    rope, axes = _rope(rot_dim=128), _axes([16, 24, 24], "sections")
    q, k, v = _inputs(24, 16, 8, 128, torch.bfloat16, True, 0)
    w = (torch.rand(128, device="cuda") + 0.5).bfloat16()
    pos = torch.arange(72, dtype=torch.int32, device="cuda").view(3, 24)
    slots = torch.arange(24, device="cuda")
    out = torch.empty(24, 16, 128, dtype=torch.bfloat16, device="cuda")
    want = pool.norm_rope_and_cache(rope, q, k, v, pos + 5, slots, q_weight=w, k_weight=w, axes=axes).clone()
    cache = pool.k_cache.clone()
    torch.cuda.synchronize()
    pool.k_cache.fill_(0xFF)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pool.norm_rope_and_cache(rope, q, k, v, pos, slots, q_weight=w, k_weight=w, axes=axes, q_out=out)
        pos += 5
        g.replay()
    side.synchronize()
    used = torch.arange(2, device="cuda")
    assert torch.equal(out, want)
    assert torch.equal(pool.layer_view("k")[used][:, :, :8], cache[:pool.layer_bytes].view_as(pool.layer_view("k"))[used][:, :, :8])
    pool.close()


def test_wrapper_refusals():
    pool = _pool("bf16", 2, 64, 2)
    rope, axes = _rope(rot_dim=64), _axes([10, 11, 11], "sections")
    q, k, v = _inputs(3, 4, 2, 64, torch.bfloat16, False, 0)
    pos, slots = torch.zeros(3, 3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    w = torch.ones(64, device="cuda").bfloat16()
    ok = dict(rope=rope, q=q, k=k, v=v, positions=pos, slot_mapping=slots, q_weight=w, k_weight=w, axes=axes)
    for bad in (dict(q=q.half()), dict(k=k[:2]), dict(positions=pos[0]), dict(positions=pos.view(-1)), dict(axes=None),
                dict(q_weight=w.half()), dict(q_weight=w[:32]), dict(k_weight=w.expand(4, 64).contiguous()),
                dict(k_weight=w.expand(2, 64).contiguous()), dict(k_weight=w.cpu()), dict(slot_mapping=slots[:2]),
                dict(q_weight=w.expand(4, 64))):
        with pytest.raises((TypeError, ValueError)):
            pool.norm_rope_and_cache(**{**ok, **bad})
    for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(weight_offset=math.inf)):
        with pytest.raises(N.PAError):
            pool.norm_rope_and_cache(**{**ok, **bad})
    pool.norm_rope_and_cache(rope, q[:0], k[:0], v[:0], pos[:, :0].contiguous(), slots[:0], axes=axes)
    pool.close()
