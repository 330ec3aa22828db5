"""pa_norm_rope_and_cache into part-filled tiles of block-scaled pools: a tile's scale grows with the normalised rows,
and the codes that are there already are rounded again to it, bit for bit.

Tolerances: test_gpu_norm_rope (a normalised and turned value's error) and test_gpu_rope (an E4M3 code's half step).  A
scale is the largest value's quotient by 448, so it is off by that value's error over 448 and 2^-23 of itself."""
import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from test_gpu_norm_rope import _axes, _exact
from test_gpu_rope import _check8, _inputs, _pool, _rope

pytestmark = pytest.mark.gpu

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _codes(x):
    return torch.from_numpy(x.clip(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


CASES = [  # H, Hq, D, rope, sections, weights, (tokens there, tokens appended) of each sequence
    (1, 4, 128, dict(rot_dim=128), [16, 24, 24], "shared", [(1, 1), (15, 1), (7, 9), (16, 1)]),
    (8, 32, 128, dict(rot_dim=128), None, "shared", [(5, 16), (31, 40), (3, 2), (14, 1), (90, 17)]),
    (5, 10, 64, dict(rot_dim=32, layout="interleaved"), None, "head", [(9, 30), (1, 14), (33, 5)]),
    (2, 2, 128, dict(rot_dim=90), [15, 15, 15], "head", [(11, 20), (2, 1), (13, 3)]),
    (9, 9, 64, dict(rot_dim=62, gain=0.7), None, "shared", [(4, 4), (15, 33)]),
]


@pytest.mark.parametrize("grow", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, grow):
    H, Hq, D, rope, sections, weights, seqs = CASES[case]
    rope = _rope(**rope)
    axes = _axes(sections, "sections") if sections else None
    pages = [-(-(a + n) // 16) for a, n in seqs]
    pool = _pool("fp8_e4m3_block", H, D, sum(pages) + 2)
    rng = np.random.default_rng(case)
    ids = rng.permutation(pool.num_blocks)
    start = np.concatenate([[0], np.cumsum(pages)])
    slot = lambda s, t: int(ids[start[s] + t // 16]) * 16 + t % 16  # noqa: E731
    old = torch.tensor([slot(s, t) for s, (a, _) in enumerate(seqs) for t in range(a)], device="cuda")
    new = torch.tensor([slot(s, a + t) for s, (a, n) in enumerate(seqs) for t in range(n)], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(case)
    # rows that are there: small ones, so that the appended ones grow the scale, or large ones, so that none does
    size = 0.05 if grow else 40.0
    k0, v0 = ((torch.randn(len(old), H, D, device="cuda", generator=g) * size).bfloat16() for _ in range(2))
    pool.reshape_and_cache(k0, v0, old)
    before = {w: (pool.layer_view(w).cpu().numpy().copy(), pool.scale_view(w).cpu().numpy().copy()) for w in ("k", "v")}
    T = len(new)
    q, k, v = _inputs(T, Hq, H, D, torch.bfloat16, True, case)
    qw, kw = ((torch.randn((h, D) if weights == "head" else (D,), device="cuda", generator=g) * 0.3 + 1).bfloat16()
              for h in (Hq, H))
    pos = torch.from_numpy(rng.integers(0, 2 ** 20, (len(sections) if sections else 1, T)).astype(np.int32)).cuda()
    pool.norm_rope_and_cache(rope, q, k, v, pos, new, q_weight=qw, k_weight=kw, eps=1e-5, axes=axes)
    assert pool.device_error() == N.PA_OK
    slots = new.cpu().numpy()
    for which, (y, err) in (("k", _exact(k, pos, rope, axes, kw, float(np.float32(1e-5)), 0.0)),
                            ("v", (v.double().cpu().numpy(), np.zeros(v.shape)))):
        codes, scales = pool.layer_view(which).cpu().numpy(), pool.scale_view(which).cpu().numpy()
        was_c, was_s = before[which]
        for blk in sorted(set((slots // 16).tolist())):
            rows = np.flatnonzero(slots // 16 == blk)
            offs = slots[rows] % 16
            first = int(offs.min())  # the rows in front of it were there
            for h in range(H):
                s = scales[blk, h]
                s_old = was_s[blk, h] if first else np.float32(0)
                want, e = np.abs(y[rows, h]).max() / 448, err[rows, h].max() / 448
                if first and not grow:
                    assert s == s_old
                else:
                    assert s > s_old and abs(float(s) - want) <= e + 2.0 ** -23 * want
                here = codes[blk, h]
                there = was_c[blk, h, :first]
                assert np.array_equal(here[:first], _codes(E4M3[there] * s_old / s) if s > s_old else there)
                _check8(torch.from_numpy(here[offs]), float(s), y[rows, h], err[rows, h])
    pool.close()
