"""pa_rope_and_cache where a token's heads fill a warp's rounds unevenly: from 2048 tokens on a
warp turns a whole token, in rounds of 32 or 64 units (16 values of a head), and the last
round of 9 heads of 128 dimensions (72 units) or of 17 and 20 of 64 (68, 80) is a part of one."""
import numpy as np
import pytest
import torch

from test_gpu_rope import _check8, _check16, _exact, _inputs, _pool, _rope, _rows
from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("T", [2048, 2500])
@pytest.mark.parametrize("kv, Hq, H, D, rope", [
    ("bf16", 9, 3, 128, dict(rot_dim=128)),
    ("bf16", 9, 9, 128, dict(rot_dim=42)),                           # partners read one by one
    ("fp16", 17, 17, 64, dict(rot_dim=64, layout="interleaved")),
    ("fp16", 17, 1, 64, dict(rot_dim=20)),
    ("fp8_e4m3", 20, 20, 64, dict(rot_dim=32)),
    ("fp8_e4m3", 33, 11, 128, dict(rot_dim=128, scaling="yarn", factor=16.0)),
    ("fp8_e4m3_block", 9, 3, 128, dict(rot_dim=128, layout="interleaved")),
    ("fp8_e4m3_block", 17, 1, 64, dict(rot_dim=62))])
def test_uneven_rounds(kv, Hq, H, D, rope, T):
    """Every head of every token against fp64, and the same bits when turned in place."""
    rope = _rope(**rope)
    blocks = -(-T // 16) + 2
    pool = _pool(kv, H, D, blocks)
    q, k, v = _inputs(T, Hq, H, D, pool.in_dtype, False, Hq)
    rng = np.random.default_rng(T + Hq)
    ids = rng.permutation(blocks)
    slots = torch.from_numpy(np.array([ids[i // 16] * 16 + i % 16 for i in range(T)])).cuda()
    pos = torch.from_numpy(rng.integers(0, 2 ** 20, T).astype(np.int32)).cuda()
    out = pool.rope_and_cache(rope, q, k, v, pos, slots)
    first = pool.k_cache.clone(), pool.v_cache.clone()
    _check16(out, *_exact(q, pos, rope), pool.in_dtype)
    for which, (y, err) in (("k", _exact(k, pos, rope)), ("v", (v.double().cpu().numpy(), np.zeros(v.shape)))):
        rows = _rows(pool, which, slots).contiguous()
        if not kv.startswith("fp8"):
            _check16(rows.view(pool.in_dtype), y, err, pool.in_dtype)
        elif kv == "fp8_e4m3":
            _check8(rows, float(np.float32(0.02 if which == "k" else 0.03)), y, err)
        else:
            sc = pool.scale_view(which)[slots // 16].double().cpu().numpy()  # [T, H]
            for h in range(H):
                _check8(rows[:, h].contiguous(), sc[:, h, None], y[:, h], err[:, h])
    same = pool.rope_and_cache(rope, q, k, v, pos, slots, q_out=q)
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, out)
    assert torch.equal(pool.k_cache, first[0]) and torch.equal(pool.v_cache, first[1])
    assert pool.device_error() == N.PA_OK
    pool.close()
