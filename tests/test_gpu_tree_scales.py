"""pa_decode_tree on block-scaled pools whose tiles' V scales lie far apart, between tiles that a node sees and
tiles that it does not, and between tiles of large and of small weight.

Tolerance: that of tree_reference, but for the weights' smallest step.  A weight times its tile's V scale is
held in binary16 with the largest such product of the row at 2^6 or above, so a key is off by at most
2^-25 of 2^6 of that product, times its code: 2^-31 max_j(p_j s_j) sum_j |c_j|."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from tree_reference import Batch, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _node_rows(b, s):
    q0 = int(b.q_start_np[s])
    return [(q0 + r, np.concatenate([np.arange(b.ctx[s] - b.sizes[s]), b.ctx[s] - b.sizes[s] + np.flatnonzero(b.sees[s][r])]))
            for r in range(b.sizes[s])]


def check_sharp(b, out):
    """Every row of a block-scaled batch against fp64, with the docstring's tolerance."""
    H, G, D = b.H, b.G, b.D
    k_all, v_all = values(b.pool, "k"), values(b.pool, "v")
    codes = b.pool.layer_view("v").contiguous().view(torch.float8_e4m3fn).double()
    scales = b.pool.scale_view("v").double()
    f32 = out.dtype == torch.float32
    for s, n in enumerate(b.ctx):
        i = np.arange(n)
        blk, off = torch.from_numpy(b.tables_np[s, i // 16].astype(np.int64)).cuda(), torch.from_numpy(i % 16).cuda()
        k, v, c, sc = k_all[blk, :, off], v_all[blk, :, off], codes[blk, :, off], scales[blk]
        for row, vis in _node_rows(b, s):
            vi = torch.from_numpy(vis).cuda()
            q = b.q[row].double().view(H, G, D)
            kk, vv = k[vi], v[vi]
            f = 1.0 / math.sqrt(D)
            p = torch.softmax(torch.einsum("hgd,mhd->hgm", q, kk) * f, -1)
            ez = torch.einsum("hgd,mhd->hgm", q.abs(), kk.abs()) * f * 2 * D * 2.0 ** -24
            ez = ez + q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).T[:, None, :] * f * 2.0 ** -17
            o, a = (torch.einsum("hgm,mhd->hgd", p, x) for x in (vv, vv.abs()))
            # an exponent of up to 128 is rounded to 2^-18 (fp32 outputs), and its tile's log2 scale to 2^-17 and the
            # sum with the row's reference to 2^-18 before (16-bit outputs); twice, for the sums' share
            rel = 4 * ez.amax(-1, keepdim=True) + (2.0 ** -21 + 2.0 ** -17 if f32 else 2.0 ** -11 + 2.0 ** -15)
            rel = rel + (len(vis) / 16 + 32) * 2.0 ** -23
            top = (p * sc[vi].T[:, None, :]).amax(-1, keepdim=True)
            e = rel * a + 2.0 ** -31 * top * c[vi].abs().sum(0)[:, None, :]
            tol = e + torch.finfo(out.dtype).eps / 2 * (o.abs() + e)
            got = out[row].double().view(H, G, D)
            over = float(((got - o).abs() - tol).max())
            assert over <= 0, f"row {row}: off by {over:.3e} over the tolerance"


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("up", [24, 32, 60, 100])
@pytest.mark.parametrize("ctx, size", [(70, 60), (300, 60), (9000, 90)])
def test_scale_of_an_unseen_tile(ctx, size, up, out_dtype):
    """A tile of nodes that a row does not see may have any finite V scale: the row's bits stay.  Rows that
    see it are held to fp64."""
    b = Batch("fp8_e4m3_block", 2, 3, 128, [ctx, 200], [size, 20], mask="tree", seed=up)
    base = ctx - size
    page = -(-base // 16) + 1  # a page of nodes alone
    nodes = np.arange(16 * page, min(16 * page + 16, ctx)) - base
    want = b.run(out_dtype=out_dtype)
    b.pool.scale_view("v")[int(b.tables_np[0, page])] *= 2.0 ** up
    out = b.run(out_dtype=out_dtype)
    seen = b.sees[0][:, nodes].any(1)
    assert 0 < seen.sum() < size
    for r in range(size):
        if not seen[r]:
            assert torch.equal(out[r], want[r]), r
    assert torch.equal(out[size:], want[size:])
    check_sharp(b, out)
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("up", [20, 40, 60])
@pytest.mark.parametrize("ctx, page", [(100, 0), (100, 4), (1000, 17), (20000, 900)])
def test_large_scale_under_a_small_weight(ctx, page, up, out_dtype):
    """A seen tile whose keys have next to no weight takes nothing from the others' weights, however
    large its values are (less than its weights are small)."""
    b = Batch("fp8_e4m3_block", 2, 1, 128, [ctx], [1], seed=up)
    blk = int(b.tables_np[0, page])
    slots = torch.arange(16, device="cuda") + 16 * blk
    k = -2.0 * b.q[0].view(1, 2, 128).expand(16, 2, 128)  # scores near -50: weights near 2^-73
    g = torch.Generator(device="cuda").manual_seed(9)
    v = torch.randn(16, 2, 128, device="cuda", generator=g).bfloat16()
    b.pool.reshape_and_cache(k.contiguous(), v, slots)
    b.pool.scale_view("v")[blk] *= 2.0 ** up
    check_sharp(b, b.run(out_dtype=out_dtype))
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp8_e4m3_block"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_from_zero(kv, sign):
    """Scores of 10^6 and more, one key far above (or the least far below) the others: its value, rounded once."""
    b = Batch(kv, 2, 1, 128, [700, 33, 9000], [1, 1, 1], seed=41)
    g = torch.Generator(device="cuda").manual_seed(4)
    for s, at in enumerate((650, 3, 100)):
        b.q[s] = (1e5 * torch.randn(2, 128, device="cuda", generator=g)).bfloat16()
        q = b.q[s].float() / 1e5
        n = b.ctx[s]
        # every key against the query (or along it), the chosen one along it (or a quarter as far)
        i = np.arange(n)
        slots = torch.from_numpy(b.tables_np[s, i // 16].astype(np.int64) * 16 + i % 16).cuda()
        k = (-q if sign > 0 else -4.0 * q).view(1, 2, 128).repeat(n, 1, 1)
        k[at] *= -1.0 if sign > 0 else 0.25
        v = torch.randn(n, 2, 128, device="cuda", generator=g).bfloat16()
        b.pool.reshape_and_cache(k.bfloat16(), v, slots)
    v_all = values(b.pool, "v")
    for dt in (None, torch.float32):
        out = b.run(out_dtype=dt)
        for s, at in enumerate((650, 3, 100)):
            want = v_all[int(b.tables_np[s, at // 16]), :, at % 16]
            # the one weight's rounding for the product with V (tree_reference), ex2's and the sums' 2^-20, and the output's
            dp = 2.0 ** -17 if kv == "bf16" else 2.0 ** -22 if dt else 2.0 ** -12
            tol = want.abs() * (torch.finfo(out.dtype).eps / 2 + dp + 2.0 ** -20)
            assert bool(((out[s].double() - want).abs() <= tol).all()), (dt, s)
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
