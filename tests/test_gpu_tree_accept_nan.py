"""pa_tree_accept on block-scaled pools where a moved row holds a NaN: the rows that move with it keep their values."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from test_gpu_tree_accept import Trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


@pytest.mark.parametrize("D", [64, 128])
def test_nan_code_among_moved_rows(D):
    """The scale grows for the finite values, bit for bit as without the NaN, whose own code stays a NaN."""
    paths = [[1, 17, 20, 37]]
    made = []
    for nan in (False, True):
        t = Trees("fp8_e4m3_block", 2, D, [48], [48], paths, layers=2, seed=8)
        for which in ("k", "v"):
            for layer in range(2):
                sc = t.pool.scale_view(which, layer)
                for page, x in enumerate((0.001, 0.03, 0.02)):
                    sc[int(t.t[0, page])] = x
                row = t.pool.layer_view(which, layer)[int(t.t[0, 1]), :, 1]  # node 17
                row[:, 5] = 0x7F if nan else 0x00
                row[:, 40] = 0xFF if nan else 0x80
        before = t.state()
        t.pool.tree_accept(**t.args)
        assert t.pool.device_error() == N.PA_OK
        made.append((before, t.state()))
        t.pool.close()
    (before, want), (_, got) = made
    for which in ("k", "v"):
        assert np.array_equal(got[which + "s"], want[which + "s"])
        grown = want[which + "s"] > before[which + "s"]
        assert grown.any()
        differ = got[which] != want[which]
        nan = (got[which] & 0x7F) == 0x7F
        # in the source row, and where it moved to: place 1 of the first page
        assert np.array_equal(differ, nan) and nan.sum() == 2 * (2 * 2 * 2)


def test_tile_without_a_scale_among_moved_rows():
    """A row from a tile whose scale is NaN becomes NaN; the others are what they are without it."""
    for D in (64, 128):
        t = Trees("fp8_e4m3_block", 3, D, [48], [48], [[1, 17, 37]], layers=1, seed=9)
        vals = {}
        for which in ("k", "v"):
            sc = t.pool.scale_view(which)
            for page, x in enumerate((0.001, math.nan, 0.02)):
                sc[int(t.t[0, page])] = x
            codes = t.pool.layer_view(which)[int(t.t[0, 2]), :, 5].view(torch.float8_e4m3fn)
            vals[which] = (codes.double() * float(np.float32(0.02))).cpu()
        t.pool.tree_accept(**t.args)
        assert t.pool.device_error() == N.PA_OK
        for which in ("k", "v"):
            dst = int(t.t[0, 0])
            rows = t.pool.layer_view(which)[dst].view(torch.float8_e4m3fn).double().cpu()
            sc = t.pool.scale_view(which)[dst].double().cpu()
            assert bool(torch.isfinite(sc).all())
            assert rows[:, 1].isnan().all()
            got = rows[:, 2] * sc[:, None]
            # half a step of E4M3 (2^-4 of the value, or half the smallest step 2^-9 scales), and the quotient's rounding
            tol = vals[which].abs() * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10 * sc[:, None]
            assert bool(((got - vals[which]).abs() <= tol).all())
        t.pool.close()
