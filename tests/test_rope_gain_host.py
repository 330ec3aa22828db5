"""The gain that make_rope takes for a "yarn" embedding when none is given."""
import math

import numpy as np
import pytest

N = pytest.importorskip("paged_kv_cache_270_gb300._native")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()


@pytest.mark.parametrize("factor, gain", [
    (0.25, 1.0), (0.5, 1.0), (1.0, 1.0), (1.5, 0.1 * math.log(1.5) + 1), (16.0, 0.1 * math.log(16.0) + 1)])
def test_default_gain(factor, gain):
    """0.1 ln(factor) + 1 where the context is stretched, one where it is not."""
    from paged_kv_cache_270_gb300.pool import make_rope
    assert make_rope(64, scaling="yarn", factor=factor).gain == np.float32(gain)
    assert make_rope(64, scaling="yarn", factor=factor, gain=0.75).gain == 0.75
    assert make_rope(64, scaling="linear", factor=factor).gain == 1.0


def test_a_factor_that_is_none():
    from paged_kv_cache_270_gb300.pool import make_rope
    for factor in (0.0, -2.0, math.nan):
        with pytest.raises(N.PAError) as e:
            make_rope(64, scaling="yarn", factor=factor)
        assert e.value.code == N.PA_ERR_INVALID
