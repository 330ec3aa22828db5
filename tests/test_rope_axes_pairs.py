"""norm_rope_and_cache refuses axes whose sections are not the embedding's pairs (CPU: the call ends before the library)."""
import copy

import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from paged_kv_cache_270_gb300 import build
from paged_kv_cache_270_gb300 import pool as P


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _pool(launched):
    """A pool without memory, whose launches are noted."""
    p = object.__new__(P.KVPool)
    p.device, p.in_dtype, p.handle = torch.device("cpu"), torch.bfloat16, None
    p.n_kv_heads, p.head_dim = 2, 128
    p._launch = lambda call, args, stream: launched.append(args)
    return p


def _call(p, rope, axes, n_axes):
    x = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    pos = torch.zeros(n_axes, 3, dtype=torch.int32)
    return p.norm_rope_and_cache(rope, x[:, :4], x[:, 4:6], x[:, 6:], pos, torch.zeros(3, dtype=torch.int64), axes=axes,
                                 q_out=torch.zeros(3, 4, 128, dtype=torch.bfloat16))


@pytest.mark.parametrize("order", ["sections", "turns"])
def test_sections_must_be_the_embeddings_pairs(order):
    launched = []
    p = _pool(launched)
    rope = P.make_rope(128)
    for sections in ([12, 10, 10], [32, 16, 15], [10, 10, 10], [1]):
        for axes in (P.make_rope_axes(sections, order), copy.copy(P.make_rope_axes(sections, order))):
            with pytest.raises(ValueError, match="pairs"):
                _call(p, rope, axes, len(sections))
    with pytest.raises(ValueError, match="pairs"):  # surplus sections
        _call(p, P.make_rope(64), P.make_rope_axes([24, 20, 20], order), 3)
    assert not launched
    _call(p, rope, P.make_rope_axes([24, 20, 20], order), 3)
    _call(p, P.make_rope(64), P.make_rope_axes([12, 10, 10], order), 3)
    assert len(launched) == 2


def test_axes_filled_by_hand_name_every_pair():
    launched = []
    axes = N.pa_rope_axes(2)
    axes.axis[63] = 1
    _call(_pool(launched), P.make_rope(128), axes, 2)
    _call(_pool(launched), P.make_rope(64), axes, 2)
    assert len(launched) == 2


def test_no_embedding_is_left_to_the_library():
    """A missing embedding reaches the library, which refuses it with its own error."""
    launched = []
    _call(_pool(launched), None, P.make_rope_axes([24, 20, 20]), 3)
    assert len(launched) == 1
