"""pa_decode_tree against attention written out in fp64 (tolerances: tree_reference)."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from tree_reference import Batch

pytestmark = pytest.mark.gpu

KINDS = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


SHAPES = [  # H, G, ctx, sizes, mask
    (1, 1, [1], [1], "tree"),
    (2, 2, [17, 100, 40, 1], [3, 7, 1, 1], "tree"),
    (1, 8, [16, 15, 128, 129, 500], [16, 15, 16, 5, 16], "tree"),     # histories of none, pages and blocks filled
    (3, 5, [333, 61, 700], [61, 61, 25], "holes"),                   # an odd group, rows that see nothing
    (2, 4, [0, 5, 0, 64, 1000], [0, 5, 0, 0, 9], "random"),           # sequences without nodes
    (1, 7, [1300, 256], [200, 256], "random"),                       # masks of four words, nodes over many tiles
    (8, 1, [2000, 130, 127], [64, 65, 1], "chain"),
    (2, 3, [128 * k + 3 for k in range(9)], [3] * 9, "tree"),         # trees across a block's border
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_against_fp64(kv, D, shape):
    H, G, ctx, sizes, mask = SHAPES[shape]
    b = Batch(kv, H, G, D, ctx, sizes, mask=mask, seed=shape)
    for dt in (None, torch.float32):
        out = b.run(out_dtype=dt)
        assert b.pool.device_error() == N.PA_OK
        b.check(out)
    b.pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_long_history(kv):
    """A long history beside short ones; the same bits again."""
    b = Batch(kv, 2, 8, 128, [20000, 300, 9], [16, 11, 9], seed=1)
    out = b.run()
    b.check(out)
    assert torch.equal(out, b.run())
    b.pool.close()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", KINDS)
def test_one_unit_on_every_sm(kv, D):
    """One kv head and one long sequence: as many pieces as SMs, and a tree whose nodes see little of it."""
    for ctx, sizes, G in (([20011], [37], 3), ([4100, 700], [1, 1], 8)):
        b = Batch(kv, 1, G, D, ctx, sizes, mask="random", seed=2)
        for dt in (None, torch.float32):
            b.check(b.run(out_dtype=dt))
        b.pool.close()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", KINDS)
def test_what_a_node_does_not_see(kv, D):
    """Infinities and NaN in keys and values of unseen nodes, and in slots behind the context,
    change nothing; those that a node sees do (FP8 has no infinity: NaN)."""
    b = Batch(kv, 2, 4, D, [150, 30, 290], [30, 30, 40], seed=2)
    want = b.run(out_dtype=torch.float32)
    bad = [math.inf, math.nan, -math.inf]
    hit = []
    for s, node in ((0, 7), (0, 29), (1, 0), (2, 39), (2, 20)):
        t = b.ctx[s] - b.sizes[s] + node
        blk = int(b.tables_np[s, t // 16])
        for which in ("k", "v"):
            row = b.pool.layer_view(which)[blk, :, t % 16]
            if b.pool.elem_bytes == 2:
                # (a key of NaN: its products are NaN; one of infinity may give either sign)
                row.view(b.pool.in_dtype)[:, 3] = math.nan if which == "k" else bad[node % 3]
            else:
                row[:, 3] = 0x7F
        hit.append((s, node))
    out = b.run(out_dtype=torch.float32)
    for s, m in enumerate(b.sees):
        q0 = int(b.q_start_np[s])
        for r in range(len(m)):
            seen = any(m[r, node] for hs, node in hit if hs == s)
            if seen:
                assert out[q0 + r].isnan().any()
            else:
                assert torch.equal(out[q0 + r], want[q0 + r]), (s, r)
    b.pool.close()


@pytest.mark.parametrize("kv", ["fp16", "bf16"])
def test_infinite_value_of_a_seen_node(kv):
    """An infinite value reaches the nodes that see it, and only its own dimension of them."""
    b = Batch(kv, 1, 2, 128, [140, 20], [20, 20], seed=3)
    t = b.ctx[0] - 5
    b.pool.layer_view("v")[int(b.tables_np[0, t // 16]), 0, t % 16].view(b.pool.in_dtype)[70] = -math.inf
    b.check(b.run())
    b.pool.close()


def test_padding_and_layers():
    """Rows behind the last tree are not touched; a layer of a deeper pool; a given output."""
    b = Batch("bf16", 2, 4, 128, [200, 77], [13, 20], seed=4, pad_rows=7, layers=3, layer=1, max_nodes=33)
    out = torch.full((b.T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = b.run(out=out)
    assert got.data_ptr() == out.data_ptr()
    b.check(out)
    assert bool((out[33:] == 7.0).all())
    b.pool.close()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_score_scales(kv, scale):
    b = Batch(kv, 2, 2, 128, [300, 40], [12, 40], seed=5, mask="holes", spread=0.5)
    b.check(b.run(softmax_scale=scale), scale=scale)
    b.pool.close()


def test_chain_is_prefill_and_decode():
    """A chain's rows are those of a prefill chunk, and one node is a decode."""
    b = Batch("bf16", 2, 8, 128, [1000, 57], [20, 57], mask="chain", seed=6)
    a = b.run(out_dtype=torch.float32)
    p = b.pool.prefill(b.q, b.q_start, b.tables, b.ctx_t, 57, out_dtype=torch.float32)
    assert float((a - p).abs().max()) <= 1e-4 * float(p.abs().max())
    one = Batch("fp8_e4m3", 2, 8, 128, [1000, 57, 16], [1, 1, 1], mask="tree", seed=7)
    a = one.run(out_dtype=torch.float32)
    p = one.pool.decode(one.q, one.tables, one.ctx_t, out_dtype=torch.float32)
    assert float((a - p).abs().max()) <= 1e-4 * float(p.abs().max())
    b.pool.close()
    one.pool.close()


def test_many_sequences():
    """More sequences than one schedule holds."""
    S = 4500
    b = Batch("bf16", 1, 2, 64, [3 + s % 5 for s in range(S)], [1 + s % 3 for s in range(S)], seed=8)
    b.check(b.run())
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_infinite_and_nan_queries(kv):
    """A query that holds an infinity or a NaN spoils its own row alone."""
    b = Batch(kv, 2, 4, 128, [300, 20], [9, 20], seed=13)
    want = b.run()
    b.q[2, 1, 5], b.q[11, 6, 100], b.q[12, 0, 0] = math.inf, -math.inf, math.nan
    out = b.run()
    bad = torch.zeros_like(out, dtype=torch.bool)
    for t, h in ((2, 1), (11, 6), (12, 0)):
        bad[t, h] = True
        assert out[t, h].isnan().all()
    assert torch.equal(out[~bad], want[~bad])
    b.pool.close()


def test_two_streams_at_once():
    """Two calls that may overlap, each with a workspace of its own."""
    b = Batch("fp8_e4m3", 8, 8, 128, [4000] * 6, [16] * 6, seed=14)
    c = Batch("bf16", 8, 4, 64, [3000, 1, 700], [16, 1, 30], seed=15)
    want = b.run(), c.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = b.run(stream=s1), c.run(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
    c.pool.close()


@pytest.mark.parametrize("off", [0, 8, 16])
def test_output_alignment(off):
    """An output that starts on 16 bytes but not on 32."""
    b = Batch("bf16", 2, 4, 128, [2000, 300], [16, 30], seed=16)
    want = b.run(), b.run(out_dtype=torch.float32)
    for w in want:
        n = off * 2 // w.element_size()
        buf = torch.zeros(w.numel() + n, dtype=w.dtype, device="cuda")
        out = buf[n:].view(w.shape)
        b.run(out=out)
        assert torch.equal(out, w)
    b.pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_lost_tiles(kv):
    """A page of NaN in the history reaches every node; in block-scaled pools, a scale of NaN or infinity
    reaches exactly the nodes that see a token of its tile."""
    b = Batch(kv, 2, 4, 128, [200, 70], [30, 40], seed=17)
    want = b.run()
    if b.pool.block_scaled:
        for which, s, page, val in (("k", 0, 12, math.nan), ("v", 1, 3, math.inf)):
            b.pool.scale_view(which)[int(b.tables_np[s, page]), 1] = val
        out = b.run()
        for s, page in ((0, 12), (1, 3)):
            base = b.ctx[s] - b.sizes[s]
            for r in range(b.sizes[s]):
                row = int(b.q_start_np[s]) + r
                seen = any(t < base or b.sees[s][r, t - base] for t in range(16 * page, min(16 * page + 16, b.ctx[s])))
                assert out[row, 4:].isnan().all() if seen else torch.equal(out[row], want[row]), (s, r)
                assert torch.equal(out[row, :4], want[row, :4])  # the other kv head
    else:
        b.pool.layer_view("v")[int(b.tables_np[0, 2]), 1] = 0x7F if b.pool.elem_bytes == 1 else 0xFF
        out = b.run()
        assert out[:30, 4:].isnan().all()
        assert torch.equal(out[:30, :4], want[:30, :4]) and torch.equal(out[30:], want[30:])
    b.pool.close()


@pytest.mark.parametrize("up", [True, False])
def test_tile_scales_far_apart(up):
    """Block-scaled tiles of V whose scales differ by more than 16-bit weights hold, zeros and subnormal
    ones among them, the largest at the end or at the start of the history."""
    b = Batch("fp8_e4m3_block", 2, 3, 128, [900, 330, 150], [9, 20, 5], seed=23)
    steps = [0.0, 2.0 ** -140, 2.0 ** -100, 2.0 ** -75, 2.0 ** -63, 2.0 ** -40, 2.0 ** -20, 2.0 ** -9, 1.0]
    sc = b.pool.scale_view("v")
    for s, n in enumerate(b.ctx):
        last = (n - b.sizes[s]) // 16 - 1  # the last page of history alone
        for page in range(last + 1):
            i = page if up else last - page
            sc[int(b.tables_np[s, page])] = 0.01 * steps[i * len(steps) // (last + 1)]
    b.check(b.run())
    b.check(b.run(out_dtype=torch.float32))
    b.pool.close()


def _bad(b, **kw):
    out = torch.full((b.T, b.H * b.G, b.D), 7.0, dtype=b.pool.in_dtype, device="cuda")
    a = dict(q_start=b.q_start, tables=b.tables, ctx=b.ctx_t, max_nodes=b.max_nodes, mask=b.mask)
    a.update(kw)
    b.pool.decode_tree(b.q, a["q_start"], a["tables"], a["ctx"], a["max_nodes"], mask=a["mask"], out=out)
    assert b.pool.device_error() == N.PA_ERR_BOUNDS
    return out


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_bad_sequences_are_skipped(kv):
    """A sequence whose lengths do not fit is reported and skipped; the others are computed.
    (A batch of other lengths is cut into other pieces, whose fp32 sums are joined in another
    order: the rows are held to fp64, not to the bits of the whole batch's call.)"""
    b = Batch(kv, 2, 4, 128, [200, 77, 300], [13, 20, 5], seed=9, mask="chain")
    b.check(b.run())
    y, tol = b.exact()
    near = lambda got, r: bool(((got[r].double() - y[r]).abs() <= tol[r]).all())  # noqa: E731
    assert b.pool.device_error() == N.PA_OK
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = [slice(0, 13), slice(13, 33), slice(33, 38)]
    width = b.tables.shape[1]
    for kw, skipped in (
            (dict(ctx=torch.tensor([200, 19, 300], **i32)), [1]),                 # shorter than its nodes
            (dict(ctx=torch.tensor([200, -4, 300], **i32)), [1]),
            (dict(ctx=torch.tensor([200, 77, 16 * width + 1], **i32)), [2]),      # longer than its table
            (dict(max_nodes=13), [1]),                                            # more nodes than announced
            (dict(q_start=torch.tensor([0, 13, 33, 39], **i32)), [2]),            # behind the rows
            (dict(q_start=torch.tensor([-3, 13, 33, 38], **i32)), [0]),
            (dict(q_start=torch.tensor([0, 13, 33, 20], **i32)), [2])):           # decreasing
        out = _bad(b, **kw)
        for s in range(3):
            if s in skipped:
                assert bool((out[rows[s]] == 7.0).all()), (kw, s)
            else:
                assert near(out, rows[s]), (kw, s)
    # a page outside the pool: reported, and the other sequences hold
    for page in (-1, b.pool.num_blocks, 2 ** 31 - 1):
        t = b.tables.clone()
        t[1, 2] = page
        out = _bad(b, tables=t)
        assert near(out, rows[0]) and near(out, rows[2])
    b.pool.close()


def test_streams_and_graphs():
    """A side stream; two captured graphs with workspaces of their own, replayed on new inputs."""
    b = Batch("bf16", 2, 4, 128, [2000, 77, 300], [13, 20, 5], seed=10)
    c = Batch("fp8_e4m3", 2, 8, 128, [1500, 20], [16, 3], seed=11)
    want_b, want_c = b.run(), c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want_b)
    graphs, outs = [], []
    keep = b.q.clone()
    for x in (b, c):
        ws = torch.empty(x.pool.tree_workspace_bytes(x.H * x.G, x.max_nodes), dtype=torch.uint8, device="cuda")
        out = torch.zeros(x.T, x.H * x.G, x.D, dtype=x.pool.in_dtype, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(out=out, workspace=ws)
        graphs.append((g, ws))
        outs.append(out)
    b.q.zero_()
    for _ in range(3):
        for g, _ws in graphs:
            g.replay()
    torch.cuda.synchronize()
    b.check(outs[0])
    assert torch.equal(outs[1], want_c)
    b.q.copy_(keep)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want_b)
    assert b.pool.device_error() == N.PA_OK
    b.pool.close()
    c.pool.close()


def test_wrapper_refusals():
    b = Batch("bf16", 2, 4, 128, [200, 77], [13, 20], seed=12)
    p = b.pool
    ok = dict(q=b.q, q_start=b.q_start, block_tables=b.tables, ctx_lens=b.ctx_t, max_nodes=20, mask=b.mask)
    for bad in (dict(q=b.q.half()), dict(q=b.q[0]), dict(q=b.q[..., :64]), dict(q=b.q.transpose(0, 1)), dict(q=b.q.cpu()),
                dict(q_start=b.q_start[:2]), dict(q_start=b.q_start.long()), dict(block_tables=b.tables[:1]),
                dict(ctx_lens=b.ctx_t[:1]), dict(mask=b.mask[:5]), dict(mask=b.mask.int()), dict(max_nodes=65),
                dict(out=b.q[:3]), dict(out=b.q.double()), dict(workspace=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises((TypeError, ValueError)):
            p.decode_tree(**{**ok, **bad})
    for bad in (dict(max_nodes=0, mask=None), dict(max_nodes=257, mask=None), dict(softmax_scale=math.nan), dict(layer=1),
                dict(out=b.q.half()), dict(q=b.q[:, :3].contiguous())):
        with pytest.raises(N.PAError):
            p.decode_tree(**{**ok, **bad})
    assert p.decode_tree(b.q[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), b.tables[:0], b.ctx_t[:0], 4).shape[0] == 0
    p.close()
