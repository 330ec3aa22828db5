"""pa_tree_accept: bytes moved in place, and scales per tile, bit for bit against numpy."""
import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N
from tree_reference import make_pool

pytestmark = pytest.mark.gpu

KINDS = ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"]
E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def _codes(x):
    return torch.from_numpy(x.clip(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


class Trees:
    def __init__(self, kv, H, D, ctx, sizes, paths, layers=2, max_path=None, seed=0):
        rng = np.random.default_rng(seed)
        self.kv, self.H, self.D, self.layers = kv, H, D, layers
        S = len(ctx)
        pages = [-(-n // 16) for n in ctx]
        self.pool = make_pool(kv, H, D, sum(pages) + 3, layers)
        for buf in (self.pool.k_cache, self.pool.v_cache):
            n = layers * self.pool.layer_bytes
            x = rng.standard_normal(n // self.pool.elem_bytes).astype(np.float32)
            if self.pool.elem_bytes == 2:
                buf[:n] = torch.from_numpy(x).to(self.pool.in_dtype).view(torch.uint8).cuda()
            else:
                buf[:n] = torch.from_numpy(x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        if self.pool.block_scaled:
            for which in ("k", "v"):
                for layer in range(layers):
                    sc = self.pool.scale_view(which, layer)
                    sc.copy_(torch.from_numpy(np.exp(rng.normal(-4, 1.5, tuple(sc.shape))).astype(np.float32)))
                    sc[0] = 0.0  # a tile of zeros
        ids = rng.permutation(self.pool.num_blocks)
        t = np.full((S, max(pages + [1]) + 1), -1, np.int32)
        at = 0
        for s, k in enumerate(pages):
            t[s, :k] = ids[at:at + k]
            at += k
        self.t = t
        self.ctx, self.sizes, self.paths = ctx, sizes, paths
        P = max_path or max([len(p) for p in paths] + [1])
        pt = np.full((S, P), -7, np.int32)
        for s, p in enumerate(paths):
            pt[s, :len(p)] = p
        qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.args = dict(paths=torch.from_numpy(pt).cuda(), path_lens=torch.tensor([len(p) for p in paths], **i32),
                         q_start=torch.from_numpy(qs).cuda(), block_tables=torch.from_numpy(t).cuda(),
                         ctx_lens=torch.tensor(ctx, **i32))

    def state(self):
        """Copies of the codes or elements [layers, blocks, H, 16, row] and scales of K and V."""
        out = {}
        for which in ("k", "v"):
            out[which] = np.stack([self.pool.layer_view(which, i).cpu().numpy() for i in range(self.layers)])
            if self.pool.block_scaled:
                out[which + "s"] = np.stack([self.pool.scale_view(which, i).cpu().numpy() for i in range(self.layers)])
        return out

    def expected(self, st, layer=0, n_layers=None, skip=()):
        new = {k: v.copy() for k, v in st.items()}
        for L in range(layer, layer + (n_layers or self.layers - layer)):
            for s, path in enumerate(self.paths):
                if s in skip:
                    continue
                base = self.ctx[s] - self.sizes[s]
                where = lambda t: (self.t[s, t // 16], t % 16)  # noqa: E731
                for which in ("k", "v"):
                    if not self.pool.block_scaled:
                        for i, node in enumerate(path):
                            (sb, so), (db, do) = where(base + node), where(base + i)
                            new[which][L, db, :, do] = st[which][L, sb, :, so]
                    else:
                        self._block(st, new, which, L, base, path, where)
        return new

    def _block(self, st, new, which, L, base, path, where):
        old_c, old_s = st[which][L], st[which + "s"][L]
        for t0 in range(base // 16 * 16, base + len(path), 16):
            rows = [(i, n) for i, n in enumerate(path) if t0 <= base + i < t0 + 16 and i != n]
            if not rows:
                continue
            db = where(t0)[0]
            for h in range(self.H):
                s_old = old_s[db, h]
                x = {}
                run = np.float32(0)
                for i, n in rows:
                    sb, so = where(base + n)
                    x[i] = E4M3[old_c[sb, h, so]] * old_s[sb, h]
                    if sb != db:
                        run = max(run, np.float32(np.abs(x[i]).max() / np.float32(448)))
                s = run if run > s_old else s_old
                if run > s_old:
                    new[which][L, db, h] = _codes(E4M3[old_c[db, h]] * s_old / s)
                    new[which + "s"][L, db, h] = s
                for i, n in rows:
                    new[which][L, db, h, (base + i) % 16] = _codes(x[i] / s if s > 0 else np.zeros(self.D, np.float32))

    def check(self, new):
        got = self.state()
        for k in new:
            assert np.array_equal(got[k].view(np.uint8 if got[k].dtype == np.uint8 else np.uint32),
                                  new[k].view(np.uint8 if new[k].dtype == np.uint8 else np.uint32)), k


CASES = [  # H, D, ctx, sizes, paths, layers
    (1, 128, [1], [1], [[0]], 1),
    (8, 128, [40, 17, 100], [16, 16, 16], [[0, 2, 5, 9, 15], [], [15]], 2),
    (3, 64, [61, 70, 33, 0, 9], [61, 25, 1, 0, 0], [[1, 2, 3, 30, 60], list(range(25)), [0], [], []], 3),
    (2, 128, [300, 256], [256, 256], [sorted(np.random.default_rng(0).permutation(256)[:100].tolist()), list(range(1, 256))], 1),
    (12, 64, [50, 51], [40, 41], [[0, 1, 2, 20, 21, 39], list(range(8, 41))], 2),
]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_numpy(kv, case):
    H, D, ctx, sizes, paths, layers = CASES[case]
    t = Trees(kv, H, D, ctx, sizes, paths, layers, seed=case)
    before = t.state()
    lens = t.pool.tree_accept(**t.args)
    assert t.pool.device_error() == N.PA_OK
    assert lens.tolist() == [c - n + len(p) for c, n, p in zip(ctx, sizes, paths)]
    t.check(t.expected(before))
    t.pool.close()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("S,H,D,layers", [(310, 8, 64, 5), (90, 3, 128, 37), (700, 1, 64, 9)])
def test_many_pairs(kv, S, H, D, layers):
    """More (sequence, layer, kv head) pairs than the GPU has warps: several to a warp, paths of
    no move, of one, and of more rows than a warp has lanes."""
    rng = np.random.default_rng(S)
    sizes = [int(rng.integers(60, 100)) if s % 45 == 7 else int(rng.integers(0, 17)) for s in range(S)]
    ctx = [n + int(rng.integers(0, 40)) for n in sizes]
    paths = [sorted(rng.permutation(n)[:int(rng.integers(0, n + 1))].tolist()) for n in sizes]
    t = Trees(kv, H, D, ctx, sizes, paths, layers, seed=S)
    before = t.state()
    lens = t.pool.tree_accept(**t.args)
    assert t.pool.device_error() == N.PA_OK
    assert lens.tolist() == [c - n + len(p) for c, n, p in zip(ctx, sizes, paths)]
    t.check(t.expected(before))
    t.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block"])
def test_some_layers(kv):
    t = Trees(kv, 2, 128, [50], [30], [[3, 7, 20]], layers=4)
    before = t.state()
    t.pool.tree_accept(**t.args, layer=1, n_layers=2)
    t.check(t.expected(before, 1, 2))
    t.pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_bad_paths_move_nothing(kv):
    """A path that does not fit its tree is reported; its sequence stays, the other one moves."""
    i32 = dict(dtype=torch.int32, device="cuda")
    for what, bad in (("down", [4, 3]), ("twice", [5, 5]), ("past", [2, 16]), ("negative", [-1, 3]), ("long", [1, 2, 3])):
        t = Trees(kv, 2, 128, [40, 40], [16, 16], [[1, 5], [2, 9]], seed=3, max_path=3)
        t.args["paths"][0, :len(bad)] = torch.tensor(bad, **i32)
        if what == "long":
            t.args["path_lens"][0] = 4
        before = t.state()
        lens = t.pool.tree_accept(**t.args)
        assert t.pool.device_error() == N.PA_ERR_BOUNDS, what
        assert lens.tolist() == [40, 26]
        t.check(t.expected(before, skip=(0,)))
        t.pool.close()
    for change in (dict(ctx_lens=[15, 40]), dict(ctx_lens=[16 * 5 + 1, 40]), dict(q_start=[17, 16, 32]), dict(q_start=[-1, 16, 32])):
        t = Trees(kv, 2, 128, [40, 40], [16, 16], [[1, 5], [2, 9]], seed=3)
        before = t.state()
        t.pool.tree_accept(**{**t.args, **{k: torch.tensor(v, **i32) for k, v in change.items()}})
        assert t.pool.device_error() == N.PA_ERR_BOUNDS, change
        t.check(t.expected(before, skip=(0,)))
        t.pool.close()


@pytest.mark.parametrize("kv", KINDS)
def test_bad_pages(kv):
    """Rows in a page that is none are skipped and reported."""
    t = Trees(kv, 2, 128, [40], [40], [[3, 33]], seed=4, layers=1)
    t.args["block_tables"][0, 2] = t.pool.num_blocks  # node 33's page
    before = t.state()
    t.pool.tree_accept(**t.args)
    assert t.pool.device_error() == N.PA_ERR_BOUNDS
    t.paths = [[3, 1]]  # place 1 stays as it is
    t.check(t.expected(before))
    t.pool.close()


def test_graph_replay_and_stream():
    t = Trees("bf16", 2, 128, [40, 100], [16, 16], [[0, 5], [2, 9]], seed=5)
    before = t.state()
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.pool.tree_accept(**t.args, new_lens=out)
    t.check(before)
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    t.check(t.expected(before))
    assert out.tolist() == [26, 86]
    t.pool.close()


def test_refusals():
    t = Trees("bf16", 2, 128, [40, 100], [16, 16], [[0, 5], [2, 9]], seed=6)
    a = t.args
    for bad in (dict(paths=a["paths"].long()), dict(paths=a["paths"][:1]), dict(path_lens=a["path_lens"][:1]),
                dict(q_start=a["q_start"][:2]), dict(block_tables=a["block_tables"][0]), dict(ctx_lens=a["ctx_lens"].cpu()),
                dict(new_lens=a["ctx_lens"][:1])):
        with pytest.raises((TypeError, ValueError)):
            t.pool.tree_accept(**{**a, **bad})
    for bad in (dict(new_lens=a["ctx_lens"]), dict(layer=2), dict(layer=1, n_layers=2), dict(n_layers=0),
                dict(paths=torch.zeros(2, 257, dtype=torch.int32, device="cuda"))):
        with pytest.raises(N.PAError):
            t.pool.tree_accept(**{**a, **bad})
    t.pool.close()
