"""Speculative decoding as a user runs it: drafts written with norms and rotary positions, checked as a tree in
every layer, the accepted path kept, and the next step on top of it, against the same tokens one by one.

Tolerances.  Cached rows of 16-bit and FP8 pools are the same bytes.  Outputs in fp32 differ by the order of
their sums and by FP8 pools' split of the queries: 1e-4 of a row's largest value, as for every fp32 output.
In block-scaled pools a tile's codes depend on the order in which its rows came (a code is rounded
again when its tile's scale grows): each rounding is 2^-4 of a value, so two of them, in keys and in values, may move
a weight by that share of its score and a value by 2^-3 of itself; held to 0.25 of a row's largest value."""
import numpy as np
import pytest
import torch

from paged_kv_cache_270_gb300 import _native as N

pytestmark = pytest.mark.gpu

H, G, D, LAYERS, VOCAB = 2, 4, 128, 2, 50


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


class Model:
    """Layers whose queries, keys and values are looked up by token id."""

    def __init__(self, kv, blocks, seed=0):
        from paged_kv_cache_270_gb300.pool import KVPool, make_rope, make_rope_axes
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = KVPool(LAYERS, blocks, H, D, kv, 0.02, 0.02)
        for buf in (self.pool.k_cache, self.pool.v_cache):
            buf.fill_(0xFF)
        dt = self.pool.in_dtype
        self.table = [torch.randn(VOCAB, H * G + 2 * H, D, device="cuda", generator=g).to(dt) for _ in range(LAYERS)]
        self.qw, self.kw = ((torch.rand(D, device="cuda", generator=g) + 0.5).to(dt) for _ in range(2))
        self.rope, self.axes = make_rope(D, theta=1e6), make_rope_axes([16, 24, 24])

    def write(self, layer, tokens, positions, slots):
        x = self.table[layer][torch.tensor(tokens, device="cuda")]
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda").expand(3, -1).contiguous()
        return self.pool.norm_rope_and_cache(self.rope, x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:], pos,
                                             torch.tensor(slots, device="cuda"), q_weight=self.qw, k_weight=self.kw,
                                             axes=self.axes, layer=layer)


def _close(a, b, rel):
    assert torch.isfinite(a).all()
    worst = ((a - b).abs().amax(-1) / b.abs().amax(-1)).max()
    assert float(worst) <= rel, float(worst)


@pytest.mark.parametrize("kv", ["fp16", "bf16", "fp8_e4m3", "fp8_e4m3_block"])
def test_tree_then_accept_equals_one_by_one(kv):
    rng = np.random.default_rng(3)
    hist = [37, 130, 5]
    sizes = [13, 24, 9]
    S, steps = 3, 3
    spec, plain = Model(kv, 40), Model(kv, 40)
    tables = {m: torch.from_numpy(np.stack([m.pool.alloc(12) for _ in range(S)])) for m in (spec, plain)}
    i32 = dict(dtype=torch.int32, device="cuda")
    slot = lambda m, s, t: [int(tables[m][s, x // 16]) * 16 + x % 16 for x in t]  # noqa: E731
    for m in (spec, plain):
        for layer in range(LAYERS):
            r = np.random.default_rng(1)
            for s, n in enumerate(hist):
                m.write(layer, r.integers(0, VOCAB, n).tolist(), list(range(n)), slot(m, s, range(n)))
    dev = {m: tables[m].cuda() for m in (spec, plain)}
    ctx = list(hist)
    rel = 0.25 if kv == "fp8_e4m3_block" else 1e-4
    for step in range(steps):
        # the trees: tokens, parents, who sees whom
        toks = [rng.integers(0, VOCAB, n).tolist() for n in sizes]
        sees, depth, paths = [], [], []
        for n in sizes:
            m = np.zeros((n, n), bool)
            dep = [0] * n
            for i in range(n):
                parent = int(rng.integers(max(-1, i - 4), i)) if i else -1
                if parent >= 0:
                    m[i] = m[parent]
                    dep[i] = dep[parent] + 1
                m[i, i] = True
            sees.append(m)
            depth.append(dep)
            leaf = int(rng.integers(0, n))
            paths.append(np.flatnonzero(m[leaf]).tolist())
        if step == 1:
            paths[2] = []  # nothing accepted
        q_start = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), **i32)
        mask = torch.tensor([int(sum(1 << j for j in np.flatnonzero(row))) for m in sees for row in m], dtype=torch.int64, device="cuda")[:, None]
        with_drafts = torch.tensor([c + n for c, n in zip(ctx, sizes)], **i32)
        outs = []
        for layer in range(LAYERS):
            q = spec.write(layer, sum(toks, []), [c + d for c, dep in zip(ctx, depth) for d in dep],
                           sum((slot(spec, s, range(ctx[s], ctx[s] + sizes[s])) for s in range(S)), []))
            outs.append(spec.pool.decode_tree(q, q_start, dev[spec], with_drafts, max(sizes), mask=mask, out_dtype=torch.float32, layer=layer))
        P = max(len(p) for p in paths) or 1
        pt = torch.full((S, P), -1, **i32)
        for s, p in enumerate(paths):
            pt[s, :len(p)] = torch.tensor(p, **i32)
        lens = spec.pool.tree_accept(pt, torch.tensor([len(p) for p in paths], **i32), q_start, dev[spec], with_drafts)
        assert lens.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
        assert spec.pool.device_error() == N.PA_OK
        # the accepted tokens one by one
        for i in range(P):
            live = [s for s in range(S) if i < len(paths[s])]
            for layer in range(LAYERS):
                q = plain.write(layer, [toks[s][paths[s][i]] for s in live], [ctx[s] + i for s in live],
                                sum((slot(plain, s, [ctx[s] + i]) for s in live), []))
                one = plain.pool.decode(q, dev[plain][live].contiguous(), torch.tensor([ctx[s] + i + 1 for s in live], **i32),
                                        out_dtype=torch.float32, layer=layer)
                tree = outs[layer][[int(q_start[s]) + paths[s][i] for s in live]]
                _close(tree, one, rel)
        ctx = lens.tolist()
    # the kept rows are those of the plain cache
    if kv != "fp8_e4m3_block":
        for which in ("k", "v"):
            for layer in range(LAYERS):
                a, b = spec.pool.layer_view(which, layer), plain.pool.layer_view(which, layer)
                for s in range(S):
                    t = torch.arange(ctx[s])
                    rows = [v[m.to("cuda").long()[s, t // 16], :, t % 16] for v, m in ((a, tables[spec]), (b, tables[plain]))]
                    assert torch.equal(*rows)
    spec.pool.close()
    plain.pool.close()
