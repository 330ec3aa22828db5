"""Attention of drafted trees, and a pool to run it on, written out in fp64.

Tolerance of an output element with weights p and values v over n tokens, from what
the kernels may do:
  * a score is an fp32 sum of head_dim products.  Tensor cores may truncate where they
    add, so a step counts 2^-23 of the products' absolute sum: 2 D 2^-24.  FP8 pools take a
    query as two E4M3 terms, of which the second has a step of 2^-9 under a row maximum
    of at least 128: 2^-17 of the largest |q| for each key element.
  * a weight then has a relative error of twice its score's (its own and the sum's), ex2's
    2^-22, and its rounding for the product with V: 2^-12 where that is binary16
    alone (FP8 pools, 16-bit output), 2^-17 with a second bfloat16 term, 2^-22 with a
    second binary16 term; twice, for the sums' shares.  A binary16 weight keeps at least a step of 2^-25
    of 2^7, the largest weight.
  * the sums over n tokens add (n / 16 + 32) 2^-23 of the absolute sum, p |v|.
  * the result is rounded once to the output type: eps / 2 of it (and half a binary16 step)."""
from __future__ import annotations

import math

import numpy as np
import torch

K_SCALE, V_SCALE = 0.0125, 0.015


def make_pool(kv, H, D, blocks, layers=1, fill=0xFF):
    from paged_kv_cache_270_gb300.pool import KVPool
    p = KVPool(layers, blocks, H, D, kv, K_SCALE, V_SCALE)
    p.k_cache.fill_(fill)
    p.v_cache.fill_(fill)
    return p


def values(pool, which, layer=0):
    """A layer's values in fp64, [blocks, H, 16, D]."""
    raw = pool.layer_view(which, layer).contiguous()
    if pool.elem_bytes == 2:
        return raw.view(pool.in_dtype).double()
    x = raw.view(torch.float8_e4m3fn).double()
    if pool.block_scaled:
        return x * pool.scale_view(which, layer).double()[:, :, None, None]
    return x * float(np.float32(K_SCALE if which == "k" else V_SCALE))


class Batch:
    """Sequences with `ctx[s]` tokens, the last `sizes[s]` of them nodes of a tree."""

    def __init__(self, kv, H, G, D, ctx, sizes, max_nodes=None, mask="tree", seed=0, pad_rows=0, spread=1.0,
                 layers=1, layer=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.H, self.G, self.D, self.layer = H, G, D, layer
        self.ctx, self.sizes = list(ctx), list(sizes)
        S = len(self.ctx)
        self.max_nodes = max_nodes or max(self.sizes + [1])
        pages = [-(-n // 16) for n in self.ctx]
        width = max(pages + [1]) + 1
        self.pool = make_pool(kv, H, D, sum(pages) + 2, layers)
        ids = rng.permutation(self.pool.num_blocks)
        t = np.full((S, width), -1, np.int32)
        at = 0
        for s, k in enumerate(pages):
            t[s, :k] = ids[at:at + k]
            at += k
        dt = self.pool.in_dtype
        for s, n in enumerate(self.ctx):
            if n == 0:
                continue
            i = np.arange(n)
            slots = torch.from_numpy(t[s, i // 16].astype(np.int64) * 16 + i % 16).cuda()
            k, v = (torch.randn(n, H, D, device="cuda", generator=g).mul_(spread).to(dt) for _ in range(2))
            self.pool.reshape_and_cache(k, v, slots, layer=layer)
        self.tables_np, self.tables = t, torch.from_numpy(t).cuda()
        self.ctx_t = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        qs = np.concatenate([[0], np.cumsum(self.sizes)]).astype(np.int32)
        self.q_start_np, self.q_start = qs, torch.from_numpy(qs).cuda()
        self.T = int(qs[-1]) + pad_rows
        self.q = torch.randn(self.T, H * G, D, device="cuda", generator=g).mul_(1.5).to(dt)
        self.sees = [self._sees(n, mask, rng) for n in self.sizes]
        self.mask = None if mask == "chain" else self._pack()

    def _sees(self, n, kind, rng):
        m = np.zeros((n, n), bool)
        for i in range(n):
            if kind == "chain":
                m[i, :i + 1] = True
            elif kind == "random":
                m[i] = rng.random(n) < 0.4  # (not a tree: any mask)
            else:
                parent = i - int(rng.integers(1, 6))
                if parent >= 0:
                    m[i] = m[parent]
                m[i, i] = True
        if kind == "holes":
            m[rng.random(n) < 0.3] = False
        return m

    def _pack(self):
        words = -(-self.max_nodes // 64)
        bits = np.zeros((self.T, words * 64), np.uint64)
        for s, m in enumerate(self.sees):
            q0 = int(self.q_start_np[s])
            bits[q0:q0 + len(m), :len(m)] = m
            bits[q0:q0 + len(m), len(m):] = 1  # bits behind the nodes count for nothing
        w = (bits.reshape(self.T, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
        return torch.from_numpy(w.view(np.int64)).cuda()

    def run(self, **kw):
        kw.setdefault("layer", self.layer)
        return self.pool.decode_tree(self.q, self.q_start, self.tables, self.ctx_t, self.max_nodes, mask=self.mask, **kw)

    def exact(self, out_dtype=None, scale=None):
        """The results in fp64 [T, Hq, D] (NaN in padding rows) and their tolerances."""
        pool, H, G, D = self.pool, self.H, self.G, self.D
        out_dtype = out_dtype or pool.in_dtype
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        k_all, v_all = values(pool, "k", self.layer), values(pool, "v", self.layer)
        f8 = pool.elem_bytes == 1
        if f8 and out_dtype != torch.float32:
            dp = 2.0 ** -12
        else:
            dp = 2.0 ** -17 if pool.in_dtype == torch.bfloat16 and not f8 else 2.0 ** -22
        y = torch.full((self.T, H * G, D), math.nan, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(y)
        for s, n in enumerate(self.ctx):
            size, q0 = self.sizes[s], int(self.q_start_np[s])
            if size == 0:
                continue
            i = np.arange(n)
            blk = torch.from_numpy(self.tables_np[s, i // 16].astype(np.int64)).cuda()
            off = torch.from_numpy(i % 16).cuda()
            k, v = k_all[blk, :, off], v_all[blk, :, off]  # [n, H, D]
            for r in range(size):
                vis = np.concatenate([np.arange(n - size), n - size + np.flatnonzero(self.sees[s][r])])
                if len(vis) == 0:
                    y[q0 + r] = 0.0
                    continue
                vi = torch.from_numpy(vis).cuda()
                q = self.q[q0 + r].double().view(H, G, D)
                kk, vv = k[vi], v[vi]  # [m, H, D]
                z = torch.einsum("hgd,mhd->hgm", q, kk) * scale
                ez = torch.einsum("hgd,mhd->hgm", q.abs(), kk.abs()) * abs(scale) * 2 * D * 2.0 ** -24
                if f8:
                    ez = ez + q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).T[:, None, :] * abs(scale) * 2.0 ** -17
                p = torch.softmax(z, -1)
                o = torch.einsum("hgm,mhd->hgd", p, vv)
                a = torch.einsum("hgm,mhd->hgd", p, vv.abs())
                worst = ez.amax(-1, keepdim=True)
                rel = 4 * worst + 2 * dp + 2.0 ** -20 + (len(vis) / 16 + 32) * 2.0 ** -23
                small = 2.0 ** -31 * vv.abs().sum(0)[:, None, :] if f8 or pool.in_dtype == torch.float16 else 0.0
                e = rel * a + small
                y[q0 + r] = o.reshape(H * G, D)
                fin = torch.finfo(out_dtype)
                tiny = 2.0 ** -25 if out_dtype == torch.float16 else 0.0
                tol[q0 + r] = (e + fin.eps / 2 * (o.abs() + e) + tiny).reshape(H * G, D)
        return y, tol

    def check(self, out, scale=None):
        y, tol = self.exact(out.dtype, scale)
        live = int(self.q_start_np[-1])
        got = out[:live].double()
        y, tol = y[:live], tol[:live]
        assert torch.equal(got.isnan(), y.isnan()), "NaN in other places"
        inf = y.isinf()
        assert torch.equal(got[inf], y[inf])
        fine = ~(y.isnan() | inf)
        over = ((got - y).abs() - tol)[fine]
        assert over.numel() == 0 or float(over.max()) <= 0, f"off by {float(over.max()):.3e} over the tolerance"
