"""PyTorch-facing wrapper of the C ABI: device memory and streams come from
PyTorch, every computation from the library's CUDA kernels.

``KVPool`` owns the two device regions of a pool (as uint8 tensors) and the
library's pool handle, and forwards each call to the C entry point of the same
name with the tensors' device pointers and the current CUDA stream.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import _native as N

KV_DTYPES = {"fp16": N.PA_FP16, "bf16": N.PA_BF16, "fp8_e4m3": N.PA_FP8_E4M3,
             "fp8_e4m3_block": N.PA_FP8_E4M3_BLOCK}
_TORCH_OUT = {N.PA_FP16: torch.float16, N.PA_BF16: torch.bfloat16, N.PA_FP32: torch.float32}


_OUT_CODES = {v: k for k, v in _TORCH_OUT.items()}


def _stream_handle(stream=None) -> int:
    if stream is None:  # the current device's current stream, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream)


def _all_need(device, *tensors) -> None:
    """_need of several (tensor, name, dtype), quick where all is well."""
    for t, name, dtype in tensors:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()):
            _need(t, name, dtype, device)


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


ROPE_LAYOUTS = {"half": N.PA_ROPE_HALF, "interleaved": N.PA_ROPE_INTERLEAVED}
ROPE_SCALINGS = {"none": N.PA_ROPE_SCALE_NONE, "linear": N.PA_ROPE_SCALE_LINEAR,
                 "ntk": N.PA_ROPE_SCALE_NTK, "bands": N.PA_ROPE_SCALE_BANDS,
                 "yarn": N.PA_ROPE_SCALE_YARN}


def make_rope(rot_dim: int, layout: str = "half", theta: float = 10000.0, scaling: str = "none",
              factor: float = 1.0, original_len: float = 8192.0, low: float = 1.0,
              high: float | None = None, gain: float | None = None, divisors=None) -> N.pa_rope:
    """A rotary embedding for ``KVPool.rope_and_cache`` (see pa_rope_desc).

    ``high`` defaults to 4 turns for "bands" and 32 for "yarn"; ``gain`` to 1, and
    for "yarn" with a factor above 1 to 0.1 ln(factor) + 1."""
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if gain is None:
        gain = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    return N.pa_rope_init(N.pa_rope_desc(ROPE_LAYOUTS[layout], rot_dim, ROPE_SCALINGS[scaling], theta,
                                         factor, original_len, low, high, gain), divisors)


def make_rope_axes(sections, order: str = "sections") -> N.pa_rope_axes:
    """Which axis each rotary pair turns with, for ``KVPool.norm_rope_and_cache``: sections[a]
    pairs turn with axis a's positions, rot_dim / 2 in all.  `order`: "sections" (the first
    sections[0] pairs with axis 0, and so on), or "turns" (pair i with axis i mod n for the
    first n sections[a] pairs of each axis a > 0; axis 0 has the rest)."""
    sections = [int(n) for n in sections]
    n, pairs = len(sections), sum(sections)
    if not 1 <= n <= N.PA_ROPE_MAX_AXES or min(sections) < 0 or not 1 <= pairs <= 64:
        raise ValueError(f"need 1 to {N.PA_ROPE_MAX_AXES} sections of 1 to 64 pairs together")
    if order == "sections":
        of = [a for a in range(n) for _ in range(sections[a])]
    elif order == "turns":
        of = [i % n if i < n * sections[i % n] else 0 for i in range(pairs)]
        if [of.count(a) for a in range(n)] != sections:
            raise ValueError(f"sections {sections} cannot take turns")
    else:
        raise ValueError("order must be 'sections' or 'turns'")
    axes = N.pa_rope_axes(n, (N.ctypes.c_uint8 * 64)(*of))
    axes.pairs = pairs
    return axes


def _check_pairs(axes, rope) -> None:
    """The sections of make_rope_axes must be those of this embedding's pairs.  (Axes filled by hand name all
    64 pairs, so they fit any.)"""
    pairs = getattr(axes, "pairs", None)
    if pairs is not None and rope is not None and 2 * pairs != rope.rot_dim:
        raise ValueError(f"axes of {pairs} pairs do not fit an embedding of {rope.rot_dim} dimensions")


def _token_rows(t: torch.Tensor, name: str, dtype, device) -> int:
    """The token stride, in elements, of a [T, heads, head_dim] tensor whose tokens may lie
    apart (a slice of a fused projection) but are contiguous in themselves."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device):
        _need(t[0:0] if isinstance(t, torch.Tensor) else t, name, dtype, device)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    T, heads, d = shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and heads > 1):
        raise ValueError(f"{name}: the heads and dimensions of a token must be contiguous")
    return st if T > 1 else heads * d


class KVPool:
    def __init__(self, n_layers: int, num_blocks: int, n_kv_heads: int, head_dim: int,
                 kv_dtype: str, k_scale: float = 1.0, v_scale: float = 1.0, device="cuda"):
        self.kv_dtype = kv_dtype
        self.code = KV_DTYPES[kv_dtype]
        self.desc = N.make_desc(n_layers, num_blocks, n_kv_heads, head_dim, self.code, k_scale,
                                v_scale)
        kb, vb = N.pa_pool_bytes(self.desc)
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.k_cache = torch.empty(kb, dtype=torch.uint8, device=self.device)
        self.v_cache = torch.empty(vb, dtype=torch.uint8, device=self.device)
        self.handle = N.pa_pool_create(self.desc, self.k_cache.data_ptr(), self.v_cache.data_ptr())
        self.n_layers, self.num_blocks = n_layers, num_blocks
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        self.elem_bytes = 1 if kv_dtype in ("fp8_e4m3", "fp8_e4m3_block") else 2
        self.block_scaled = kv_dtype == "fp8_e4m3_block"
        # bytes of one layer's tiles in each region (a block-scaled region ends
        # with the scale table [n_layers][num_blocks][n_kv_heads] of fp32)
        self.layer_bytes = num_blocks * n_kv_heads * 16 * head_dim * self.elem_bytes
        self.in_dtype = torch.float16 if kv_dtype == "fp16" else torch.bfloat16
        self.in_code = N.PA_FP16 if kv_dtype == "fp16" else N.PA_BF16

    # ----------------------------------------------------------------- life
    def close(self):
        if getattr(self, "handle", None):
            N.pa_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ----------------------------------------------------------- allocator
    def alloc(self, n: int) -> np.ndarray:
        return N.pa_block_alloc(self.handle, n)

    def free(self, ids) -> None:
        N.pa_block_free(self.handle, ids)

    def incref(self, ids) -> None:
        N.pa_block_incref(self.handle, ids)

    def refcount(self, block: int) -> int:
        return N.pa_block_refcount(self.handle, block)

    def stats(self):
        return N.pa_pool_stats(self.handle)

    def cow_prepare(self, table_row: np.ndarray, ctx_len: int):
        return N.pa_cow_prepare(self.handle, table_row, ctx_len)

    # -------------------------------------------------------- prefix cache
    def prefix_lookup(self, hashes) -> np.ndarray:
        return N.pa_prefix_lookup(self.handle, hashes)

    def prefix_register(self, hashes, ids) -> None:
        N.pa_prefix_register(self.handle, hashes, ids)

    def prefix_evict(self, max_blocks: int) -> int:
        return N.pa_prefix_evict(self.handle, max_blocks)

    def prefix_stats(self):
        return N.pa_prefix_stats(self.handle)

    # --------------------------------------------------------------- views
    def layer_view(self, which: str, layer: int = 0) -> torch.Tensor:
        """uint8 view [num_blocks, n_kv_heads, 16, head_dim * elem_bytes] of one layer."""
        buf = self.k_cache if which == "k" else self.v_cache
        per = self.layer_bytes
        return buf[layer * per:(layer + 1) * per].view(self.num_blocks, self.n_kv_heads, 16,
                                                         self.head_dim * self.elem_bytes)

    def scale_view(self, which: str, layer: int = 0) -> torch.Tensor:
        """float32 view [num_blocks, n_kv_heads] of one layer's K or V tile scales
        (block-scaled FP8 pools)."""
        if not self.block_scaled:
            raise ValueError("only block-scaled FP8 pools keep per-tile scales")
        buf = self.k_cache if which == "k" else self.v_cache
        n = self.num_blocks * self.n_kv_heads * 4
        off = self.n_layers * self.layer_bytes + layer * n
        return buf[off:off + n].view(torch.float32).view(self.num_blocks, self.n_kv_heads)

    # --------------------------------------------------------- device calls
    def _launch(self, call, args, stream) -> None:
        """call(*args, stream) with the pool's device current: the library launches there,
        and without a stream given it is that device's current one."""
        if torch._C._cuda_getDevice() == self.device.index:
            call(*args, _stream_handle(stream))
        else:
            with torch.cuda.device(self.device):
                call(*args, _stream_handle(stream))

    def _new(self, shape, dtype, stream) -> torch.Tensor:
        """A tensor for the call's stream to write: allocated in that stream's order, so neither
        its memory's last use nor its next one overlaps the call."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def reshape_and_cache(self, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                          layer: int = 0, stream=None) -> None:
        _need(k, "k", self.in_dtype, self.device)
        _need(v, "v", self.in_dtype, self.device)
        _need(slot_mapping, "slot_mapping", torch.int64, self.device)
        T = slot_mapping.numel()
        if k.numel() != T * self.n_kv_heads * self.head_dim or v.numel() != k.numel():
            raise ValueError("k and v must be [T, n_kv_heads, head_dim]")
        N.pa_reshape_and_cache(self.handle, layer, k.data_ptr(), v.data_ptr(),
                               slot_mapping.data_ptr(), T, _stream_handle(stream))

    def _rope_args(self, q, k, v, positions, slot_mapping, q_out, n_axes, stream):
        """Checks what the rotary writes share; returns q_out and the C call's last arguments."""
        dt, dev = self.in_dtype, self.device
        qs = _token_rows(q, "q", dt, dev)
        ks = _token_rows(k, "k", dt, dev)
        vs = _token_rows(v, "v", dt, dev)
        _all_need(dev, (positions, "positions", torch.int32), (slot_mapping, "slot_mapping", torch.int64))
        shape = q.shape
        T, Hq, D = shape
        kv = (T, self.n_kv_heads, self.head_dim)
        if D != self.head_dim or k.shape != kv or v.shape != kv:
            raise ValueError("q must be [T, n_q_heads, head_dim], k and v [T, n_kv_heads, head_dim]")
        if positions.numel() != n_axes * T or slot_mapping.numel() != T:
            raise ValueError("positions and slot_mapping must hold one entry per token (positions: and axis)")
        if q_out is None:
            q_out = self._new(shape, dt, stream)
        else:
            _all_need(dev, (q_out, "q_out", dt))
            if q_out.shape != shape:
                raise ValueError("q_out must have q's shape")
        return q_out, (q.data_ptr(), qs, q_out.data_ptr(), Hq, k.data_ptr(), ks, v.data_ptr(), vs,
                       positions.data_ptr(), slot_mapping.data_ptr(), T)

    def rope_and_cache(self, rope: N.pa_rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       positions: torch.Tensor, slot_mapping: torch.Tensor,
                       q_out: torch.Tensor | None = None, layer: int = 0, stream=None) -> torch.Tensor:
        """Rotate q [T, Hq, D] and k [T, Hkv, D] at `positions` (int32) and write k and v
        into their slots; returns the rotated q (`q_out`, which may be q itself when it is
        contiguous).  q, k and v may be slices of one fused projection."""
        q_out, args = self._rope_args(q, k, v, positions, slot_mapping, q_out, 1, stream)
        self._launch(N.pa_rope_and_cache, (self.handle, layer, rope, *args), stream)
        return q_out

    def _head_weight(self, w, name, heads) -> int:
        """The address of a norm's weights, [head_dim] or [heads, head_dim]."""
        _all_need(self.device, (w, name, self.in_dtype))
        shape, D = w.shape, self.head_dim
        if shape != (D,) and shape != (heads, D):
            raise ValueError(f"{name} must be [head_dim] or [heads, head_dim]")
        return w.data_ptr()

    def norm_rope_and_cache(self, rope: N.pa_rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            positions: torch.Tensor, slot_mapping: torch.Tensor,
                            q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                            eps: float = 1e-6, weight_offset: float = 0.0,
                            axes: N.pa_rope_axes | None = None, q_out: torch.Tensor | None = None,
                            layer: int = 0, stream=None) -> torch.Tensor:
        """``rope_and_cache`` that first divides every head of q and of k by its root mean square
        and multiplies it with `weight_offset` + its weights ([D], or [heads, D] for both; None: that
        side is not normalised).  With `axes` (``make_rope_axes``) positions is [n_axes, T]."""
        n_axes = 1
        if axes is not None:
            _check_pairs(axes, rope)
            n_axes = axes.n_axes
        q_out, args = self._rope_args(q, k, v, positions, slot_mapping, q_out, n_axes, stream)
        qw = kw = per_head = 0
        if q_weight is not None:
            qw = self._head_weight(q_weight, "q_weight", q.shape[1])
            per_head = q_weight.dim() - 1
        if k_weight is not None:
            kw = self._head_weight(k_weight, "k_weight", self.n_kv_heads)
            if q_weight is not None and k_weight.dim() - 1 != per_head:
                raise ValueError("q_weight and k_weight must both be [head_dim] or both [heads, head_dim]")
            per_head = k_weight.dim() - 1
        if n_axes > 1 and (positions.dim() != 2 or positions.shape[0] != n_axes):
            raise ValueError("positions must be [n_axes, T]")
        self._launch(N.pa_norm_rope_and_cache, (self.handle, layer, rope, axes, qw, kw, per_head, eps, weight_offset, *args),
                     stream)
        return q_out

    def copy_blocks(self, pairs: torch.Tensor, layer: int = 0, stream=None) -> None:
        _need(pairs, "pairs", torch.int32, self.device)
        N.pa_copy_blocks(self.handle, layer, pairs.data_ptr(), pairs.numel() // 2,
                         _stream_handle(stream))

    def swap_block_bytes(self) -> int:
        return N.pa_swap_block_bytes(self.handle)

    def swap_out(self, ids: torch.Tensor, host_buf: torch.Tensor, stream=None) -> None:
        """Copy blocks `ids` (device int32) into pinned host memory `host_buf`."""
        _need(ids, "ids", torch.int32, self.device)
        if not host_buf.is_pinned():
            raise ValueError("host_buf must be pinned host memory")
        if host_buf.numel() * host_buf.element_size() < ids.numel() * self.swap_block_bytes():
            raise ValueError("host_buf too small")
        N.pa_swap_out(self.handle, ids.numel(), ids.data_ptr(), host_buf.data_ptr(),
                      _stream_handle(stream))

    def swap_in(self, ids: torch.Tensor, host_buf: torch.Tensor, stream=None) -> None:
        """Copy a swap buffer back into blocks `ids` (device int32)."""
        _need(ids, "ids", torch.int32, self.device)
        if not host_buf.is_pinned():
            raise ValueError("host_buf must be pinned host memory")
        if host_buf.numel() * host_buf.element_size() < ids.numel() * self.swap_block_bytes():
            raise ValueError("host_buf too small")
        N.pa_swap_in(self.handle, ids.numel(), ids.data_ptr(), host_buf.data_ptr(),
                     _stream_handle(stream))

    def num_splits(self, S: int, n_q_heads: int, max_blocks_per_seq: int) -> int:
        return N.pa_decode_num_splits(self.handle, S, n_q_heads, max_blocks_per_seq)

    def workspace_bytes(self, S: int, n_q_heads: int, max_blocks_per_seq: int,
                        num_splits: int = 0) -> int:
        return N.pa_decode_workspace_bytes(self.handle, S, n_q_heads, max_blocks_per_seq,
                                           num_splits)

    def decode(self, q: torch.Tensor, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
               out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
               softmax_scale: float | None = None, num_splits: int = 0, layer: int = 0,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        _need(q, "q", self.in_dtype, self.device)
        _need(block_tables, "block_tables", torch.int32, self.device)
        _need(ctx_lens, "ctx_lens", torch.int32, self.device)
        S, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError("q head_dim mismatch")
        max_blocks = block_tables.shape[1]
        if out is None:
            out = torch.empty((S, Hq, D), dtype=out_dtype or q.dtype, device=self.device)
        _need(out, "out", None, self.device)
        code = _OUT_CODES[out.dtype]
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(D)
        ws_bytes = N.pa_decode_workspace_bytes(self.handle, S, Hq, max_blocks, num_splits)
        ws_ptr = 0
        if ws_bytes:
            if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device)
            ws_ptr = workspace.data_ptr()
        N.pa_decode(self.handle, layer, out.data_ptr(), code, q.data_ptr(),
                    block_tables.data_ptr(), max_blocks, ctx_lens.data_ptr(), S, Hq,
                    float(softmax_scale), num_splits, ws_ptr, ws_bytes, _stream_handle(stream))
        return out

    def weights_workspace_bytes(self, S: int, n_q_heads: int, max_blocks_per_seq: int) -> int:
        with torch.cuda.device(self.device):
            return N.pa_decode_weights_workspace_bytes(self.handle, S, n_q_heads, max_blocks_per_seq)

    def decode_weights(self, q: torch.Tensor, block_tables: torch.Tensor, ctx_lens: torch.Tensor,
                       weights: torch.Tensor | None, weights_out: torch.Tensor | None = None,
                       decay: float = 1.0, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype | None = None, softmax_scale: float | None = None,
                       layer: int = 0, workspace: torch.Tensor | None = None, stream=None):
        """``decode`` that also adds each token's attention weight to its running total:
        `weights` fp32 [S, n_kv_heads, tokens], updated in place unless `weights_out` is
        given (None: totals that start at zero).  Returns (out, weights_out)."""
        dev = self.device
        if weights_out is None:
            weights_out = weights
        _all_need(dev, (q, "q", self.in_dtype), (block_tables, "block_tables", torch.int32),
                  (ctx_lens, "ctx_lens", torch.int32), (weights_out, "weights_out", torch.float32))
        S, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError("q head_dim mismatch")
        if block_tables.dim() != 2 or block_tables.shape[0] != S or ctx_lens.numel() != S:
            raise ValueError("block_tables must be [S, max_blocks] and ctx_lens [S]")
        max_blocks = block_tables.shape[1]
        if weights_out.dim() != 3 or weights_out.shape[:2] != (S, self.n_kv_heads):
            raise ValueError("weights must be [S, n_kv_heads, tokens]")
        if weights is not None and weights is not weights_out:
            _need(weights, "weights", torch.float32, dev)
            if weights.shape != weights_out.shape:
                raise ValueError("weights and weights_out must have one shape")
        if out is None:
            out = self._new((S, Hq, D), out_dtype or q.dtype, stream)
        else:
            _need(out, "out", None, dev)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(D)
        if workspace is None:
            workspace = self._new(self.weights_workspace_bytes(S, Hq, max_blocks), torch.uint8, stream)
        else:
            _need(workspace, "workspace", None, dev)
        self._launch(N.pa_decode_weights,
                     (self.handle, layer, out.data_ptr(), _OUT_CODES[out.dtype], q.data_ptr(),
                      block_tables.data_ptr(), max_blocks, ctx_lens.data_ptr(), S, Hq, softmax_scale,
                      weights.data_ptr() if weights is not None else 0, weights_out.data_ptr(),
                      weights_out.shape[2], decay, workspace.data_ptr(),
                      workspace.numel() * workspace.element_size()), stream)
        return out, weights_out

    def evict_select(self, weights: torch.Tensor, ctx_lens: torch.Tensor, budget: int, sinks: int = 0,
                     recent: int = 0, keep: torch.Tensor | None = None,
                     kept_lens: torch.Tensor | None = None, stream=None):
        """The tokens that stay when each sequence is cut to `budget`: the first `sinks`, the
        last `recent` and the heaviest in between, by their totals `weights` [S, heads, tokens].
        Returns (keep int32 [S, heads, budget], ascending, -1 behind; kept_lens int32 [S])."""
        dev = self.device
        _all_need(dev, (weights, "weights", torch.float32), (ctx_lens, "ctx_lens", torch.int32))
        if weights.dim() != 3 or ctx_lens.numel() != weights.shape[0]:
            raise ValueError("weights must be [S, heads, tokens] and ctx_lens [S]")
        S, H, tokens = weights.shape
        if keep is None:
            keep = self._new((S, H, max(budget, 0)), torch.int32, stream)
        if kept_lens is None:
            kept_lens = self._new(S, torch.int32, stream)
        _all_need(dev, (keep, "keep", torch.int32), (kept_lens, "kept_lens", torch.int32))
        if keep.shape != (S, H, max(budget, 0)) or kept_lens.numel() != S:
            raise ValueError("keep must be [S, heads, budget] and kept_lens [S]")
        self._launch(N.pa_evict_select,
                     (self.handle, weights.data_ptr(), tokens, ctx_lens.data_ptr(), S, H, budget, sinks,
                      recent, keep.data_ptr(), kept_lens.data_ptr()), stream)
        return keep, kept_lens

    def evict_compact(self, keep: torch.Tensor, kept_lens: torch.Tensor, block_tables: torch.Tensor,
                      dst_tables: torch.Tensor, weights: torch.Tensor | None = None,
                      weights_out: torch.Tensor | None = None, layer: int = 0, stream=None):
        """Copy the kept tokens of `block_tables` together into the blocks of `dst_tables`
        (freshly allocated ones), and their totals from `weights` into `weights_out`, whose rows
        are zeroed behind them (a new tensor of the same shape when not given).  Returns weights_out."""
        _all_need(self.device, (keep, "keep", torch.int32), (kept_lens, "kept_lens", torch.int32),
                  (block_tables, "block_tables", torch.int32), (dst_tables, "dst_tables", torch.int32))
        if keep.dim() != 3:
            raise ValueError("keep must be [S, heads, budget]")
        S, H, budget = keep.shape
        if (kept_lens.numel() != S or block_tables.dim() != 2 or block_tables.shape[0] != S
                or dst_tables.dim() != 2 or dst_tables.shape[0] != S):
            raise ValueError("kept_lens must be [S], the tables [S, blocks]")
        w_in = w_out = in_stride = out_stride = 0
        if weights is None and weights_out is not None:
            raise ValueError("weights_out needs weights")
        if weights is not None:
            if weights_out is None:
                weights_out = self._new(weights.shape, torch.float32, stream)
            _all_need(self.device, (weights, "weights", torch.float32), (weights_out, "weights_out", torch.float32))
            for t, name in ((weights, "weights"), (weights_out, "weights_out")):
                if t.dim() != 3 or t.shape[:2] != (S, H):
                    raise ValueError(f"{name} must be [S, heads, tokens] with keep's heads")
            w_in, in_stride = weights.data_ptr(), weights.shape[2]
            w_out, out_stride = weights_out.data_ptr(), weights_out.shape[2]
        self._launch(N.pa_evict_compact,
                     (self.handle, layer, keep.data_ptr(), H, budget, kept_lens.data_ptr(),
                      block_tables.data_ptr(), block_tables.shape[1], dst_tables.data_ptr(),
                      dst_tables.shape[1], S, w_in, in_stride, w_out, out_stride), stream)
        return weights_out

    def tree_workspace_bytes(self, n_q_heads: int, max_nodes: int) -> int:
        with torch.cuda.device(self.device):
            return N.pa_decode_tree_workspace_bytes(self.handle, n_q_heads, max_nodes)

    def decode_tree(self, q: torch.Tensor, q_start: torch.Tensor, block_tables: torch.Tensor,
                    ctx_lens: torch.Tensor, max_nodes: int, mask: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                    softmax_scale: float | None = None, layer: int = 0,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of a tree of drafted tokens per sequence: rows q_start[s] .. q_start[s+1]-1 of
        q [T, Hq, D] are sequence s's nodes, the last ones of its ctx_lens[s] cached tokens.  Each
        attends to the history in front of them and to the nodes whose bits are set in its row of
        `mask`, int64 [T, ceil(max_nodes / 64)] (None: those before it and itself).  Rows of q
        and out behind q_start[S] are neither read nor written; out must not overlap q."""
        dev = self.device
        _all_need(dev, (q, "q", self.in_dtype), (q_start, "q_start", torch.int32),
                  (block_tables, "block_tables", torch.int32), (ctx_lens, "ctx_lens", torch.int32))
        if q.dim() != 3 or q.shape[2] != self.head_dim:
            raise ValueError("q must be [T, n_q_heads, head_dim]")
        T, Hq, D = q.shape
        S = ctx_lens.numel()
        if block_tables.dim() != 2 or block_tables.shape[0] != S or q_start.numel() != S + 1:
            raise ValueError("block_tables must be [S, max_blocks], ctx_lens [S] and q_start [S + 1]")
        if mask is not None:
            _need(mask, "mask", torch.int64, dev)
            if mask.shape != (T, -(-max_nodes // 64)):
                raise ValueError("mask must be [T, ceil(max_nodes / 64)]")
        if out is None:
            out = self._new((T, Hq, D), out_dtype or q.dtype, stream)
        else:
            _need(out, "out", None, dev)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        if out.dtype not in _OUT_CODES:
            raise TypeError(f"out cannot be {out.dtype}")
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(D)
        if workspace is None:
            workspace = self._new(self.tree_workspace_bytes(Hq, max_nodes), torch.uint8, stream)
        else:
            _need(workspace, "workspace", None, dev)
        self._launch(N.pa_decode_tree,
                     (self.handle, layer, out.data_ptr(), _OUT_CODES[out.dtype], q.data_ptr(), T, q_start.data_ptr(),
                      block_tables.data_ptr(), block_tables.shape[1], ctx_lens.data_ptr(), S, Hq, max_nodes,
                      mask.data_ptr() if mask is not None else 0, softmax_scale, workspace.data_ptr(),
                      workspace.numel() * workspace.element_size()), stream)
        return out

    def tree_accept(self, paths: torch.Tensor, path_lens: torch.Tensor, q_start: torch.Tensor,
                    block_tables: torch.Tensor, ctx_lens: torch.Tensor, new_lens: torch.Tensor | None = None,
                    layer: int = 0, n_layers: int | None = None, stream=None) -> torch.Tensor:
        """Move the K and V of the accepted nodes paths[s, :path_lens[s]] (ascending) of each sequence's
        tree right behind its history, in `n_layers` layers from `layer` on (None: all that follow).
        Returns the new context lengths (`new_lens`, which must not be one of the inputs)."""
        _all_need(self.device, (paths, "paths", torch.int32), (path_lens, "path_lens", torch.int32),
                  (q_start, "q_start", torch.int32), (block_tables, "block_tables", torch.int32),
                  (ctx_lens, "ctx_lens", torch.int32))
        S = ctx_lens.numel()
        if paths.dim() != 2 or paths.shape[0] != S or path_lens.numel() != S or q_start.numel() != S + 1:
            raise ValueError("paths must be [S, max_path], path_lens and ctx_lens [S], q_start [S + 1]")
        if block_tables.dim() != 2 or block_tables.shape[0] != S:
            raise ValueError("block_tables must be [S, max_blocks]")
        if new_lens is None:
            new_lens = self._new(S, torch.int32, stream)
        else:
            _need(new_lens, "new_lens", torch.int32, self.device)
            if new_lens.numel() != S:
                raise ValueError("new_lens must be [S]")
        if n_layers is None:
            n_layers = self.n_layers - layer
        self._launch(N.pa_tree_accept,
                     (self.handle, layer, n_layers, paths.data_ptr(), paths.shape[1], path_lens.data_ptr(),
                      q_start.data_ptr(), block_tables.data_ptr(), block_tables.shape[1], ctx_lens.data_ptr(), S,
                      new_lens.data_ptr()), stream)
        return new_lens

    def prefill(self, q: torch.Tensor, q_start: torch.Tensor, block_tables: torch.Tensor,
                ctx_lens: torch.Tensor, max_chunk: int, out: torch.Tensor | None = None,
                out_dtype: torch.dtype | None = None, softmax_scale: float | None = None,
                layer: int = 0, stream=None) -> torch.Tensor:
        """Causal attention of packed chunks q [T, Hq, D] (rows q_start[s] ..
        q_start[s+1]-1 for sequence s) over their paged history."""
        _need(q, "q", self.in_dtype, self.device)
        _need(q_start, "q_start", torch.int32, self.device)
        _need(block_tables, "block_tables", torch.int32, self.device)
        _need(ctx_lens, "ctx_lens", torch.int32, self.device)
        T, Hq, D = q.shape
        if out is None:
            out = torch.empty((T, Hq, D), dtype=out_dtype or q.dtype, device=self.device)
        _need(out, "out", None, self.device)
        code = _OUT_CODES[out.dtype]
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(D)
        N.pa_prefill(self.handle, layer, out.data_ptr(), code, q.data_ptr(), q_start.data_ptr(),
                     block_tables.data_ptr(), block_tables.shape[1], ctx_lens.data_ptr(),
                     ctx_lens.numel(), Hq, int(max_chunk), float(softmax_scale),
                     _stream_handle(stream))
        return out

    def device_error(self, stream=None) -> int:
        return N.pa_get_device_error(self.handle, _stream_handle(stream))
