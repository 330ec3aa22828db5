// pa_accept.cu -- the accepted path of a drafted tree moved together behind its
// sequence's history, in place.
//
// Node path[i] goes to place i.  The path ascends, so path[i] >= i: a place is never
// the source of a later one, and a warp that goes through the path in order, its loads
// before its stores, needs no copy.  A (layer, sequence, kv head) belongs to one warp;
// rows move as 16-byte vectors.
//
// There is little to move (the floor of 64 paths in 32 layers is 1.9 us of HBM's time), so what
// counts is the chain of dependent loads: lengths, path, table, rows (block-scaled tiles: and
// scales).  One layer, 64 paths, bf16: 2.9 us; 32 layers, FP8: 5.6 us; 32 layers, 33 paths,
// block-scaled: 18.6 us, issue slots 55% busy with the new codes (a quotient per value).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kAcceptThreads = 256;
constexpr int kWave = 152 * 4;  // CTAs that the GPU (152 SMs) holds at 64 registers a thread; a size, not a limit

struct AcceptArgs {
  const int32_t* paths;  // [S][max_path]
  const int32_t* lens;
  const int32_t* q_start;
  const int32_t* tables;
  const int32_t* ctx;
  int32_t* new_lens;
  int max_path, max_blocks, S, Hkv, num_blocks;
  int units_per_seq;        // warps of one sequence
  long long ctas_per_seq;
  uint8_t* k;  // the first layer's regions
  uint8_t* v;
  size_t layer_bytes;
  float* ksc;  // block-scaled pools: the first layer's scales
  float* vsc;
  unsigned int* err;
};

// A sequence's path: its history and length, or length 0 where something is wrong with it.
struct Path {
  int base, len, ctx;
};

__device__ __forceinline__ Path check_path(const AcceptArgs& a, int s) {
  const int lane = threadIdx.x & 31;
  const int q0 = a.q_start[s], q1 = a.q_start[s + 1], len = a.lens[s];
  Path p;
  p.ctx = a.ctx[s];
  const long long n = (long long)q1 - q0;
  bool bad = q0 < 0 || n < 0 || n > PA_TREE_MAX_NODES || p.ctx < n || p.ctx > 16ll * a.max_blocks || len < 0 || len > a.max_path ||
             len > n;
  if (!bad) {
    int before = -1;  // the node in front of these 32
    for (int i0 = 0; i0 < len; i0 += 32) {
      const int node = i0 + lane < len ? a.paths[(long long)s * a.max_path + i0 + lane] : 0x7FFFFFFF;
      int prev = __shfl_up_sync(kAll, node, 1);
      if (lane == 0) prev = before;
      before = __shfl_sync(kAll, node, 31);
      bad = bad || (i0 + lane < len && (node <= prev || node >= n));
    }
  }
  bad = __any_sync(kAll, bad);
  if (bad && lane == 0) record_error(a.err, PA_ERR_BOUNDS);
  p.base = bad ? p.ctx : p.ctx - (int)n;
  p.len = bad ? 0 : len;
  return p;
}

// The block and place, 16 * block + offset, of token t of sequence s; -1 where its table entry is
// no block (reported).
__device__ __forceinline__ long long place_of(const AcceptArgs& a, int s, int t) {
  const int b = a.tables[(long long)s * a.max_blocks + (t >> 4)];
  if (b < 0 || b >= a.num_blocks) {
    record_error(a.err, PA_ERR_BOUNDS);
    return -1;
  }
  return 16ll * b + (t & 15);
}

// The row (block * Hkv + h) * 16 + offset of a place.
__device__ __forceinline__ long long row_at(const AcceptArgs& a, long long place, int h) {
  return place < 0 ? -1 : ((place >> 4) * a.Hkv + h) * 16 + (place & 15);
}

// Rows of ROW bytes as they are.  The rows of a warp's (layer, kv head) pairs are one list, pair
// by pair, so that BATCH instructions' loads are in flight however short the path is.
template <int ROW>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs a) {
  constexpr int VPR = ROW / 16, RPW = 32 / VPR;  // vectors per row, rows per warp instruction
  constexpr int BATCH = 4;                       // warp instructions whose loads are in flight together, for K and V each
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int s = (int)(blockIdx.x / a.ctas_per_seq);
  const int first = (int)(blockIdx.x % a.ctas_per_seq) * (kAcceptThreads / 32) + (int)(threadIdx.x >> 5);
  const int step = (int)a.ctas_per_seq * (kAcceptThreads / 32);
  if (first >= a.units_per_seq) return;
  const int units = (a.units_per_seq - first + step - 1) / step;
  const Path p = check_path(a, s);
  if (first == 0 && lane == 0) a.new_lens[s] = p.base + p.len;
  for (int i0 = 0; i0 < p.len; i0 += 32) {
    // lane i: where place i0 + i is, and where its row comes from
    long long src = -1, dst = -1;
    const int i = i0 + lane;
    if (i < p.len) {
      const int node = a.paths[(long long)s * a.max_path + i];
      if (node != i) {
        src = place_of(a, s, p.base + node);
        dst = place_of(a, s, p.base + i);
      }
    }
    // nodes in their place already are the path's first ones
    const unsigned moves = __ballot_sync(kAll, src >= 0 && dst >= 0);
    if (moves == 0) continue;
    const int r_first = __ffs(moves) - 1, rows = 32 - __clz(moves) - r_first;
    int u = (lane / VPR) / rows, r = (lane / VPR) - u * rows;
    while (true) {
      uint4 xk[BATCH], xv[BATCH];
      uint8_t* to[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const long long from = __shfl_sync(kAll, src, r_first + r), at = __shfl_sync(kAll, dst, r_first + r);
        to[b] = nullptr;
        if (u < units && from >= 0 && at >= 0) {
          const int unit = first + u * step, layer = unit / a.Hkv, h = unit - layer * a.Hkv;
          uint8_t* kp = a.k + layer * a.layer_bytes + (lane % VPR) * 16;
          to[b] = kp + row_at(a, at, h) * ROW;
          const uint8_t* x = kp + row_at(a, from, h) * ROW;
          xk[b] = *reinterpret_cast<const uint4*>(x);
          xv[b] = *reinterpret_cast<const uint4*>(x + (a.v - a.k));
        }
        r += RPW;
        while (r >= rows) r -= rows, ++u;
      }
      __syncwarp();
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        if (to[b]) {
          *reinterpret_cast<uint4*>(to[b]) = xk[b];
          *reinterpret_cast<uint4*>(to[b] + (a.v - a.k)) = xv[b];
        }
      __syncwarp();
      if (__all_sync(kAll, u >= units)) break;
    }
  }
}

// E4M3 codes of 16 values given as codes, times s_src, over s.
__device__ __forceinline__ uint4 recode(uint4 x, float s_src, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t f[2];
    e4m3x4_to_f16x2x2(w[q], f[0], f[1]);
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 u = unpack2<false>(f[j]);
      float2 y = make_float2(0.f, 0.f);
      if (s > 0.f) y = make_float2(__fdiv_rn(__fmul_rn(u.x, s_src), s), __fdiv_rn(__fmul_rn(u.y, s_src), s));
      c[j] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    }
    o[q] = c[0] | (c[1] << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Bits of the largest |code value| times s_src of 16 codes.  A NaN counts for nothing: the tile's scale grows for the
// other values, which would be cut off at the old one.
__device__ __forceinline__ uint32_t top_bits(uint4 x, float s_src) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __half2 top = __float2half2_rn(0.f);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t f[2];
    e4m3x4_to_f16x2x2(w[q], f[0], f[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) top = __hmax2(top, __habs2(*reinterpret_cast<__half2*>(&f[j])));
  }
  const float2 t = __half22float2(top);
  return __float_as_uint(fmaxf(fmaxf(fabsf(__fmul_rn(t.x, s_src)), fabsf(__fmul_rn(t.y, s_src))), 0.f));
}

// A scale per tile: a warp per (layer, kv head, K or V), destination tile by
// destination tile.  Lane l holds vectors 32 j + l of the tile and of the rows that move
// into it, so a place's old code and its new one are the same lane's.
template <int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_block_kernel(const AcceptArgs a) {
  constexpr int VPR = D / 16, PER = 16 * VPR / 32;  // vectors per row, per lane
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int s = (int)(blockIdx.x / a.ctas_per_seq);
  const int unit = (int)(blockIdx.x % a.ctas_per_seq) * (kAcceptThreads / 32) + (int)(threadIdx.x >> 5);
  if (unit >= a.units_per_seq) return;
  const int which = unit & 1, layer = (unit >> 1) / a.Hkv, h = (unit >> 1) - layer * a.Hkv;
  const Path p = check_path(a, s);
  if (unit == 0 && lane == 0) a.new_lens[s] = p.base + p.len;
  uint8_t* pool = (which ? a.v : a.k) + layer * a.layer_bytes;
  float* scales = (which ? a.vsc : a.ksc) + (long long)layer * a.num_blocks * a.Hkv;
  for (int t0 = p.base & ~15; t0 < p.base + p.len; t0 += 16) {  // the tile's first token
    // lane r < 16: where row r comes from
    const int i = t0 + lane - p.base;
    long long src = -1;
    if (lane < 16 && i >= 0 && i < p.len) {
      const int node = a.paths[(long long)s * a.max_path + i];
      if (node != i) src = row_at(a, place_of(a, s, p.base + node), h);
    }
    if (!__any_sync(kAll, src >= 0)) continue;
    const long long dtile = row_at(a, place_of(a, s, t0), h) >> 4;  // (-1 stays negative)
    if (dtile < 0) continue;
    const float s_old = scales[dtile];
    const float s_src = src >= 0 ? scales[src >> 4] : 0.f;
    uint4 x[PER];
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int r = (32 * j + lane) / VPR;
      const long long from = __shfl_sync(kAll, src, r);
      const float sr = __shfl_sync(kAll, s_src, r);
      x[j] = make_uint4(0, 0, 0, 0);
      if (from >= 0) x[j] = *reinterpret_cast<const uint4*>(pool + from * D + (lane % VPR) * 16);
      if (from >= 0 && (from >> 4) != dtile) mb = max(mb, top_bits(x[j], sr));
    }
    mb = __reduce_max_sync(kAll, mb);
    const float s_run = __fdiv_rn(__uint_as_float(mb), 448.f);
    const bool grow = s_run > s_old;
    const float sn = grow ? s_run : s_old;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int r = (32 * j + lane) / VPR;
      const long long from = __shfl_sync(kAll, src, r);
      const float sr = __shfl_sync(kAll, s_src, r);
      uint4* at = reinterpret_cast<uint4*>(pool + dtile * 16 * D) + 32 * j + lane;
      if (from >= 0) *at = recode(x[j], sr, sn);
      else if (grow) *at = recode(*at, s_old, sn);
    }
    if (lane == 0 && grow) scales[dtile] = sn;
    __syncwarp();
  }
}

typedef void (*AcceptKernel)(AcceptArgs);

AcceptKernel pick_accept(const pa_pool* pool) {
  const int row = pool->desc.head_dim * pool->elem_bytes;
  if (pool->block_scaled) return row == 64 ? accept_block_kernel<64> : accept_block_kernel<128>;
  return row == 64 ? accept_kernel<64> : row == 128 ? accept_kernel<128> : accept_kernel<256>;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_tree_accept(pa_pool* pool, int layer, int n_layers, const int32_t* paths_dev, int max_path,
                   const int32_t* path_lens_dev, const int32_t* q_start_dev, const int32_t* block_tables_dev,
                   int max_blocks_per_seq, const int32_t* ctx_lens_dev, int S, int32_t* new_lens_dev, void* stream) {
  pa::TraceRange trace_("pa_tree_accept");
  int st = check_pool_layer(pool, layer);
  if (st) return st;
  const pa_pool_desc& d = pool->desc;
  if (n_layers < 1 || n_layers > d.n_layers - layer)
    return fail(PA_ERR_INVALID, "n_layers must be 1 to %d from layer %d on (got %d)", d.n_layers - layer, layer, n_layers);
  if (S > 65535) return fail(PA_ERR_UNSUPPORTED, "at most 65535 sequences per call");
  if (S < 0 || max_path < 0 || max_path > PA_TREE_MAX_NODES || max_blocks_per_seq < 1)
    return fail(PA_ERR_INVALID, "need S >= 0, max_path 0 to %d and tables of at least one block", PA_TREE_MAX_NODES);
  if (max_blocks_per_seq > (1 << 27) - 256)
    return fail(PA_ERR_UNSUPPORTED, "tables of at most 2^27 - 256 blocks (got %d)", max_blocks_per_seq);
  if (S == 0) return PA_OK;
  if (!path_lens_dev || !q_start_dev || !block_tables_dev || !ctx_lens_dev || !new_lens_dev || (max_path > 0 && !paths_dev))
    return fail(PA_ERR_INVALID, "null argument");
  const size_t lens_bytes = (size_t)S * 4;
  if (overlap(new_lens_dev, lens_bytes, ctx_lens_dev, lens_bytes) ||
      overlap(new_lens_dev, lens_bytes, path_lens_dev, lens_bytes) ||
      overlap(new_lens_dev, lens_bytes, q_start_dev, lens_bytes + 4) ||
      overlap(new_lens_dev, lens_bytes, block_tables_dev, lens_bytes * max_blocks_per_seq) ||
      overlap(new_lens_dev, lens_bytes, paths_dev, lens_bytes * max_path))
    return fail(PA_ERR_INVALID, "new_lens must be another buffer than the inputs, which every head reads");
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  AcceptArgs a = {};
  a.paths = paths_dev;
  a.lens = path_lens_dev;
  a.q_start = q_start_dev;
  a.tables = block_tables_dev;
  a.ctx = ctx_lens_dev;
  a.new_lens = new_lens_dev;
  a.max_path = max_path;
  a.max_blocks = max_blocks_per_seq;
  a.S = S;
  a.Hkv = d.n_kv_heads;
  a.num_blocks = d.num_blocks;
  const long long units = (long long)n_layers * d.n_kv_heads * (pool->block_scaled ? 2 : 1);
  if (units > (1 << 30)) return fail(PA_ERR_UNSUPPORTED, "too many layers and kv heads for one call");
  long long ctas = (units + kAcceptThreads / 32 - 1) / (kAcceptThreads / 32);
  // Plain rows: one wave of CTAs, whose warps take several (layer, kv head) pairs each and find their path
  // once (64 paths in 32 layers of 8 kv heads, FP8: 5.6 us, 9.5 with a pair per warp).
  // Block-scaled tiles, which need arithmetic more than loads in flight: a warp per layer, head and
  // region (33 paths in 32 layers of 8 kv heads: 18.7 us, 24 in one wave).
  if (!pool->block_scaled) ctas = std::min(ctas, std::max(1ll, (long long)kWave / S));
  if (ctas * S > 0x7FFFFFFF) return fail(PA_ERR_UNSUPPORTED, "too many sequences, layers and kv heads for one call");
  a.units_per_seq = (int)units;
  a.ctas_per_seq = ctas;
  a.k = pool->k + (size_t)layer * pool->layer_bytes;
  a.v = pool->v + (size_t)layer * pool->layer_bytes;
  a.layer_bytes = pool->layer_bytes;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  a.err = err;
  pick_accept(pool)<<<(unsigned)(ctas * S), kAcceptThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "tree_accept launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
