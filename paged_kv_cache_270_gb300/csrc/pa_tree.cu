// pa_tree.cu -- attention of a tree of drafted tokens per sequence over the paged KV cache.
//
// A node's result is softmax(scale q K^T) V over its sequence's history and the nodes
// whose bits its mask row has.  One warp per (node, kv head): the group's queries
// in registers, one token at a time.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

struct TreeArgs {
  const uint16_t* q;
  void* out;
  const uint64_t* mask;
  const int32_t* q_start;
  const int32_t* tables;
  const int32_t* ctx;
  const uint8_t* k;
  const uint8_t* v;
  const float* ksc;
  const float* vsc;
  int T, S, Hq, Hkv, G, max_blocks, num_blocks, max_nodes, words;
  float scale, k_scale, v_scale;
  unsigned int* err;
};

// Two neighbouring elements of a row.
template <int KV>
__device__ __forceinline__ float2 elem2(const uint8_t* row, int pair) {
  if constexpr (KV == PA_FP16 || KV == PA_BF16)
    return unpack2<KV == PA_BF16>(reinterpret_cast<const uint32_t*>(row)[pair]);
  else
    return unpack2<false>(e4m3x2_to_f16x2(reinterpret_cast<const uint16_t*>(row)[pair]));
}

template <int KV, int D, bool F32>
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a) {
  constexpr int EB = KV == PA_FP16 || KV == PA_BF16 ? 2 : 1;
  constexpr int P = D / 64;  // pairs of dimensions a lane holds
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(unit % a.Hkv), node0 = (int)(unit / a.Hkv % a.max_nodes);
  const long long s = unit / a.Hkv / a.max_nodes;
  if (s >= a.S) return;
  const int q0 = a.q_start[s], q1 = a.q_start[s + 1];
  const long long n = (long long)q1 - q0;
  if (n == 0) return;
  const int ctx = a.ctx[s];
  if (q0 < 0 || n < 0 || q1 > a.T || n > a.max_nodes || ctx < n || ctx > 16ll * a.max_blocks) {
    if (lane == 0) record_error(a.err, PA_ERR_BOUNDS);
    return;
  }
  if (node0 >= n) return;
  const int t = q0 + node0;
  const int base = ctx - (int)n;
  float2 q[8][P], o[8][P];
  float m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      o[g][p] = make_float2(0.f, 0.f);
      q[g][p] = make_float2(0.f, 0.f);
      if (g < a.G)
        q[g][p] = unpack2<KV != PA_FP16>(reinterpret_cast<const uint32_t*>(a.q + ((size_t)t * a.Hq + h * a.G + g) * D)[32 * p + lane]);
    }
  }
  for (int j = 0; j < ctx; ++j) {
    const int node = j - base;
    if (node >= 0 && !(a.mask ? a.mask[(size_t)t * a.words + (node >> 6)] >> (node & 63) & 1 : node <= t - q0)) continue;
    const int blk = a.tables[(size_t)s * a.max_blocks + (j >> 4)];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) record_error(a.err, PA_ERR_BOUNDS);
      continue;
    }
    const size_t tile = (size_t)blk * a.Hkv + h;
    const uint8_t* kr = a.k + (tile * 16 + (j & 15)) * D * EB;
    const uint8_t* vr = a.v + (tile * 16 + (j & 15)) * D * EB;
    const float ks = a.ksc ? a.ksc[tile] : a.k_scale, vs = a.vsc ? a.vsc[tile] : a.v_scale;
    float2 k[P], v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      k[p] = elem2<KV>(kr, 32 * p + lane);
      v[p] = elem2<KV>(vr, 32 * p + lane);
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (g >= a.G) break;
      float x = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) x += q[g][p].x * k[p].x + q[g][p].y * k[p].y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
      x *= a.scale * ks;
      const float mn = fmaxf(m[g], x);
      if (mn == -INFINITY && x == x) continue;  // (a NaN counts)
      const float f = expf(m[g] - mn), w = expf(x - mn);
      m[g] = mn;
      l[g] = l[g] * f + w;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        o[g][p].x = o[g][p].x * f + w * (v[p].x * vs);
        o[g][p].y = o[g][p].y * f + w * (v[p].y * vs);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (g >= a.G) break;
    const float inv = m[g] == -INFINITY ? 0.f : 1.f / l[g];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const size_t at = ((size_t)t * a.Hq + h * a.G + g) * (D / 2) + 32 * p + lane;
      const float x = o[g][p].x * inv, y = o[g][p].y * inv;
      if constexpr (F32) static_cast<float2*>(a.out)[at] = make_float2(x, y);
      else static_cast<uint32_t*>(a.out)[at] = pack2<KV != PA_FP16>(x, y);
    }
  }
}

typedef void (*TreeKernel)(TreeArgs);

template <int KV>
TreeKernel pick_tree(int D, bool f32) {
  if (D == 64) return f32 ? tree_kernel<KV, 64, true> : tree_kernel<KV, 64, false>;
  return f32 ? tree_kernel<KV, 128, true> : tree_kernel<KV, 128, false>;
}

TreeKernel pick_tree(int kv, int D, bool f32) {
  if (kv == PA_FP16) return pick_tree<PA_FP16>(D, f32);
  return kv == PA_BF16 ? pick_tree<PA_BF16>(D, f32) : pick_tree<PA_FP8_E4M3>(D, f32);
}

// What both calls check of a batch's trees.
int check_tree(const pa_pool* pool, int n_q_heads, int max_nodes) {
  const int st = check_shape(pool, 1, n_q_heads, 1);
  if (st) return st;
  if (max_nodes < 1 || max_nodes > PA_TREE_MAX_NODES)
    return fail(PA_ERR_INVALID, "max_nodes must be 1 to %d (got %d)", PA_TREE_MAX_NODES, max_nodes);
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_decode_tree_workspace_bytes(const pa_pool* pool, int n_q_heads, int max_nodes, size_t* bytes) {
  const int st = check_tree(pool, n_q_heads, max_nodes);
  if (st) return st;
  if (!bytes) return fail(PA_ERR_INVALID, "null output");
  *bytes = 16;
  return PA_OK;
}

int pa_decode_tree(pa_pool* pool, int layer, void* out, int out_dtype, const void* q, int T, const int32_t* q_start_dev,
                   const int32_t* block_tables_dev, int max_blocks_per_seq, const int32_t* ctx_lens_dev, int S,
                   int n_q_heads, int max_nodes, const uint64_t* tree_mask_dev, float softmax_scale, void* workspace,
                   size_t workspace_bytes, void* stream) {
  pa::TraceRange trace_("pa_decode_tree");
  int st = check_decode_args(pool, layer, out_dtype, S, n_q_heads, max_blocks_per_seq, softmax_scale);
  if (st) return st;
  if ((st = check_tree(pool, n_q_heads, max_nodes))) return st;
  if (max_blocks_per_seq > (1 << 27) - 256)
    return fail(PA_ERR_UNSUPPORTED, "tables of at most 2^27 - 256 blocks (got %d)", max_blocks_per_seq);
  if (T < 0) return fail(PA_ERR_INVALID, "T must be >= 0");
  if (S == 0 || T == 0) return PA_OK;
  st = check_decode_ptrs(out, q, block_tables_dev, ctx_lens_dev);
  if (st) return st;
  if (!q_start_dev) return fail(PA_ERR_INVALID, "null argument");
  if ((uintptr_t)tree_mask_dev & 7u) return fail(PA_ERR_INVALID, "tree_mask must be 8-byte aligned");
  if (!workspace || ((uintptr_t)workspace & 15u))
    return fail(PA_ERR_INVALID, "a 16-byte aligned workspace is needed");
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  const pa_pool_desc& d = pool->desc;
  TreeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.out = out;
  a.mask = tree_mask_dev;
  a.q_start = q_start_dev;
  a.tables = block_tables_dev;
  a.ctx = ctx_lens_dev;
  a.k = pool->k + (size_t)layer * pool->layer_bytes;
  a.v = pool->v + (size_t)layer * pool->layer_bytes;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  a.T = T;
  a.S = S;
  a.Hq = n_q_heads;
  a.Hkv = d.n_kv_heads;
  a.G = n_q_heads / d.n_kv_heads;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = d.num_blocks;
  a.max_nodes = max_nodes;
  a.words = (max_nodes + 63) / 64;
  a.scale = softmax_scale;
  a.k_scale = d.kv_dtype == PA_FP8_E4M3 ? d.k_scale : 1.f;
  a.v_scale = d.kv_dtype == PA_FP8_E4M3 ? d.v_scale : 1.f;
  a.err = err;
  const long long ctas = ((long long)S * max_nodes * d.n_kv_heads + 3) / 4;
  if (ctas > 0x7FFFFFFF) return fail(PA_ERR_UNSUPPORTED, "too many rows for one call");
  pick_tree(d.kv_dtype, d.head_dim, out_dtype == PA_FP32)<<<(unsigned)ctas, 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "decode_tree launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
