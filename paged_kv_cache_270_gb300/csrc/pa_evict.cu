// pa_evict.cu -- eviction by accumulated attention weight: which tokens of a
// sequence stay (pa_evict_select), and the move of their keys, values and
// totals into other pages (pa_evict_compact).
//
// "Capítulo 8 -- Gestión de caché KV de nueva generación", section 8.2: the
// tokens with the largest accumulated attention stay, with the first tokens and
// a window of the last ones; the rest give their pages back.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- selection
// The k-th largest of a row is found digit by digit, most significant first
// (four 8-bit digits of an order-preserving integer key, a histogram each),
// then one ordered pass writes what lies above it and the first of what equals
// it.  A row is shared by a cluster of CTAs, which hold its keys in shared
// memory (the row is read from HBM once) and add up their histograms through
// distributed shared memory.  Counts are integers, so the result depends on no
// order of execution.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxKeys = 49152;  // keys a CTA keeps (192 KiB); longer shares are read again in each pass

struct SelectArgs {
  const float* w;
  long long stride;
  const int32_t* ctx;
  int S, H;
  int budget, sinks, recent;
  int32_t* keep;
  int32_t* kept;
  int max_keys;  // keys of the CTA's dynamic shared memory
  unsigned int* err;
};

// Larger floats have larger keys; -0 counts as 0, NaN comes below every number.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Adds each lane's digit (those with `in`) to the histogram.  Totals crowd
// into few bins (all the tokens that nothing attends to share one), and a
// shared-memory atomic serialises on equal addresses: the lanes that agree with
// the first remaining one are counted by a ballot, twice, before the rest add
// one by one.
__device__ __forceinline__ void hist_add(uint32_t* hist, uint32_t digit, bool in) {
  const int lane = threadIdx.x & 31;
  unsigned left = __ballot_sync(kAll, in);
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    if (!left) return;
    const int lead = __ffs(left) - 1;
    const uint32_t d = __shfl_sync(kAll, digit, lead);
    const unsigned same = __ballot_sync(kAll, digit == d) & left;
    if (lane == lead) atomicAdd(&hist[d], (uint32_t)__popc(same));
    left &= ~same;
  }
  if ((left >> lane) & 1u) atomicAdd(&hist[digit], 1u);
}

template <int C>
__device__ __forceinline__ void row_sync() {
  if constexpr (C == 1) __syncthreads();
  else cg::this_cluster().sync();
}

template <int C>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2][256];
  __shared__ uint32_t s_scan[8];
  __shared__ uint32_t s_digit, s_rem;
  __shared__ uint2 s_warp[kSelWarps];
  __shared__ uint2 s_cta;  // (above, equal) of this CTA's share
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / C, rank = blockIdx.x % C;
  const int seq = row / a.H;
  grid_dependents_launch();
  int n = a.ctx[seq];
  if (n < 0 || n > a.stride) {
    if (tid == 0 && rank == 0) record_error(a.err, PA_ERR_BOUNDS);
    n = n < 0 ? 0 : (int)a.stride;
  }
  int32_t* keep = a.keep + (long long)row * a.budget;
  if (tid == 0 && rank == 0 && row == seq * a.H) a.kept[seq] = min(n, a.budget);
  if (n <= a.budget) {  // everything stays (the same for all CTAs of the row)
    for (int i = rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads) keep[i] = i < n ? i : -1;
    return;
  }
  for (int i = rank * kSelThreads + tid; i < a.sinks + a.recent; i += C * kSelThreads)
    keep[i < a.sinks ? i : a.budget - a.recent + (i - a.sinks)] = i < a.sinks ? i : n - a.recent + (i - a.sinks);
  const int k = a.budget - a.sinks - a.recent;
  if (k == 0) return;

  // this CTA's share of the m tokens between the first and the last ones
  const int m = n - a.sinks - a.recent;
  const int chunk = ((m + C - 1) / C + 31) / 32 * 32;
  const int begin = (int)min((long long)m, (long long)rank * chunk), cnt = min(chunk, m - begin);
  const float* src = a.w + (long long)row * a.stride + a.sinks + begin;
  auto key_at = [&](int i) { return i < a.max_keys ? keys[i] : order_key(src[i]); };

  for (int i = tid; i < 512; i += kSelThreads) hist[i >> 8][i & 255] = 0;
  __syncthreads();
  uint32_t prefix = 0;
  uint32_t rem = k;  // still to be taken among the keys that start with the prefix
#pragma unroll 1
  for (int p = 0; p < 4; ++p) {
    uint32_t* h = hist[p & 1];
    const int shift = 24 - 8 * p;
    if (p == 0) {
      // eight loads in flight per thread
      for (int i0 = 0; i0 < cnt; i0 += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + j * kSelThreads + tid;
          x[j] = i < cnt ? src[i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + j * kSelThreads + tid;
          const uint32_t key = order_key(x[j]);
          if (i < cnt && i < a.max_keys) keys[i] = key;
          if (i0 + j * kSelThreads < cnt) hist_add(h, key >> 24, i < cnt);  // (uniform per CTA)
        }
      }
    } else {
      for (int i0 = 0; i0 < cnt; i0 += kSelThreads) {
        const int i = i0 + tid;
        const uint32_t key = i < cnt ? key_at(i) : 0u;
        hist_add(h, (key >> shift) & 255u, i < cnt && (key >> (shift + 8)) == prefix);
      }
    }
    row_sync<C>();  // every CTA's histogram is complete
    // the bins of the whole row from the top down, and the one that holds the rem-th key
    uint32_t c = 0;
    if (tid < 256) {
      if constexpr (C == 1) {
        c = h[255 - tid];
      } else {
#pragma unroll
        for (int r = 0; r < C; ++r) c += cg::this_cluster().map_shared_rank(h, r)[255 - tid];
      }
      uint32_t x = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, x, off);
        if (lane >= off) x += y;
      }
      if (lane == 31) s_scan[warp] = x;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      uint32_t before = x - c;
      for (int w = 0; w < warp; ++w) before += s_scan[w];
      if (before < rem && rem <= before + c) {
        s_digit = 255 - tid;
        s_rem = rem - before;
      }
    } else {
      // the other buffer's readers passed the barrier above: clear it for the next digit
      hist[(p + 1) & 1][tid - 256] = 0;
    }
    __syncthreads();
    prefix = (prefix << 8) | s_digit;
    rem = s_rem;
  }

  // ---- above the threshold key, and equal to it: counts per warp, each warp
  // one stretch of the share
  const int seg = ((cnt + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(cnt, warp * seg), w1 = min(cnt, w0 + seg);
  uint32_t above = 0, equal = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t key = key_at(i);
    above += key > prefix;
    equal += key == prefix;
  }
  above = __reduce_add_sync(kAll, above);
  equal = __reduce_add_sync(kAll, equal);
  if (lane == 0) s_warp[warp] = make_uint2(above, equal);
  __syncthreads();
  uint32_t ga = 0, ge = 0, ta = 0, te = 0;  // before this warp in the CTA; of the CTA
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint2 v = s_warp[w];
    ga += w < warp ? v.x : 0;
    ge += w < warp ? v.y : 0;
    ta += v.x;
    te += v.y;
  }
  if constexpr (C > 1) {
    if (tid == 0) s_cta = make_uint2(ta, te);
    cg::this_cluster().sync();
    for (int r = 0; r < rank; ++r) {
      const uint2 v = *cg::this_cluster().map_shared_rank(&s_cta, r);
      ga += v.x;
      ge += v.y;
    }
  }
  // ---- the taken tokens in order: all above, and the first rem of the equal ones
  const unsigned lower = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < w1 ? key_at(i) : 0u;
    const bool is_a = i < w1 && key > prefix, is_e = i < w1 && key == prefix;
    const unsigned ba = __ballot_sync(kAll, is_a), be = __ballot_sync(kAll, is_e);
    const uint32_t ea = ga + __popc(ba & lower), ee = ge + __popc(be & lower);
    if (is_a || (is_e && ee < rem)) keep[a.sinks + ea + min(ee, rem)] = a.sinks + begin + i;
    ga += __popc(ba);
    ge += __popc(be);
  }
  if constexpr (C > 1) cg::this_cluster().sync();  // no CTA leaves while another may read its memory
}

// ---------------------------------------------------------------- compaction
// One warp per destination tile (sequence, kv head, page): 16 rows, gathered
// from wherever they lie.  Lanes 0-15 resolve the rows' addresses; the rows
// then move as 16-byte vectors, all loads of a batch in flight before the
// first store.
struct CompactArgs {
  const int32_t* keep;
  int keep_heads, budget;
  const int32_t* kept;
  const int32_t* src_tables;
  int src_blocks;  // columns
  const int32_t* dst_tables;
  int dst_blocks;
  int S, Hkv, num_blocks;
  uint8_t* k;
  uint8_t* v;
  float* ksc;  // block-scaled pools
  float* vsc;
  const float* w_in;  // nullptr: no totals
  long long w_in_stride;
  float* w_out;
  long long w_out_stride;
  int warps_per_row;  // >= the destination pages of a row
  unsigned int* err;
};

constexpr int kCompactThreads = 256;

// ROW: bytes of one token row of a tile (64, 128 or 256).
template <int ROW, bool BLK>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactArgs a) {
  constexpr int VPR = ROW / 16;       // vectors per row
  constexpr int PER = 16 * VPR / 32;  // vectors of a tile per lane
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kCompactThreads / 32) + (threadIdx.x >> 5);
  const int page = (int)(unit % a.warps_per_row);
  const long long row = unit / a.warps_per_row;
  const int h = (int)(row % a.Hkv);
  if (row / a.Hkv >= a.S) return;
  const int seq = (int)(row / a.Hkv);
  int kept = a.kept[seq];
  if (kept < 0 || kept > a.budget || kept > 16ll * a.dst_blocks) {
    if (lane == 0 && page == 0) record_error(a.err, PA_ERR_BOUNDS);
    kept = kept < 0 ? 0 : (int)min((long long)min(kept, a.budget), 16ll * a.dst_blocks);
  }
  // lane r < 16: where row r of the page comes from
  const int i = 16 * page + lane;
  const bool live = lane < 16 && i < kept;
  const int kh = a.keep_heads == 1 ? 0 : h;
  long long src = -1;  // row index (block * Hkv + h) * 16 + offset in the layer
  int dst = 0, tok = -1;
  if (16 * page < kept) {
    dst = a.dst_tables[(long long)seq * a.dst_blocks + page];
    bool bad = dst < 0 || dst >= a.num_blocks;
    if (live) {
      tok = a.keep[((long long)seq * a.keep_heads + kh) * a.budget + i];
      if (tok < 0 || tok >= 16ll * a.src_blocks) {
        bad = true;
      } else {
        const int b = a.src_tables[(long long)seq * a.src_blocks + (tok >> 4)];
        if (b < 0 || b >= a.num_blocks) bad = true;
        else if (!bad) src = ((long long)b * a.Hkv + h) * 16 + (tok & 15);
      }
    }
    if (bad) record_error(a.err, PA_ERR_BOUNDS);
    const long long dtile = ((long long)dst * a.Hkv + h) * 16;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint8_t* pool = which ? a.v : a.k;
      uint4 x[PER];
      long long from[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int vec = j * 32 + lane;
        from[j] = __shfl_sync(kAll, src, vec / VPR);
        x[j] = make_uint4(0, 0, 0, 0);
        if (from[j] >= 0) x[j] = *reinterpret_cast<const uint4*>(pool + from[j] * ROW + (vec % VPR) * 16);
      }
      if constexpr (BLK) {
        // the rows' values under their tiles' scales, one scale for the new tile
        float* sc = which ? a.vsc : a.ksc;
        float y[PER][16];
        uint32_t mb = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const float s = from[j] >= 0 ? sc[from[j] >> 4] : 0.f;
          const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(w[q], lo, hi);
            const float2 u0 = unpack2<false>(lo), u1 = unpack2<false>(hi);
            y[j][4 * q] = __fmul_rn(u0.x, s);
            y[j][4 * q + 1] = __fmul_rn(u0.y, s);
            y[j][4 * q + 2] = __fmul_rn(u1.x, s);
            y[j][4 * q + 3] = __fmul_rn(u1.y, s);
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) mb = max(mb, __float_as_uint(y[j][q]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mb = max(mb, __shfl_xor_sync(kAll, mb, off));
        const float s = __fdiv_rn(__uint_as_float(mb), 448.f);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float2 f = make_float2(0.f, 0.f);
            if (s > 0.f) f = make_float2(__fdiv_rn(y[j][2 * q], s), __fdiv_rn(y[j][2 * q + 1], s));
            w[q] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
          }
          x[j] = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
        }
        if (lane == 0 && dst >= 0 && dst < a.num_blocks) sc[dtile >> 4] = s;
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int vec = j * 32 + lane;
        if (from[j] >= 0) *reinterpret_cast<uint4*>(pool + (dtile + vec / VPR) * ROW + (vec % VPR) * 16) = x[j];
      }
    }
  }
  // ---- totals: of the page's tokens, and this warp's part of the zeros behind them
  if (a.w_in && kh == h) {
    const long long wrow = (long long)seq * a.keep_heads + kh;
    float* wo = a.w_out + wrow * a.w_out_stride;
    if (live && i < a.w_out_stride) {
      float w = 0.f;
      if (tok >= 0 && tok < a.w_in_stride) w = a.w_in[wrow * a.w_in_stride + tok];
      else record_error(a.err, PA_ERR_BOUNDS);
      wo[i] = w;
    } else if (live) {
      record_error(a.err, PA_ERR_BOUNDS);
    }
    const long long zeros = a.w_out_stride - kept;
    if (zeros > 0) {
      const long long each = (zeros + a.warps_per_row - 1) / a.warps_per_row;
      const long long z0 = kept + each * page, z1 = min(a.w_out_stride, z0 + each);
      for (long long z = z0 + lane; z < z1; z += 32) wo[z] = 0.f;
    }
  }
}

typedef void (*CompactKernel)(CompactArgs);

CompactKernel pick_compact(const pa_pool* pool) {
  const int row = pool->desc.head_dim * pool->elem_bytes;
  if (pool->block_scaled) return row == 64 ? compact_kernel<64, true> : compact_kernel<128, true>;
  return row == 64 ? compact_kernel<64, false> : row == 128 ? compact_kernel<128, false> : compact_kernel<256, false>;
}

template <int C>
cudaError_t launch_select(const SelectArgs& a, int smem, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(select_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.S * a.H * C);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<C>, a);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_evict_select(pa_pool* pool, const float* weights, size_t weights_stride, const int32_t* ctx_lens_dev, int S,
                    int n_heads, int budget, int sinks, int recent, int32_t* keep_dev, int32_t* kept_lens_dev,
                    void* stream) {
  pa::TraceRange trace_("pa_evict_select");
  if (!pool) return fail(PA_ERR_INVALID, "null pool");
  if (S < 0 || n_heads < 1) return fail(PA_ERR_INVALID, "need S >= 0 and n_heads >= 1");
  if (budget < 1 || budget > 0x7FFFFFFF - 1024 || sinks < 0 || recent < 0 || (long long)sinks + recent > budget)
    return fail(PA_ERR_INVALID, "need budget 1 to 2^31 - 1025, sinks >= 0, recent >= 0 and sinks + recent <= budget");
  if (weights_stride < 1 || weights_stride > 0x7FFFFFFF - 1024)
    return fail(PA_ERR_INVALID, "weights_stride must be 1 to 2^31 - 1025");
  if ((long long)S * n_heads > (1 << 27)) return fail(PA_ERR_UNSUPPORTED, "at most 2^27 rows per call");
  if (S == 0) return PA_OK;
  if (!weights || !ctx_lens_dev || !keep_dev || !kept_lens_dev) return fail(PA_ERR_INVALID, "null argument");
  if ((uintptr_t)weights & 15u) return fail(PA_ERR_INVALID, "weights must be 16-byte aligned");
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  SelectArgs a;
  a.w = weights;
  a.stride = (long long)weights_stride;
  a.ctx = ctx_lens_dev;
  a.S = S;
  a.H = n_heads;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.keep = keep_dev;
  a.kept = kept_lens_dev;
  a.err = err;
  // CTAs per row: one up to 8192 tokens, then enough that a share is at most
  // 16384 keys (64 KiB, three CTAs per SM), up to the portable cluster of eight.
  const long long tokens = a.stride;
  const int C = tokens <= 8192 ? 1 : tokens <= 32768 ? 2 : tokens <= 65536 ? 4 : 8;
  a.max_keys = (int)std::min<long long>(((tokens + C - 1) / C + 31) / 32 * 32, kSelMaxKeys);
  const int smem = a.max_keys * 4;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = C == 1   ? launch_select<1>(a, smem, st)
                        : C == 2 ? launch_select<2>(a, smem, st)
                        : C == 4 ? launch_select<4>(a, smem, st)
                                 : launch_select<8>(a, smem, st);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "evict_select launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

int pa_evict_compact(pa_pool* pool, int layer, const int32_t* keep_dev, int keep_heads, int budget,
                     const int32_t* kept_lens_dev, const int32_t* src_tables_dev, int src_max_blocks,
                     const int32_t* dst_tables_dev, int dst_max_blocks, int S, const float* weights_in,
                     size_t weights_in_stride, float* weights_out, size_t weights_out_stride, void* stream) {
  pa::TraceRange trace_("pa_evict_compact");
  int st = check_pool_layer(pool, layer);
  if (st) return st;
  const pa_pool_desc& d = pool->desc;
  if (keep_heads != 1 && keep_heads != d.n_kv_heads)
    return fail(PA_ERR_INVALID, "keep_heads must be 1 or n_kv_heads = %d (got %d)", d.n_kv_heads, keep_heads);
  if (S < 0 || budget < 1 || budget > 0x7FFFFFFF - 1024 || src_max_blocks < 1 || dst_max_blocks < 1)
    return fail(PA_ERR_INVALID, "need S >= 0, budget 1 to 2^31 - 1025 and tables of at least one block");
  if ((weights_in == nullptr) != (weights_out == nullptr))
    return fail(PA_ERR_INVALID, "weights_in and weights_out come together");
  if (weights_in && (weights_in == weights_out || weights_in_stride < 1 || weights_out_stride < 1 ||
                     weights_in_stride > 0x7FFFFFFF - 1024 || weights_out_stride > 0x7FFFFFFF - 1024))
    return fail(PA_ERR_INVALID, "the totals need two buffers and strides of 1 to 2^31 - 1025");
  if (S == 0) return PA_OK;
  if (!keep_dev || !kept_lens_dev || !src_tables_dev || !dst_tables_dev) return fail(PA_ERR_INVALID, "null argument");
  if (src_tables_dev == dst_tables_dev)
    return fail(PA_ERR_INVALID, "the destination table must name other blocks than the source table");
  if (((uintptr_t)weights_in | (uintptr_t)weights_out) & 15u)
    return fail(PA_ERR_INVALID, "the weights must be 16-byte aligned");
  // a row's warps: one per destination page, and enough that none zeroes more than 1024 totals
  long long per_row = (std::min<long long>(budget, 16ll * dst_max_blocks) + 15) / 16;
  if (weights_in) per_row = std::max<long long>(per_row, ((long long)weights_out_stride + 1023) / 1024);
  const long long warps = (long long)S * d.n_kv_heads * per_row;
  const long long ctas = (warps + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  if (per_row > 0x7FFFFFFF || ctas > 0x7FFFFFFF) return fail(PA_ERR_UNSUPPORTED, "too many pages for one call");
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  CompactArgs a;
  a.keep = keep_dev;
  a.keep_heads = keep_heads;
  a.budget = budget;
  a.kept = kept_lens_dev;
  a.src_tables = src_tables_dev;
  a.src_blocks = src_max_blocks;
  a.dst_tables = dst_tables_dev;
  a.dst_blocks = dst_max_blocks;
  a.S = S;
  a.Hkv = d.n_kv_heads;
  a.num_blocks = d.num_blocks;
  a.k = pool->k + (size_t)layer * pool->layer_bytes;
  a.v = pool->v + (size_t)layer * pool->layer_bytes;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  a.w_in = weights_in;
  a.w_in_stride = (long long)weights_in_stride;
  a.w_out = weights_out;
  a.w_out_stride = (long long)weights_out_stride;
  a.warps_per_row = (int)per_row;
  a.err = err;
  pick_compact(pool)<<<(unsigned)ctas, kCompactThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "evict_compact launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
