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
// (11, 11 and 10 bits of an order-preserving integer key, a histogram each),
// then one ordered pass writes what lies above it and the first of what equals
// it.  A row is shared by a cluster of CTAs, which hold its keys in shared
// memory (the row is read from HBM once) and add up their histograms through
// distributed shared memory.  Counts are integers, so the result depends on no
// order of execution.
//
// What bounds it is the instructions per key and the latency of the passes,
// not the 4 bytes per key.  The first digit holds the sign, the exponent and two
// bits of mantissa: wide enough that few keys share its bin with the k-th
// one, so the later passes only compare and skip.
constexpr int kSelBins = 2048;
constexpr int kSelMaxKeys = 49152;  // keys a CTA keeps (192 KiB); longer shares are read again in each pass

struct SelectArgs {
  const float* w;
  long long stride;
  const int32_t* ctx;
  int S, H;
  int budget, sinks, recent;
  int32_t* keep;
  int32_t* kept;
  int max_keys;  // keys of the CTA's dynamic shared memory, a multiple of 32
  unsigned int* err;
};

// Larger floats have larger keys; -0 counts as 0, NaN comes below every number.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Adds each lane's digit (those with `in`) to the histogram.  Totals crowd
// (all the tokens that nothing attends to share one bin), and a shared-memory
// atomic serialises on equal addresses: the lanes that agree with the first one
// are counted by a ballot, the rest add one by one.
__device__ __forceinline__ void hist_add(uint32_t* hist, uint32_t digit, bool in) {
  const unsigned all = __ballot_sync(kAll, in);
  if (!all) return;
  const int lead = __ffs(all) - 1;
  const uint32_t d = __shfl_sync(kAll, digit, lead);
  const unsigned same = __ballot_sync(kAll, in && digit == d);
  const int lane = threadIdx.x & 31;
  if (lane == lead) atomicAdd(&hist[d], (uint32_t)__popc(same));
  else if (in && digit != d) atomicAdd(&hist[digit], 1u);
}

template <int C>
__device__ __forceinline__ void row_sync() {
  if constexpr (C == 1) __syncthreads();
  else cg::this_cluster().sync();
}

// C CTAs of NT threads per row.  Single CTAs take 256 threads: with short rows
// the passes' latency counts, and six CTAs on an SM hide it better than three.
template <int C, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 2) select_kernel(const SelectArgs a) {
  constexpr int kSelThreads = NT, kSelWarps = NT / 32, BPT = kSelBins / NT;  // BPT: bins per thread
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[2][kSelBins];
  __shared__ uint32_t s_scan[kSelWarps];
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
  // keys i .. i + 3 of the share (i a multiple of 4); those from cnt on are anything
  auto keys4 = [&](int i) {
    if (i < a.max_keys) return *reinterpret_cast<const uint4*>(keys + i);
    uint4 v;
    v.x = i < cnt ? order_key(src[i]) : 0u;
    v.y = i + 1 < cnt ? order_key(src[i + 1]) : 0u;
    v.z = i + 2 < cnt ? order_key(src[i + 2]) : 0u;
    v.w = i + 3 < cnt ? order_key(src[i + 3]) : 0u;
    return v;
  };

  for (int i = tid; i < 2 * kSelBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  uint32_t prefix = 0;
  uint32_t rem = k;  // still to be taken among the keys that start with the prefix
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t* h = hist[p & 1];
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
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
          if (i0 + j * kSelThreads < cnt) hist_add(h, key >> 21, i < cnt);  // (uniform per CTA)
        }
      }
    } else {
      for (int i0 = 0; i0 < cnt; i0 += 4 * kSelThreads) {
        const int i = i0 + 4 * tid;
        const uint4 v = i < cnt ? keys4(i) : make_uint4(0, 0, 0, 0);
        const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          hist_add(h, (key[j] >> kShift[p]) & ((1u << kBits[p]) - 1u),
                   i + j < cnt && (key[j] >> (kShift[p] + kBits[p])) == prefix);
      }
    }
    row_sync<C>();  // every CTA's histogram is complete
    // the bins of the whole row from the top down, BPT per thread, and the one
    // that holds the rem-th key
    uint32_t c[BPT];
#pragma unroll
    for (int j = 0; j < BPT; ++j) c[j] = 0;
    const int b0 = kSelBins - BPT - BPT * tid;  // bins b0 + BPT - 1 down to b0
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint32_t* hr = h;
      if constexpr (C > 1) hr = cg::this_cluster().map_shared_rank(h, r);
#pragma unroll
      for (int j = 0; j < BPT; j += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(hr + b0 + BPT - 4 - j);
        c[j] += v.w;
        c[j + 1] += v.z;
        c[j + 2] += v.y;
        c[j + 3] += v.x;
      }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < BPT; ++j) mine += c[j];
    uint32_t x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    // the other buffer's readers passed the barrier above: clear it for the next digit
    if (p == 1)
      for (int i = tid; i < kSelBins / 4; i += NT) reinterpret_cast<uint4*>(hist[0])[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint32_t before = x - mine;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) before += w < warp ? s_scan[w] : 0u;
    if (before < rem && rem <= before + mine) {
      uint32_t at = before;
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        if (at < rem && rem <= at + c[j]) {
          s_digit = b0 + BPT - 1 - j;
          s_rem = rem - at;
        }
        at += c[j];
      }
    }
    __syncthreads();
    prefix = (prefix << kBits[p]) | s_digit;
    rem = s_rem;
  }

  // ---- above the threshold key, and equal to it: counts per warp, each warp
  // one stretch of the share
  const int seg = ((cnt + kSelWarps - 1) / kSelWarps + 127) / 128 * 128;
  const int w0 = min(cnt, warp * seg), w1 = min(cnt, w0 + seg);
  uint32_t above = 0, equal = 0;
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    const uint4 v = keys4(i);
    const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      above += i + j < w1 && key[j] > prefix;
      equal += i + j < w1 && key[j] == prefix;
    }
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
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint2 v = *cg::this_cluster().map_shared_rank(&s_cta, r);
      ga += r < rank ? v.x : 0;
      ge += r < rank ? v.y : 0;
    }
  }
  // ---- the taken tokens in order: all above, and the first rem of the equal ones.
  // A lane holds four neighbours; (above, equal) counts are scanned over the
  // warp in one word, at most 128 each.
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint4 v = i < w1 ? keys4(i) : make_uint4(0, 0, 0, 0);
    const uint32_t key[4] = {v.x, v.y, v.z, v.w};
    uint32_t f[4], own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = i + j < w1 ? (key[j] > prefix ? 1u : key[j] == prefix ? 0x10000u : 0u) : 0u;
      own += f[j];
    }
    uint32_t x = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, off);
      if (lane >= off) x += y;
    }
    const uint32_t sum = __shfl_sync(kAll, x, 31);
    x -= own;
    uint32_t ea = ga + (x & 0xFFFFu), ee = ge + (x >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (f[j] == 1u || (f[j] != 0u && ee < rem)) keep[a.sinks + ea + min(ee, rem)] = a.sinks + begin + i + j;
      ea += f[j] & 1u;
      ee += f[j] >> 16;
    }
    ga += sum & 0xFFFFu;
    ge += sum >> 16;
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
    if constexpr (!BLK) {
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
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int vec = j * 32 + lane;
          if (from[j] >= 0) *reinterpret_cast<uint4*>(pool + (dtile + vec / VPR) * ROW + (vec % VPR) * 16) = x[j];
        }
      }
    } else {
      // Lane r holds row r's K and V tile scales.  A tile's largest |value| is the
      // largest of its rows' largest codes under their scales (codes order like
      // their values), so it takes no conversion to fp32 per code; the new code
      // is the old one's value times the row's ratio of scales.
      float s_src[2] = {0.f, 0.f};
      if (src >= 0) {
        s_src[0] = a.ksc[src >> 4];
        s_src[1] = a.vsc[src >> 4];
      }
      uint4 x[2][PER];
      bool have[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int vec = j * 32 + lane;
        const long long from = __shfl_sync(kAll, src, vec / VPR);
        have[j] = from >= 0;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          x[which][j] = make_uint4(0, 0, 0, 0);
          if (have[j])
            x[which][j] = *reinterpret_cast<const uint4*>((which ? a.v : a.k) + from * ROW + (vec % VPR) * 16);
        }
      }
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint32_t c[PER][8];  // the codes as binary16 pairs
        uint32_t mb = 0;     // bits of the largest |value|
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const uint32_t w[4] = {x[which][j].x, x[which][j].y, x[which][j].z, x[which][j].w};
          __half2 top = __float2half2_rn(0.f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            e4m3x4_to_f16x2x2(w[q], c[j][2 * q], c[j][2 * q + 1]);
            top = __hmax2_nan(top, __habs2(*reinterpret_cast<__half2*>(&c[j][2 * q])));
            top = __hmax2_nan(top, __habs2(*reinterpret_cast<__half2*>(&c[j][2 * q + 1])));
          }
          const float2 t = __half22float2(top);
          const float s = __shfl_sync(kAll, s_src[which], (j * 32 + lane) / VPR);
          mb = max(mb, max(__float_as_uint(__fmul_rn(t.x, s)) & 0x7FFFFFFFu,
                           __float_as_uint(__fmul_rn(t.y, s)) & 0x7FFFFFFFu));
        }
        mb = __reduce_max_sync(kAll, mb);
        const float s = __fdiv_rn(__uint_as_float(mb), 448.f);
        // (a row of zeros may have any scale: its ratio is kept finite)
        const float ratio = s > 0.f ? fminf(__fdiv_rn(s_src[which], s), 0x1p100f) : 0.f;
        uint8_t* pool = which ? a.v : a.k;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int vec = j * 32 + lane;
          const float r = __shfl_sync(kAll, ratio, vec / VPR);
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float2 u = unpack2<false>(c[j][q]);
            w[q] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(u.x, r), __fmul_rn(u.y, r)), __NV_SATFINITE, __NV_E4M3);
          }
          if (have[j])
            *reinterpret_cast<uint4*>(pool + (dtile + vec / VPR) * ROW + (vec % VPR) * 16) =
                make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
        }
        if (lane == 0 && dst >= 0 && dst < a.num_blocks) (which ? a.vsc : a.ksc)[dtile >> 4] = s;
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
  constexpr int NT = C == 1 ? 256 : 512;
  if (smem > 24 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(select_kernel<C, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.S * a.H * C);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<C, NT>, a);
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
  const int smem = a.max_keys * 4;  // keys, besides the histograms' 16 KiB
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
