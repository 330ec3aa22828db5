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
#include <atomic>

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
// What bounds it is instructions per key and the latency of the passes, not the
// 4 bytes per key.  So keys go four at a time; the first digit holds the sign,
// the exponent and two bits of mantissa, wide enough that few keys share its bin
// with the k-th one; every key of the share has a value (the tokens that stay
// anyway above all others, places behind the context below all), so no pass
// tests where a key lies; and the bin search reads 64 sums of 32 bins from each
// CTA, then 32 bins.  32 rows of 131072 tokens: 21 us (their 17 MB would take 2.5
// at a copy's rate), with eight-bit digits and one key at a time 46; 512 rows of up to
// 4096: 10.3 us.
constexpr int kSelBins = 2048;
constexpr int kSelMaxKeys = 49152;  // keys a CTA keeps (192 KiB); longer shares are read again in each pass
constexpr uint32_t kKeyNone = 0u;            // behind the context
constexpr uint32_t kKeyNaN = 1u;             // below every number
constexpr uint32_t kKeyZero = 0x80000000u;
constexpr uint32_t kKeyStays = 0xFFFFFFFFu;  // first and last tokens

struct SelectArgs {
  const float* w;
  long long stride;
  const int32_t* ctx;
  int S, H;
  int budget, sinks, recent;
  int32_t* keep;
  int32_t* kept;
  int max_keys;  // keys of the CTA's dynamic shared memory, a multiple of 128
  int vec;       // rows are 16-byte aligned
  unsigned int* err;
};

// Larger floats have larger keys; -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return x == x ? k : kKeyNaN;
}

template <int C>
__device__ __forceinline__ void row_sync() {
  if constexpr (C == 1) __syncthreads();
  else cg::this_cluster().sync();
}

// p in CTA r of the row's cluster.
template <int C, typename T>
__device__ __forceinline__ const T* of_rank(T* p, int r) {
  if constexpr (C == 1) return p;
  else return cg::this_cluster().map_shared_rank(p, r);
}

// Inclusive sum over the lanes from the highest down.
__device__ __forceinline__ uint32_t scan_down(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_down_sync(kAll, x, off);
    if (lane + off < 32) x += y;
  }
  return x;
}

// C CTAs of NT threads per row.
template <int C, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 2) select_kernel(const SelectArgs a) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[2][kSelBins];
  __shared__ __align__(16) uint32_t sums[2][64];  // of 32 bins each
  __shared__ uint32_t s_digit, s_rem;
  __shared__ uint2 s_warp[NW];
  __shared__ uint2 s_cta, s_before;  // (above, equal): of this CTA's share, of the shares before it
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
    for (long long i = rank * NT + tid; i < a.budget; i += C * NT) keep[i] = i < n ? (int)i : -1;
    return;
  }

  // this CTA's share of the row: tokens [begin, begin + cnt), in groups of four
  const int chunk = ((n + C - 1) / C + 127) / 128 * 128;
  const int begin = (int)min((long long)n, (long long)rank * chunk), cnt = min(chunk, n - begin);
  const int groups = (cnt + 3) / 4;
  const int tail = n - a.recent - begin, head = a.sinks - begin;  // in the share: i < head or i >= tail stays
  const float* src = a.w + (long long)row * a.stride + begin;
  auto load_keys = [&](int i) {  // keys of tokens i .. i + 3 of the share
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.vec) {
      x = *reinterpret_cast<const float4*>(src + i);  // (the row's stride reaches past its last group)
    } else {
      x.x = src[i];
      if (i + 1 < cnt) x.y = src[i + 1];
      if (i + 2 < cnt) x.z = src[i + 2];
      if (i + 3 < cnt) x.w = src[i + 3];
    }
    uint4 k = make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
    if (i < head || i + 3 >= tail) {  // (tail <= cnt - recent: the share's end is behind it)
      uint32_t* e[4] = {&k.x, &k.y, &k.z, &k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j < head || i + j >= tail) *e[j] = kKeyStays;
        if (i + j >= cnt) *e[j] = kKeyNone;
      }
    }
    return k;
  };
  auto keys4 = [&](int i) { return i < a.max_keys ? *reinterpret_cast<const uint4*>(keys + i) : load_keys(i); };

  for (int i = tid; i < 2 * kSelBins / 4; i += NT) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  uint32_t prefix = 0;
  uint32_t rem = a.budget - a.sinks - a.recent;  // still to be taken among the keys that start with the prefix
  const bool search = rem > 0;                   // (else what stays anyway fills the budget)
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t* h = hist[p & 1];
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
    // Shared-memory atomics serialise on equal addresses, and one value is met by the
    // thousand: the zero of tokens that nothing attended to.  Each thread counts its
    // own; the rest spread over the bins.
    uint32_t zeros = 0;
    auto add = [&](uint32_t key) {
      const bool in = p == 0 ? key - 1u < kKeyStays - 1u : (key >> (kShift[p] + kBits[p])) == prefix;
      if (in && key != kKeyZero) atomicAdd(&h[(key >> kShift[p]) & ((1u << kBits[p]) - 1u)], 1u);
      zeros += key == kKeyZero;
    };
    if (p == 0) {
      constexpr int LD = NT == 256 ? 2 : 4;  // loads in flight per thread
      for (int g0 = tid; g0 < groups; g0 += LD * NT) {
        uint4 v[LD];
#pragma unroll
        for (int j = 0; j < LD; ++j)
          if (g0 + j * NT < groups) v[j] = load_keys(4 * (g0 + j * NT));
#pragma unroll
        for (int j = 0; j < LD; ++j)
          if (g0 + j * NT < groups) {
            const int i = 4 * (g0 + j * NT);
            if (i < a.max_keys) *reinterpret_cast<uint4*>(keys + i) = v[j];
            add(v[j].x);
            add(v[j].y);
            add(v[j].z);
            add(v[j].w);
          }
      }
    } else if (search) {
      for (int g = tid; g < groups; g += NT) {
        const uint4 v = keys4(4 * g);
        add(v.x);
        add(v.y);
        add(v.z);
        add(v.w);
      }
    }
    if (!search) continue;
    if (p == 0 || (kKeyZero >> (kShift[p] + kBits[p])) == prefix) {
      zeros = __reduce_add_sync(kAll, zeros);
      if (lane == 0 && zeros) atomicAdd(&h[(kKeyZero >> kShift[p]) & ((1u << kBits[p]) - 1u)], zeros);
    }
    __syncthreads();
    for (int b = 4 * tid; b < kSelBins; b += 4 * NT) {
      const uint4 v = *reinterpret_cast<const uint4*>(h + b);
      uint32_t x = v.x + v.y + v.z + v.w;
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) x += __shfl_xor_sync(kAll, x, off);
      if ((lane & 7) == 0) sums[p & 1][b / 32] = x;
    }
    row_sync<C>();  // every CTA's histogram is complete
    if (warp == 0) {
      uint2 c = make_uint2(0, 0);  // sums 2 lane, 2 lane + 1 of the whole row
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const uint2 v = *reinterpret_cast<const uint2*>(of_rank<C>(sums[p & 1], r) + 2 * lane);
        c.x += v.x;
        c.y += v.y;
      }
      uint32_t upto = scan_down(c.x + c.y), above = upto - c.x - c.y;
      // the sum that holds the rem-th key from above, and what lies above it
      const bool hi = above < rem && rem <= above + c.y, lo = above + c.y < rem && rem <= upto;
      const unsigned who = __ballot_sync(kAll, hi || lo);
      const int from = __ffs(who) - 1;
      const int bin32 = __shfl_sync(kAll, 2 * lane + (hi ? 1 : 0), from);
      const uint32_t left = rem - __shfl_sync(kAll, above + (hi ? 0 : c.y), from);
      uint32_t f = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) f += of_rank<C>(h, r)[32 * bin32 + lane];
      upto = scan_down(f);
      above = upto - f;
      if (above < left && left <= upto) {
        s_digit = 32 * bin32 + lane;
        s_rem = left - above;
      }
    } else if (p == 1) {
      // the first buffer's readers passed the barrier above: clear it for the last digit
      for (int i = tid - 32; i < kSelBins / 4; i += NT - 32) reinterpret_cast<uint4*>(hist[0])[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    prefix = (prefix << kBits[p]) | s_digit;
    rem = s_rem;
  }
  if (!search) {  // nothing but what stays anyway
    prefix = kKeyStays;
    rem = 1u << 31;
    __syncthreads();  // (the keys)
  }

  // ---- above the threshold key, and equal to it: counts per warp, each warp one
  // stretch of the share
  const int seg = ((groups + NW - 1) / NW + 31) / 32 * 32;
  const int w0 = min(groups, warp * seg), w1 = min(groups, w0 + seg);
  uint32_t above = 0, equal = 0;
  for (int g = w0 + lane; g < w1; g += 32) {
    const uint4 v = keys4(4 * g);
    above += (v.x > prefix) + (v.y > prefix) + (v.z > prefix) + (v.w > prefix);
    equal += (v.x == prefix) + (v.y == prefix) + (v.z == prefix) + (v.w == prefix);
  }
  above = __reduce_add_sync(kAll, above);
  equal = __reduce_add_sync(kAll, equal);
  if (lane == 0) s_warp[warp] = make_uint2(above, equal);
  __syncthreads();
  uint32_t ga = 0, ge = 0;  // before this warp's stretch
  {
    uint32_t ta = 0, te = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const uint2 v = s_warp[w];
      ga += w < warp ? v.x : 0;
      ge += w < warp ? v.y : 0;
      ta += v.x;
      te += v.y;
    }
    if constexpr (C > 1) {
      if (tid == 0) s_cta = make_uint2(ta, te);
      cg::this_cluster().sync();
      if (warp == 0) {
        uint2 v = make_uint2(0, 0);
        if (lane < rank) v = *of_rank<C>(&s_cta, lane);
        v.x = __reduce_add_sync(kAll, v.x);
        v.y = __reduce_add_sync(kAll, v.y);
        if (lane == 0) s_before = v;
      }
      __syncthreads();
      ga += s_before.x;
      ge += s_before.y;
      cg::this_cluster().barrier_arrive();  // this CTA reads no other's memory any more
    }
  }
  // ---- the taken tokens in order: all above, and the first rem of the equal ones.
  // A warp whose equal keys are all taken, or none, compares once per key.
  const bool mixed = ge < rem && ge + equal > rem;
  const uint32_t least = ge < rem ? prefix : prefix + 1u;  // (prefix + 1: only where some key lies above)
  const bool none = ge >= rem && prefix == kKeyStays;
  uint32_t at = ga + min(ge, rem);
  for (int g0 = w0; g0 < w1 && !none; g0 += 32) {
    const int g = g0 + lane;
    const uint4 v = g < w1 ? keys4(4 * g) : make_uint4(0, 0, 0, 0);
    uint32_t t[4];
    t[0] = v.x >= least;
    t[1] = v.y >= least;
    t[2] = v.z >= least;
    t[3] = v.w >= least;
    if (mixed) {  // (few warps: the one where the equal ones run out)
      const uint32_t e = (v.x == prefix) + (v.y == prefix) + (v.z == prefix) + (v.w == prefix);
      const uint32_t up = e + (scan_down(e) - e);  // this lane and those behind it
      uint32_t rank_e = ge + __shfl_sync(kAll, up, 0) - up;  // equal ones before this lane
      ge += __shfl_sync(kAll, up, 0);
      const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (key[j] == prefix) t[j] = rank_e++ < rem;
    }
    const uint32_t own = t[0] + t[1] + t[2] + t[3];
    uint32_t x = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, off);
      if (lane >= off) x += y;
    }
    int32_t* out = keep + at + (x - own);
    at += __shfl_sync(kAll, x, 31);
    const int tok = begin + 4 * g;
    if (t[0]) *out++ = tok;
    if (t[1]) *out++ = tok + 1;
    if (t[2]) *out++ = tok + 2;
    if (t[3]) *out = tok + 3;
  }
  if constexpr (C > 1) cg::this_cluster().barrier_wait();  // no CTA leaves while another may read its memory
}

// ---------------------------------------------------------------- compaction
// One warp per destination page of a (sequence, kv head): 16 rows, gathered
// from wherever they lie.  Lanes 0-15 resolve the rows' addresses; the rows
// then move as 16-byte vectors, all loads of a batch in flight before the
// first store.  Bound by HBM where rows are copied: 4 x 32768 of 131072 tokens,
// bf16 166 us (6.5 TB/s), FP8 87 us (6.2).  With a scale per tile 117 us, and 127
// with totals in rows of 131072: the conversions between the loads and the
// stores; 296 with a division per code.
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
  unsigned ctas_per_row;
  int pages_per_row;  // >= the destination pages of a row
  unsigned int* err;
};

constexpr int kCompactThreads = 256;

// ROW: bytes of one token row of a tile (64, 128 or 256).
template <int ROW, bool BLK>
__global__ void __launch_bounds__(kCompactThreads, BLK ? 4 : 5) compact_kernel(const CompactArgs a) {
  constexpr int VPR = ROW / 16;       // vectors per row
  constexpr int PER = 16 * VPR / 32;  // vectors of a tile per lane
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const unsigned row = blockIdx.x / a.ctas_per_row;
  const int unit = (int)(blockIdx.x - row * a.ctas_per_row) * (kCompactThreads / 32) + (int)(threadIdx.x >> 5);
  const int page = BLK ? unit >> 1 : unit, which_blk = BLK ? unit & 1 : 0;
  if (page >= a.pages_per_row) return;
  const int seq = (int)(row / (unsigned)a.Hkv), h = (int)(row - (unsigned)seq * a.Hkv);
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
  }
  // Totals of the page's tokens (loaded here, stored at the end) and this warp's part
  // of the zeros behind them.
  const bool totals = a.w_in && kh == h && which_blk == 0;
  float* wo = nullptr;
  float w = 0.f;
  if (totals) {
    const long long wrow = (long long)seq * a.keep_heads + kh;
    wo = a.w_out + wrow * a.w_out_stride;
    if (live) {
      if (tok >= 0 && tok < a.w_in_stride) w = a.w_in[wrow * a.w_in_stride + tok];
      if (tok < 0 || tok >= a.w_in_stride || i >= a.w_out_stride) record_error(a.err, PA_ERR_BOUNDS);
    }
    const long long zeros = a.w_out_stride - kept;
    if (zeros > 0) {
      const long long each = (zeros + a.pages_per_row - 1) / a.pages_per_row;
      const long long z0 = kept + each * page, z1 = min(a.w_out_stride, z0 + each);
      for (long long z = z0 + lane; z < z1; z += 32) wo[z] = 0.f;
    }
  }
  if (16 * page < kept) {
    const long long dtile = ((long long)dst * a.Hkv + h) * 16;
    if constexpr (!BLK) {
      // The 2 PER vectors of a lane, K's then V's, in batches of at most eight (128 bytes
      // a lane in flight; larger batches cost resident warps more than they gain).
      constexpr int BATCH = 2 * PER < 8 ? 2 * PER : 8;
#pragma unroll
      for (int m0 = 0; m0 < 2 * PER; m0 += BATCH) {
        uint4 x[BATCH];
        bool have[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int j = (m0 + b) % PER, vec = j * 32 + lane;
          const long long from = __shfl_sync(kAll, src, vec / VPR);
          have[b] = from >= 0;
          x[b] = make_uint4(0, 0, 0, 0);
          if (have[b]) x[b] = *reinterpret_cast<const uint4*>((m0 + b < PER ? a.k : a.v) + from * ROW + (vec % VPR) * 16);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int j = (m0 + b) % PER;
          if (have[b]) *reinterpret_cast<uint4*>((m0 + b < PER ? a.k : a.v) + dtile * ROW + lane * 16 + j * 512) = x[b];
        }
      }
    } else {
      // A warp for the K tile, one for the V tile.  Lane r holds row r's tile scale.
      // The new tile's largest |value| is the largest of its rows' largest codes under
      // their scales (codes order like their values), so it takes no conversion
      // to fp32 per code; the new code is the old one's value times the row's
      // ratio of scales.
      uint8_t* pool = which_blk ? a.v : a.k;
      float* scales = which_blk ? a.vsc : a.ksc;
      const float s_src = src >= 0 ? scales[src >> 4] : 0.f;
      uint4 x[PER];
      bool have[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int vec = j * 32 + lane;
        const long long from = __shfl_sync(kAll, src, vec / VPR);
        have[j] = from >= 0;
        x[j] = make_uint4(0, 0, 0, 0);
        if (have[j]) x[j] = *reinterpret_cast<const uint4*>(pool + from * ROW + (vec % VPR) * 16);
      }
      uint32_t c[PER][8];  // the codes as binary16 pairs
      uint32_t mb = 0;     // bits of the largest |value|
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        __half2 top = __float2half2_rn(0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          e4m3x4_to_f16x2x2(w[q], c[j][2 * q], c[j][2 * q + 1]);
          top = __hmax2_nan(top, __habs2(*reinterpret_cast<__half2*>(&c[j][2 * q])));
          top = __hmax2_nan(top, __habs2(*reinterpret_cast<__half2*>(&c[j][2 * q + 1])));
        }
        const float2 t = __half22float2(top);
        const float s = __shfl_sync(kAll, s_src, (j * 32 + lane) / VPR);
        mb = max(mb, max(__float_as_uint(__fmul_rn(t.x, s)) & 0x7FFFFFFFu,
                         __float_as_uint(__fmul_rn(t.y, s)) & 0x7FFFFFFFu));
      }
      mb = __reduce_max_sync(kAll, mb);
      const float s = __fdiv_rn(__uint_as_float(mb), 448.f);
      // (a row of zeros may have any scale: its ratio is kept finite)
      const float ratio = s > 0.f ? fminf(__fdiv_rn(s_src, s), 0x1p100f) : 0.f;
      uint8_t* out = pool + dtile * ROW + lane * 16;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float r = __shfl_sync(kAll, ratio, (j * 32 + lane) / VPR);
        uint32_t w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 u = unpack2<false>(c[j][q]);
          w[q] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(u.x, r), __fmul_rn(u.y, r)), __NV_SATFINITE, __NV_E4M3);
        }
        if (have[j])
          *reinterpret_cast<uint4*>(out + j * 512) =
              make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
      }
      if (lane == 0 && dst >= 0 && dst < a.num_blocks) scales[dtile >> 4] = s;
    }
  }
  if (totals && live && i < a.w_out_stride) wo[i] = w;
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
  static std::atomic<bool> opted[128];  // per device: more than 48 KiB of shared memory
  int dev = 0;
  if (smem > 24 * 1024 && (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128 || !opted[dev])) {
    const cudaError_t e =
        cudaFuncSetAttribute(select_kernel<C, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) opted[dev] = true;
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
  // 16384 keys (64 KiB; with the histograms' 16 two CTAs fit an SM), up to the portable
  // cluster of eight: past 131072 tokens the shares grow.
  const long long tokens = a.stride;
  const int C = tokens <= 8192 ? 1 : tokens <= 32768 ? 2 : tokens <= 65536 ? 4 : 8;
  a.max_keys = (int)std::min<long long>(((tokens + C - 1) / C + 127) / 128 * 128, kSelMaxKeys);
  a.vec = weights_stride % 4 == 0;
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
  // a row's pages: the destination's, and enough that no warp zeroes more than 1024 totals
  long long per_row = (std::min<long long>(budget, 16ll * dst_max_blocks) + 15) / 16;
  if (weights_in) per_row = std::max<long long>(per_row, ((long long)weights_out_stride + 1023) / 1024);
  const long long ctas_per_row = (per_row * (pool->block_scaled ? 2 : 1) + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  const long long ctas = (long long)S * d.n_kv_heads * ctas_per_row;
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
  a.ctas_per_row = (unsigned)ctas_per_row;
  a.pages_per_row = (int)per_row;
  a.err = err;
  pick_compact(pool)<<<(unsigned)ctas, kCompactThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "evict_compact launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
