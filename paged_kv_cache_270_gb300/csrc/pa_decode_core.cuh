// pa_decode_core.cuh -- what the decode kernels share: the shapes and argument
// block, the per-page step of a consumer warp, and the balanced-schedule
// kernel, of which pa_decode and pa_decode_weights have builds of their own.
// The design is described at the head of pa_decode.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"

namespace pa {

enum KvKind { KV_F16 = 0, KV_BF16 = 1, KV_E4M3 = 2, KV_E4M3B = 4 };  // KV_E4M3B: scale per tile
enum OutKind { OUT_F16 = 0, OUT_BF16 = 1, OUT_F32 = 3 };

constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr unsigned kFull = 0xffffffffu;

template <int KV, int D>
struct Cfg {
  static constexpr bool kFp8 = (KV == KV_E4M3) || (KV == KV_E4M3B);
  static constexpr bool kBlockScaled = (KV == KV_E4M3B);
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;    // one token row of a tile
  static constexpr int kTile = 16 * kRowBytes;   // bytes of one (block, kv head) tile
  // Rows of 128 or 256 bytes are loaded with 128-byte TMA swizzling, which
  // makes every shared-memory read of the consumers below bank-conflict free.
  static constexpr bool kSwizzle = (kRowBytes % 128) == 0;
  static constexpr int kTmaRank = kRowBytes == 256 ? 3 : 2;
  static constexpr int kStages = 8;
  // Consumer warp w takes pages w, w + 4, ...; with a stage count that is a
  // multiple of the warp count, the previous page of a stage is the same
  // warp's, so a warp waits on a full barrier at most one phase behind (the
  // parity wait cannot tell phases further apart).
  static_assert(kStages % kConsumerWarps == 0, "stages must be a multiple of the consumer warps");
  static constexpr int kStageBytes = 2 * kTile;  // K tile + V tile
  static constexpr int kRingBytes = kStages * kStageBytes;
  // merge area: per warp, 8 heads x (D + 4) floats (the pad spreads a warp's
  // stores over all banks) plus (m, l) per head
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMergeBytes = kConsumerWarps * 8 * (kMergeStride + 2) * 4;
  static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kAlign = 1024;  // a 128-byte-swizzled TMA destination is 1 KiB aligned
  // FP8 pools keep the query fragments in shared memory instead of 16 registers
  // per thread ([warp][D/16 pairs][32 lanes] x 8 bytes), which lets five CTAs
  // share an SM; 16-bit pools are limited by their ring size anyway.
  static constexpr bool kQInSmem = kFp8;
  static constexpr int kQBytes = kQInSmem ? kConsumerWarps * (D / 16) * 32 * 8 : 0;
  // block-scaled pools: the (K, V) scales of the page in each stage
  static constexpr int kScaleBytes = kBlockScaled ? kStages * 8 : 0;
  static constexpr int kSmem = kDataBytes + 2 * kStages * 8 + kQBytes + kScaleBytes + kAlign;
  // register budget, in CTAs per SM (16-bit pools: what their ring size allows).
  // Block-scaled FP8 spills a little at five, so it has a second build for four
  // (kMinBlocksLow), taken by launches that put at most four CTAs on an SM.
  static constexpr int kMinBlocks = kQInSmem ? 5 : (D == 128 ? 3 : 4);
  static constexpr int kMinBlocksLow = kBlockScaled ? 4 : kMinBlocks;
  static constexpr bool kMmaBf16 = (KV == KV_BF16);
  static_assert(kStageBytes % kAlign == 0 || !kSwizzle, "tiles must stay 1 KiB aligned");
};

// The balanced schedule gives every CTA at least this many pages.
constexpr int kMinPagesPerCta = 8;

// Fixed splits: how a sequence's pages are cut.  Uniform: split k covers pages
// [k pps, (k + 1) pps).  Guided (the automatic layout of launches of several
// waves): split k covers [b[k], b[k + 1]), sizes falling geometrically, and
// the split index is the slowest grid dimension, so the block scheduler hands
// out every sequence's first (largest) split first and the small last splits
// last: the CTAs still running as the grid drains are short ones.
constexpr int kGuidedSplits = 8;
struct SplitLayout {
  int splits, pps;
  int guided;
  int b[kGuidedSplits + 1];
};

struct DecodeArgs {
  const uint16_t* q;     // [S][Hq][D]
  void* out;             // [S][Hq][D]
  // split partials.  Fixed splits: [S][Hq][splits][D] and [S][Hq][splits][2]
  // (m in log2 units, l).  Balanced schedule: [2 * ctas][G][D] and [2 * ctas][G][2].
  float* ws_o;
  float* ws_ml;
  int4* jobs;            // balanced schedule: [ctas] merge jobs (sequence, kv head, last CTA, slot)
  const int32_t* tables;
  const int32_t* ctx;
  int max_blocks;
  int S, Hq, Hkv, G, num_blocks;
  int splits, pages_per_split;  // fixed splits (uniform layout)
  SplitLayout sl;               // fixed splits: the layout (uniform or guided)
  int ctas;                     // balanced schedule: CTAs of the launch
  float qk_scale_log2;  // softmax_scale * log2(e) (* k_scale for FP8)
  float v_scale;        // 1 for 16-bit and block-scaled pools
  const float* ksc;     // block-scaled pools: this layer's scales [num_blocks][Hkv]
  const float* vsc;
  unsigned int* err;
  // the scored build (pa_decode_weights): every token's scores, fp32
  // [S][Hkv][max_blocks * 16][gs] in log2 units, each CTA's range of the
  // schedule [ctas], and the running totals [S][Hkv][w_stride]
  float* scores;
  struct RangeStart* ranges;
  int gs;     // G, or the next even number (8-byte stores)
  int whole;  // a CTA takes whole units (every unit costs 1), so none is left over
  const float* w_in;  // nullptr: zeros
  float* w_out;
  long long w_stride;
  float decay;
};

// Where a CTA's range of the balanced schedule starts: position pos_begin lies in
// sequence seq, whose units start at position cost; positions per CTA and in all.
struct RangeStart {
  int seq, pad;
  long long pos_begin, pos_end, cost, T;
};

__device__ __forceinline__ int clamp_ctx(int c, int max_blocks) { return c < 0 ? 0 : min(c, max_blocks * 16); }

// Pages [pb, pe) of split k (the guided bounds are read with constant indices,
// so the layout stays in the parameter space).
__device__ __forceinline__ void split_pages(const SplitLayout& L, int k, int& pb, int& pe) {
  if (L.guided) {
    pb = 0;
    pe = 0;
#pragma unroll
    for (int i = 0; i < kGuidedSplits; ++i)
      if (i == k) {
        pb = L.b[i];
        pe = L.b[i + 1];
      }
  } else {
    pb = k * L.pps;
    pe = pb + L.pps;
  }
}
__device__ __forceinline__ int first_split_pages(const SplitLayout& L) { return L.guided ? L.b[1] : L.pps; }


// Exclusive prefix sum over the CTA's threads (every thread must call it);
// `total` receives the sum over all of them.
template <int NTHREADS>
__device__ __forceinline__ long long block_exclusive_scan(long long v, long long* warp_sums,
                                                          long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NTHREADS / 32; ++w) {
    const long long s = warp_sums[w];
    before += w < warp ? s : 0;
    total += s;
  }
  return before + x - v;
}

template <int OUT>
__device__ __forceinline__ void store_out(void* out, size_t idx, float v) {
  if constexpr (OUT == OUT_F32) {
    static_cast<float*>(out)[idx] = v;
  } else if constexpr (OUT == OUT_BF16) {
    static_cast<__nv_bfloat16*>(out)[idx] = __float2bfloat16_rn(v);
  } else {
    static_cast<__half*>(out)[idx] = __float2half_rn(v);
  }
}

// Loads the K or V tile of `row0` (= (block * Hkv + head) * 16) through the map.
template <int RANK>
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* map, int row0,
                                          uint64_t* bar, uint64_t policy) {
  if constexpr (RANK == 3) tma_load_3d(dst, map, 0, 0, row0, bar, policy);
  else tma_load_2d(dst, map, 0, row0, bar, policy);
}

template <bool SWZ>
__device__ __forceinline__ uint32_t tile_off(uint32_t off) {
  if constexpr (SWZ) return swizzle128(off);
  else return off;
}

// The largest first + i * step below end, i >= 0 (below first if there is none).
__device__ __forceinline__ int last_round(int first, int end, int step) {
  return end > first ? first + (end - 1 - first) / step * step : first - step;
}

// Stores two floats that are read again soon: L2 is asked to keep the line.
__device__ __forceinline__ void store_kept(float* p, float a, float b) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(p), "f"(a), "f"(b), "l"(policy) : "memory");
}

// Drops a warp's round of scores from L2 once its lanes have used them: bytes
// [0, bytes) at p (128-byte aligned; whole lines only, one per lane at a time)
// need no write-back to HBM, for nothing reads them again.
__device__ __forceinline__ void drop_lines(const float* p, int bytes) {
  __syncwarp();
  for (int at = 128 * (threadIdx.x & 31); at + 128 <= bytes; at += 32 * 128)
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(reinterpret_cast<const uint8_t*>(p) + at) : "memory");
}

// Turns the scores of tokens [t0, t1) of a unit (t0 a multiple of 16) into
// weights, sum over heads of 2^(x - M) / L, and adds them to the totals.  ml:
// (M, 1 / L) of the gs heads, (0, 0) for a padding one, whose scores are 0.  Called
// by NT threads.
// With eight heads two lanes share a token (16-byte loads, 512 contiguous bytes
// per warp instruction) and swap halves, so each lane writes one token of two
// load rounds; with four heads a lane holds a token; other groups are loaded as
// pairs of heads.  The score loads of a round (UNR x 64 or UNR x 128 tokens per
// warp) are all issued before the first use: the pass is bound by their latency.
template <int NT, int UNR>
__device__ __forceinline__ void add_weights(const float* sc, int gs, const float2* ml, const float* wi, float* wo,
                                            float decay, int t0, int t1) {
  constexpr int NW = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (gs == 8) {
    float M[4], inv[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float2 v = ml[4 * (lane & 1) + g];
      M[g] = v.x;
      inv[g] = v.y;
    }
    const float4* s4 = reinterpret_cast<const float4*>(sc);
    // from the last round back: the scores written last are the likeliest to be in L2
    for (int base = last_round(t0 + warp * 64 * UNR, t1, NW * 64 * UNR); base >= t0; base -= NW * 64 * UNR) {
      float4 x[4 * UNR];
      float w[2 * UNR];
#pragma unroll
      for (int j = 0; j < 4 * UNR; ++j) {
        const int t = base + 16 * j + (lane >> 1);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < t1) x[j] = __ldcg(s4 + 2 * (size_t)t + (lane & 1));
      }
#pragma unroll
      for (int j = 0; j < 2 * UNR; ++j) {  // even lanes write round 2j, odd ones round 2j + 1
        const int t = base + 16 * (2 * j + (lane & 1)) + (lane >> 1);
        w[j] = wi && t < t1 ? decay * wi[t] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 2 * UNR; ++j) {
        float p[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float4 v = x[2 * j + r];
          p[r] = fast_exp2(v.x - M[0]) * inv[0] + fast_exp2(v.y - M[1]) * inv[1] + fast_exp2(v.z - M[2]) * inv[2] +
                 fast_exp2(v.w - M[3]) * inv[3];
        }
        const float other = __shfl_xor_sync(kFull, lane & 1 ? p[0] : p[1], 1);
        const int t = base + 16 * (2 * j + (lane & 1)) + (lane >> 1);
        // (the even lane's heads first, for either lane's token)
        const float sum = lane & 1 ? other + p[1] : p[0] + other;
        if (t < t1) wo[t] = w[j] + sum;
      }
      drop_lines(sc + (size_t)base * 8, min(64 * UNR, (t1 - base + 15) & ~15) * 32);
    }
  } else if (gs == 4) {
    const float2 m0 = ml[0], m1 = ml[1], m2 = ml[2], m3 = ml[3];
    const float4* s4 = reinterpret_cast<const float4*>(sc);
    for (int base = last_round(t0 + warp * 128 * UNR, t1, NW * 128 * UNR); base >= t0; base -= NW * 128 * UNR) {
      float4 x[4 * UNR];
      float w[4 * UNR];
#pragma unroll
      for (int j = 0; j < 4 * UNR; ++j) {
        const int t = base + 32 * j + lane;
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < t1) x[j] = __ldcg(s4 + t);
        w[j] = wi && t < t1 ? decay * wi[t] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4 * UNR; ++j) {
        const int t = base + 32 * j + lane;
        const float p = fast_exp2(x[j].x - m0.x) * m0.y + fast_exp2(x[j].y - m1.x) * m1.y +
                        fast_exp2(x[j].z - m2.x) * m2.y + fast_exp2(x[j].w - m3.x) * m3.y;
        if (t < t1) wo[t] = w[j] + p;
      }
      drop_lines(sc + (size_t)base * 4, min(128 * UNR, (t1 - base + 15) & ~15) * 16);
    }
  } else if (gs == 1) {
    const float2 m = ml[0];
    for (int base = t0 + warp * 128; base < t1; base += NW * 128) {
      float x[4], w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = base + 32 * j + lane;
        x[j] = t < t1 ? __ldcg(sc + t) : 0.f;
        w[j] = wi && t < t1 ? decay * wi[t] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = base + 32 * j + lane;
        if (t < t1) wo[t] = w[j] + fast_exp2(x[j] - m.x) * m.y;
      }
    }
  } else {  // two or six heads
    for (int base = t0 + warp * 64; base < t1; base += NW * 64) {
      float2 x[2][3];
      float w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = base + 32 * j + lane;
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          x[j][g] = make_float2(0.f, 0.f);
          if (t < t1 && 2 * g < gs) x[j][g] = __ldcg(reinterpret_cast<const float2*>(sc + (size_t)t * gs) + g);
        }
        w[j] = wi && t < t1 ? decay * wi[t] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = base + 32 * j + lane;
        float p = 0.f;
#pragma unroll
        for (int g = 0; g < 3; ++g)
          if (2 * g < gs)
            p += fast_exp2(x[j][g].x - ml[2 * g].x) * ml[2 * g].y + fast_exp2(x[j][g].y - ml[2 * g + 1].x) * ml[2 * g + 1].y;
        if (t < t1) wo[t] = w[j] + p;
      }
    }
  }
}

// The tokens of a unit's pages up to `end` that have a place in a totals row.
__device__ __forceinline__ int totals_end(int end, const DecodeArgs& a) {
  if (end <= a.w_stride) return end;
  if (threadIdx.x == 0) record_error(a.err, PA_ERR_BOUNDS);
  return (int)a.w_stride;
}

// One page of a consumer warp: S^T = K_page . Q^T for the group, the online
// softmax update of (m, l) and the rescale of O, then O^T += V_page^T . P^T.
// The product with V takes P in V's 16-bit type, as it is rounded to that (2^-12 of
// a weight in binary16, 2^-9 in bfloat16), or with PSPLIT as the sum of that
// and what the rounding dropped, in a second product (2^-22, 2^-17): bfloat16
// pools, fp32 outputs and pa_decode_weights.  Row sums and maxima are fp32.
// Ks, Vs: the page's K and V tiles in shared memory; tok0: its first token;
// sc: its (K, V) tile scales (block-scaled pools).  SC: the page's scores are
// also stored, at score [16 tokens][gs heads] (behind the context: -inf), of the
// group's `heads`; the place of a head that an odd group lacks gets 0, whatever the
// key (its product with the absent query is NaN where the key is infinite).
template <int KV, int D, bool PSPLIT, bool SC = false>
__device__ __forceinline__ void consume_page(const uint8_t* Ks, const uint8_t* Vs, int tok0, int ctx,
                                             float qk_scale, const uint32_t (&qf)[D / 8],
                                             const uint2* qsm, const float2* sc, float& m0, float& m1,
                                             float& l0, float& l1, float (&o)[D / 16][4], float& vinv,
                                             float* score = nullptr, int gs = 0, int heads = 0) {
  using C = Cfg<KV, D>;
  constexpr bool BF = C::kMmaBf16;
  constexpr bool SWZ = C::kSwizzle;
  constexpr bool F8 = C::kFp8;
  constexpr bool BLK = C::kBlockScaled;
  constexpr int NT = D / 16;
  constexpr bool LDT = F8 && SWZ;
  constexpr bool LD16 = !F8 && SWZ;
  constexpr int KB = D / 4 * C::kElem;  // K bytes per row per thread
  constexpr int VB = D / 8 * C::kElem;  // V bytes per row per thread
  constexpr int RB = C::kRowBytes;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // ---- issue every shared-memory read of the page up front
    // The page's 16 tokens are taken in a fixed order lambda = 0..15 (the rows
    // of S^T and the K index of P V).  The transposed-ldmatrix path hands each
    // thread tokens 4t .. 4t+3 of a V column, so there lambda = 2t, 2t+1,
    // 2t+8, 2t+9 are the tokens 4t .. 4t+3, and the accumulator rows g, g+8
    // read K rows 2g - (g & 1) and that + 2; otherwise lambda is the token.
    constexpr int VW = VB / 4;  // V words per row per thread
    const int rows[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
    const int kg0 = LDT ? 2 * g - (g & 1) : g, kg1 = LDT ? kg0 + 2 : g + 8;
    uint4 kr[2][KB / 16];
    uint32_t vw[4][VW];
    uint32_t vt[NT][2];  // LDT: V codes, tokens 4t .. 4t+3 of dims 16i + g and 16i + g + 8
    // LD16: V pairs, tokens (2t, 2t+1) of dims 16i + g, 16i + g + 8, then tokens (2t+8, 2t+9)
    uint32_t vh[NT][4];
    {
#pragma unroll
      for (int c = 0; c < KB / 16; ++c) {
        kr[0][c] = lds128(Ks + tile_off<SWZ>(kg0 * RB + t * KB + 16 * c));
        kr[1][c] = lds128(Ks + tile_off<SWZ>(kg1 * RB + t * KB + 16 * c));
      }
      if constexpr (LDT) {
#pragma unroll
        for (int i = 0; i < NT; i += 2)
          ldsm_x2_trans_b8(Vs + tile_off<SWZ>((lane & 15) * RB + 16 * (i + (lane >> 4))), vt[i][0], vt[i][1],
                           vt[i + 1][0], vt[i + 1][1]);
      } else if constexpr (LD16) {
        // matrix m of m-tile i: tokens 8 (m >> 1) .. +7, dims 16i + 8 (m & 1) .. +7
        const uint32_t vrow = ((lane & 7) + ((lane >> 4) << 3)) * RB + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          ldsm_x4_trans_b16(Vs + tile_off<SWZ>(vrow + 32 * i), vh[i][0], vh[i][1], vh[i][2], vh[i][3]);
      } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t vo = rows[r] * RB + g * VB;
        if constexpr (VB == 8) {
          const uint2 u = lds64(Vs + tile_off<SWZ>(vo));
          vw[r][0] = u.x;
          vw[r][1] = u.y;
        } else {
#pragma unroll
          for (int c = 0; c < VB / 16; ++c) {
            const uint4 u = lds128(Vs + tile_off<SWZ>(vo + 16 * c));
            vw[r][4 * c] = u.x;
            vw[r][4 * c + 1] = u.y;
            vw[r][4 * c + 2] = u.z;
            vw[r][4 * c + 3] = u.w;
          }
        }
      }
      }
    }

    // ---- S^T[token][head] = K_page . Q^T
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < KB / 16; ++c) {
      const uint4 r0 = kr[0][c], r1 = kr[1][c];
      if constexpr (F8) {
        const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w};
        const uint32_t w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int j = 4 * c + jj;
          uint32_t af[4];
          e4m3x4_to_f16x2x2(w0[jj], af[0], af[2]);
          e4m3x4_to_f16x2x2(w1[jj], af[1], af[3]);
          const uint2 qj = qsm[j * 32 + lane];
          mma16816<false>(s, af, qj.x, qj.y);
        }
      } else {
        const uint32_t a0[4] = {r0.x, r1.x, r0.y, r1.y};
        mma16816<BF>(s, a0, qf[4 * c], qf[4 * c + 1]);
        const uint32_t a1[4] = {r0.z, r1.z, r0.w, r1.w};
        mma16816<BF>(s, a1, qf[4 * c + 2], qf[4 * c + 3]);
      }
    }

    // ---- online softmax over this page (tokens g and g+8; heads 2t, 2t+1)
    const float qks = BLK ? qk_scale * sc[0].x : qk_scale;
    float x0 = s[0] * qks, x1 = s[1] * qks;
    float x2 = s[2] * qks, x3 = s[3] * qks;
    if (tok0 + 16 > ctx) {  // last, partial page (warp-uniform): slots past ctx hold anything
      if (tok0 + kg0 >= ctx) x0 = x1 = -INFINITY;
      if (tok0 + kg1 >= ctx) x2 = x3 = -INFINITY;
      if constexpr (LDT) {
        const int nv = ctx - tok0 - 4 * t;  // valid tokens among this thread's 4
        const uint32_t keep = nv >= 4 ? 0xFFFFFFFFu : (nv <= 0 ? 0u : (1u << (8 * nv)) - 1u);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          vt[i][0] &= keep;
          vt[i][1] &= keep;
        }
      } else if constexpr (LD16) {
        const int r0 = ctx - tok0 - 2 * t;  // tokens 2t, 2t+1 valid when r0 > 0, r0 > 1
        const uint32_t klo = (r0 > 0 ? 0x0000FFFFu : 0u) | (r0 > 1 ? 0xFFFF0000u : 0u);
        const uint32_t khi = (r0 > 8 ? 0x0000FFFFu : 0u) | (r0 > 9 ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          vh[i][0] &= klo;
          vh[i][1] &= klo;
          vh[i][2] &= khi;
          vh[i][3] &= khi;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tok0 + rows[r] >= ctx) {
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[r][w] = 0u;
          }
      }
    }
    if constexpr (SC) {  // heads 2t, 2t + 1 of tokens kg0 and kg1
      if (gs == 1) {
        if (t == 0) {
          score[kg0] = x0;
          score[kg1] = x2;
        }
      } else if (2 * t < gs) {
        const bool pair = 2 * t + 1 < heads;
        store_kept(score + kg0 * gs + 2 * t, x0, pair ? x1 : 0.f);
        store_kept(score + kg1 * gs + 2 * t, x2, pair ? x3 : 0.f);
      }
    }
    float pm0 = fmaxf(x0, x2), pm1 = fmaxf(x1, x3);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      pm0 = fmaxf(pm0, __shfl_xor_sync(kFull, pm0, off));
      pm1 = fmaxf(pm1, __shfl_xor_sync(kFull, pm1, off));
    }
    // token 0 of every page is valid, so the new maxima are finite
    const float mn0 = fmaxf(m0, pm0), mn1 = fmaxf(m1, pm1);
    // warp-uniform: one scale per page; sv * (1 / vref) > 1 is sv > vref, also
    // for vref = 0 (inf > 1, and 0 * inf is NaN, not > 1)
    const bool vgrow = BLK && sc[0].y * vinv > 1.f;
    if (__any_sync(kFull, (mn0 != m0) | (mn1 != m1)) || vgrow) {  // rescale only when needed
      const float al0 = fast_exp2(m0 - mn0), al1 = fast_exp2(m1 - mn1);
      l0 *= al0;
      l1 *= al1;
      float ov0 = al0, ov1 = al1;
      if constexpr (BLK) {
        if (vgrow) {
          const float sv = sc[0].y;
          const float r = 1.f / (vinv * sv);  // vref / sv: 0 on the first page with a nonzero scale
          ov0 *= r;
          ov1 *= r;
          vinv = 1.f / sv;
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        o[i][0] *= ov0;
        o[i][1] *= ov1;
        o[i][2] *= ov0;
        o[i][3] *= ov1;
      }
      m0 = mn0;
      m1 = mn1;
    }
    float p0 = fast_exp2(x0 - m0), p1 = fast_exp2(x1 - m1);
    float p2 = fast_exp2(x2 - m0), p3 = fast_exp2(x3 - m1);
    l0 += p0 + p2;
    l1 += p1 + p3;
    if constexpr (BLK) {  // weights of this page's V codes: P * sv / vref
      const float f = sc[0].y * vinv;
      p0 *= f;
      p1 *= f;
      p2 *= f;
      p3 *= f;
    }

    // ---- P^T as the B operand: rows (tokens 2t, 2t+1 | 2t+8, 2t+9), column head g
    const uint32_t plo = pack2<BF>(p0, p1), phi = pack2<BF>(p2, p3);
    const uint32_t pb0 = movmatrix_trans(plo), pb1 = movmatrix_trans(phi);
    uint32_t rb0 = 0, rb1 = 0;
    if constexpr (PSPLIT) {
      const float2 u0 = unpack2<BF>(plo), u1 = unpack2<BF>(phi);
      rb0 = movmatrix_trans(pack2<BF>(p0 - u0.x, p1 - u0.y));
      rb1 = movmatrix_trans(pack2<BF>(p2 - u1.x, p3 - u1.y));
    }

    // ---- O^T[dim][head] += V_page^T . P^T
    {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint32_t af[4];
        if constexpr (LDT) {
          e4m3x4_to_f16x2x2(vt[i][0], af[0], af[2]);
          e4m3x4_to_f16x2x2(vt[i][1], af[1], af[3]);
        } else if constexpr (LD16) {
          af[0] = vh[i][0];
          af[1] = vh[i][1];
          af[2] = vh[i][2];
          af[3] = vh[i][3];
        } else if constexpr (F8) {
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          const uint32_t x01 = __byte_perm(vw[0][i >> 1], vw[1][i >> 1], sel);
          const uint32_t x23 = __byte_perm(vw[2][i >> 1], vw[3][i >> 1], sel);
          e4m3x4_to_f16x2x2(x01, af[0], af[1]);
          e4m3x4_to_f16x2x2(x23, af[2], af[3]);
        } else {
          af[0] = __byte_perm(vw[0][i], vw[1][i], 0x5410u);
          af[1] = __byte_perm(vw[0][i], vw[1][i], 0x7632u);
          af[2] = __byte_perm(vw[2][i], vw[3][i], 0x5410u);
          af[3] = __byte_perm(vw[2][i], vw[3][i], 0x7632u);
        }
        mma16816<BF>(o[i], af, pb0, pb1);
        if constexpr (PSPLIT) mma16816<BF>(o[i], af, rb0, rb1);
      }
    }
}

// ---------------------------------------------------------------- balanced schedule
// Shared memory of the balanced kernel: the ring and its barriers as in the
// fixed-split kernel, then the per-warp query fragments (FP8 pools), the merge
// slots, the staged query rows of the next unit with its descriptor, and the
// (m, l) exchange of the four warps.
template <int KV, int D>
struct BalCfg {
  using C = Cfg<KV, D>;
  static constexpr int kSlotBytes = 8 * D * 4;      // [8 heads][D] fp32
  // FP8 pools merge through two slots that alias the per-warp query fragments
  // (dead once a unit's last page is done); 16-bit pools keep their fragments
  // in registers and have one slot of their own.
  static constexpr int kMergeSlots = C::kQInSmem ? 2 : 1;
  static_assert(!C::kQInSmem || C::kQBytes == 2 * kSlotBytes, "two merge slots fill the fragment area");
  static constexpr int kOffBars = C::kRingBytes;    // full[S], empty[S], q_full, q_empty
  static constexpr int kOffFrag = kOffBars + (2 * C::kStages + 2) * 8;
  static constexpr int kFragBytes = C::kQInSmem ? C::kQBytes : kSlotBytes;
  static constexpr int kOffQStage = kOffFrag + kFragBytes;  // raw query rows [<= 8][D] (16-bit)
  static constexpr int kOffMl = kOffQStage + 8 * D * 2;     // [4 warps][8 heads] (m, l)
  static constexpr int kOffDesc = kOffMl + kConsumerWarps * 8 * 8;
  // the staged unit's descriptor, then each consumer warp's copy of its current one
  static constexpr int kOffScale = kOffDesc + (1 + kConsumerWarps) * 32;  // block-scaled: [stages] scales
  static constexpr int kSmem = kOffScale + C::kScaleBytes + C::kAlign;
  // The launch asks for at least 48 KiB, so at most four CTAs share an SM
  // (five would need 5 x (48 + 1) KiB, more than the SM's 228 KiB).  The grid
  // is four CTAs per SM with equal page counts; a build that fits five would
  // let the block scheduler put five on some SMs and three on others whenever
  // other work holds part of the GPU as the grid starts (a dependent launch
  // starts before the kernel ahead of it has finished), and the CTAs of a
  // five-CTA SM stream 4/5 as fast, which sets the time of the whole grid.
  static constexpr int kLaunchSmem = kSmem > 48 * 1024 ? kSmem : 48 * 1024;
  // What finishing a unit costs a CTA, in page-times (per-unit traces of a
  // batch of 28-page units: ~3-4 us for the merge, the output rows and the next
  // unit's start, against ~0.3 us a page for FP8 and about twice that for
  // 16-bit pages).
  static constexpr int kUnitCostPages = C::kFp8 ? 12 : 6;
  static_assert(kOffFrag % 16 == 0 && kOffQStage % 16 == 0, "bulk-copy destinations are 16-byte aligned");
};

// The unit the producer hands to the consumers with its query rows.
struct SegDesc {
  int seq, h, pg0, len, ctx, npages, last_cta;
};

// Bounded wait that also gives up once another thread of the CTA has raised
// the abort flag; a wait that runs out raises it and records PA_ERR_TIMEOUT.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              unsigned int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > pipe_wait_limit()) {
      *abort_flag = 1;
      record_error(err, PA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void consumers_sync() {  // the four consumer warps only
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumerWarps * 32) : "memory");
}

// Balanced schedule.  The grid is one CTA per resident slot.  Every CTA adds
// up the pages of all (sequence, kv head) units from the context lengths on
// the device; the units' pages, in (sequence, kv head, page) order, are cut
// into equal contiguous ranges, one per CTA.  A range crosses unit
// boundaries without draining the pipeline: the producer streams the pages
// of one unit after the other, and ahead of each unit it stages the unit's
// query rows (one bulk copy) and a descriptor; the consumer warps finish a
// unit (merge of their states through shared memory, then the output rows, or
// a partial when the unit goes on in another CTA) while the ring keeps
// filling.  A unit split across CTAs is merged by merge_jobs_kernel: the CTA
// holding its first page records the job.  The scored build (SC, for
// pa_decode_weights) stores every token's scores as it goes.  A unit that lies
// whole in the CTA's range gets its weights right after its last page, its scores
// still in L2 (all such units of a CTA use one area, the first one's, so the
// lines are written over before they need to go to HBM); the others' are
// left for weights_finish_kernel, with the range's start.
template <int KV, int D, int OUT, bool PSPLIT, int MINB, bool SC = false>
__global__ void __launch_bounds__(kThreads, MINB) decode_bal_kernel(const DecodeArgs a,
                                                              const __grid_constant__ CUtensorMap tmk,
                                                              const __grid_constant__ CUtensorMap tmv) {
  using C = Cfg<KV, D>;
  using B = BalCfg<KV, D>;
  constexpr bool F8 = C::kFp8;
  constexpr bool BLK = C::kBlockScaled;
  constexpr int NT = D / 16;
  constexpr bool LDT = F8 && C::kSwizzle;
  constexpr bool LD16 = !F8 && C::kSwizzle;
  constexpr int QW = D / 8;  // 32-bit query words per thread
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ long long s_warp_sums[kThreads / 32];
  __shared__ long long s_start_off, s_rbegin, s_rend;
  __shared__ long long s_start_cost;  // scored build
  __shared__ int s_start_seq;
  __shared__ int s_abort;
  __shared__ int s_go;
  __shared__ int4 s_job;
  __shared__ float2 s_unit_ml[SC ? 8 : 1];  // scored build: (M, 1 / L) of a whole unit's heads
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + C::kAlign - 1) & ~uintptr_t(C::kAlign - 1));
  uint8_t* ring = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + B::kOffBars);
  uint64_t* empty = full + C::kStages;
  uint64_t* q_full = empty + C::kStages;
  uint64_t* q_empty = q_full + 1;
  uint8_t* frag = smem + B::kOffFrag;
  const uint16_t* qstage = reinterpret_cast<const uint16_t*>(smem + B::kOffQStage);
  float2* mlx = reinterpret_cast<float2*>(smem + B::kOffMl);  // [warp][head] (m, l)
  SegDesc* desc = reinterpret_cast<SegDesc*>(smem + B::kOffDesc);
  float2* stage_scale = reinterpret_cast<float2*>(smem + B::kOffScale);
  volatile int* abort_flag = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();  // the kernel before may still write q, tables, pages

  // ---------------------------------------------------------------- schedule
  // Cost of every sequence (a contiguous share of the sequences per thread)
  // and its prefix sum.  A unit (sequence, kv head) of n pages costs n + kUnit
  // page-times: finishing a unit (the warps' merge, the output rows, the next
  // unit's query rows) costs a CTA about kUnit pages' worth of streaming, so a
  // range of short units gets fewer pages.  Positions: sequence s's units
  // start at the cost of the sequences before s; within a unit the first kUnit
  // positions hold no page, page p sits at kUnit + p.  The ranges are cut in
  // cost; the real pages of position x are R(x) = Hkv * (pages before s) +
  // h * n + max(0, v - kUnit) for x in unit h of s at offset v.
  constexpr int kUnit = B::kUnitCostPages;
  const bool whole = SC && a.whole;
  auto span = [&](int np) { return whole ? 1 : np + kUnit; };  // a unit's cost
  const int per = (a.S + kThreads - 1) / kThreads;
  const int s0 = min(a.S, (int)threadIdx.x * per), s1 = min(a.S, s0 + per);
  long long mine = 0, mine_pg = 0;
  for (int s = s0; s < s1; ++s) {
    int c = a.ctx[s];
    if (c < 0 || c > a.max_blocks * 16) {
      record_error(a.err, PA_ERR_BOUNDS);
      c = clamp_ctx(c, a.max_blocks);
    }
    const int np = (c + 15) >> 4;
    mine_pg += np;
    mine += np > 0 ? (long long)a.Hkv * span(np) : 0;
  }
  long long total, total_pg;
  const long long before = block_exclusive_scan<kThreads>(mine, s_warp_sums, total);
  __syncthreads();  // the scan's partial sums are read before the second scan writes them
  const long long before_pg = block_exclusive_scan<kThreads>(mine_pg, s_warp_sums, total_pg);
  const long long ptot = total;  // in cost
  const long long T = max((ptot + a.ctas - 1) / a.ctas, whole ? 1LL : (long long)kMinPagesPerCta);
  const long long pos_begin = (long long)blockIdx.x * T;
  const long long pos_end = min(ptot, pos_begin + T);
  // Sequences without context get a zero output row, written by CTA s mod ctas.
  for (int s = blockIdx.x; s < a.S; s += a.ctas) {
    if (a.ctx[s] > 0) continue;
    for (int i = threadIdx.x; i < a.Hq * D; i += kThreads) store_out<OUT>(a.out, (size_t)s * a.Hq * D + i, 0.f);
  }
  // The thread whose sequences hold a boundary finds its sequence and real page.
  auto locate = [&](long long x, bool start) {
    long long cum = before, cum_pg = before_pg * a.Hkv;
    for (int s = s0; s < s1; ++s) {
      const long long np = (clamp_ctx(a.ctx[s], a.max_blocks) + 15) >> 4;
      const long long n = np > 0 ? (long long)a.Hkv * span((int)np) : 0;
      if (x < cum + n) {
        const long long off = x - cum, hh = off / span((int)np), v = off - hh * span((int)np);
        const long long r = cum_pg + hh * np + max(0LL, v - kUnit);
        if (start) {
          s_start_seq = s;
          s_start_off = off;
          if constexpr (SC) s_start_cost = cum;
          s_rbegin = r;
        } else {
          s_rend = r;
        }
        return;
      }
      cum += n;
      cum_pg += np * a.Hkv;
    }
  };
  if (before <= pos_begin && pos_begin < before + mine) locate(pos_begin, true);
  if (before <= pos_end && pos_end < before + mine) locate(pos_end, false);
  if (threadIdx.x == 0 && pos_end >= ptot) s_rend = total_pg * a.Hkv;
  if (threadIdx.x == 0 && pos_begin >= ptot) s_rbegin = total_pg * a.Hkv;
  __syncthreads();
  const int n_pages = (int)(s_rend - s_rbegin);  // real pages of this CTA
  if (n_pages <= 0) {  // no pages for this CTA: no partial and no merge job
    if (threadIdx.x == 0) a.jobs[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if constexpr (SC)
      if (threadIdx.x == 0) a.ranges[blockIdx.x].seq = -1;
    return;
  }
  if constexpr (SC)
    if (threadIdx.x == 0) a.ranges[blockIdx.x] = RangeStart{s_start_seq, 0, pos_begin, pos_end, s_start_cost, T};
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_job = make_int4(-1, 0, 0, 0);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, kConsumerWarps);
    fence_barrier_init();
  }
  if (threadIdx.x == kConsumerWarps * 32) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------ producer
    const uint64_t policy = l2_evict_first_policy();
    int seq = s_start_seq;
    int ctx = clamp_ctx(a.ctx[seq], a.max_blocks);
    int npages = (ctx + 15) >> 4;
    int h = (int)(s_start_off / span(npages));
    const int v0 = (int)(s_start_off - (long long)h * span(npages));
    int pg0 = max(0, v0 - kUnit);
    long long ucost = pos_begin - v0;  // cost position of the current unit's start
    int left = n_pages;                // real pages still to stream
    int kb = 0;  // CTA-local index of the unit's first page
    int issued = 0, nq = 0;  // page copies and query-row copies issued (lane 0)
    bool abort = false;
    for (int j = 0; !abort; ++j) {
      const int len = min(npages - pg0, left);
      // the unit's descriptor and query rows, once the consumers hold the previous ones
      int stop = 0;
      if (lane == 0) {
        if (j > 0 && !wait_or_abort(q_empty, (j - 1) & 1, abort_flag, a.err)) {
          stop = 1;
        } else {
          SegDesc sd;
          sd.seq = seq;
          sd.h = h;
          sd.pg0 = pg0;
          sd.len = len;
          sd.ctx = ctx;
          sd.npages = npages;
          sd.last_cta = (int)((ucost + kUnit + npages - 1) / T);  // the CTA of the unit's last page
          *desc = sd;
          const uint32_t qbytes = (uint32_t)(a.G * D * 2);
          mbar_arrive_expect_tx(q_full, qbytes);
          bulk_g2s(smem + B::kOffQStage, a.q + ((size_t)seq * a.Hq + (size_t)h * a.G) * D, qbytes, q_full,
                   policy);
          ++nq;
        }
      }
      if (__shfl_sync(kFull, stop, 0)) break;
      // the unit's pages; lane i holds the table entry (and tile scales) of page base + i
      const int32_t* trow = a.tables + (size_t)seq * a.max_blocks + pg0;
      for (int base = 0; base < len && !abort; base += 32) {
        int phys = 0;
        float sk = 0.f, sv = 0.f;
        if (base + lane < len) {
          phys = trow[base + lane];
          if (phys < 0 || phys >= a.num_blocks) {
            record_error(a.err, PA_ERR_BOUNDS);
            phys = 0;
          }
          if constexpr (BLK) {
            sk = a.ksc[(size_t)phys * a.Hkv + h];
            sv = a.vsc[(size_t)phys * a.Hkv + h];
          }
        }
        const int cnt = min(32, len - base);
        for (int i = 0; i < cnt; ++i) {
          const int ph = __shfl_sync(kFull, phys, i);
          float ski = 0.f, svi = 0.f;
          if constexpr (BLK) {
            ski = __shfl_sync(kFull, sk, i);
            svi = __shfl_sync(kFull, sv, i);
          }
          int st2 = 0;
          if (lane == 0) {
            const int k = kb + base + i, stage = k % C::kStages;
            if (k >= C::kStages && !wait_or_abort(&empty[stage], ((k / C::kStages) - 1) & 1, abort_flag, a.err)) {
              st2 = 1;
            } else {
              uint8_t* dst = ring + stage * C::kStageBytes;
              const int row0 = (ph * a.Hkv + h) * 16;
              if constexpr (BLK) stage_scale[stage] = make_float2(ski, svi);
              mbar_arrive_expect_tx(&full[stage], 2 * C::kTile);
              load_tile<C::kTmaRank>(dst, &tmk, row0, &full[stage], policy);
              load_tile<C::kTmaRank>(dst + C::kTile, &tmv, row0, &full[stage], policy);
              ++issued;
            }
          }
          if (__shfl_sync(kFull, st2, 0)) {
            abort = true;
            break;
          }
        }
      }
      if (abort) break;
      kb += len;
      left -= len;
      if (left <= 0) break;
      // the next unit, from its first page
      ucost += span(npages);
      pg0 = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {  // sequences without pages hold no position; one with pages lies ahead
          if (++seq >= a.S) break;
          ctx = clamp_ctx(a.ctx[seq], a.max_blocks);
        } while (ctx == 0);
        if (seq >= a.S) {  // the lengths changed under the kernel
          if (lane == 0) {
            record_error(a.err, PA_ERR_BOUNDS);
            *abort_flag = 1;
          }
          break;
        }
        npages = (ctx + 15) >> 4;
      }
    }
    // Wait (bounded, whatever the abort flag) until every copy this CTA issued
    // has landed, so no bulk write targets shared memory once the CTA exits.
    if (lane == 0) {
      for (int s = 0; s < C::kStages && s < issued; ++s) {  // each stage's last use
        const int uses = (issued - 1 - s) / C::kStages + 1;
        if (!mbar_wait(&full[s], (uses - 1) & 1)) record_error(a.err, PA_ERR_TIMEOUT);
      }
      if (nq > 0 && !mbar_wait(q_full, (nq - 1) & 1)) record_error(a.err, PA_ERR_TIMEOUT);
    }
    grid_dependents_launch();  // the merge may be scheduled (it waits for this grid)
  } else {
    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, t = lane & 3;
    uint32_t qf[QW];
    uint2* qsm = C::kQInSmem ? reinterpret_cast<uint2*>(frag) + warp * (QW / 2) * 32 : nullptr;
    float* slot = reinterpret_cast<float*>(frag);  // merge slot(s) [kMergeSlots][8][D]
    SegDesc* mine_d = desc + 1 + warp;             // this warp's copy of its unit's descriptor
    int kb = 0;
    long long area = -1;  // scored build: the unit whose score area this CTA's whole units use
    for (int j = 0; kb < n_pages; ++j) {
      // ---- the unit: descriptor and query rows
      const bool have_q = __all_sync(kFull, wait_or_abort(q_full, j & 1, abort_flag, a.err));
      if (lane == 0) *mine_d = *desc;
      __syncwarp();
      float qk_scale = a.qk_scale_log2;
      {
        uint32_t raw[QW];
        const uint4* qrow = reinterpret_cast<const uint4*>(qstage + g * D + t * (D / 4));
#pragma unroll
        for (int c = 0; c < QW / 4; ++c) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (g < a.G && have_q) u = qrow[c];
          raw[4 * c] = u.x;
          raw[4 * c + 1] = u.y;
          raw[4 * c + 2] = u.z;
          raw[4 * c + 3] = u.w;
        }
        if constexpr (F8) {
          // bfloat16 q -> binary16 with a power-of-two prescale shared by the group
          float amax = 0.f;
#pragma unroll
          for (int w = 0; w < QW; ++w) {
            amax = fmaxf(amax, fabsf(bf16_bits_to_float(raw[w] & 0xFFFFu)));
            amax = fmaxf(amax, fabsf(bf16_bits_to_float(raw[w] >> 16)));
          }
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, off));
          int ex = 0;
          if (amax > 0.f) frexpf(amax, &ex);
          const float qs = amax > 0.f ? ldexpf(1.f, 15 - ex) : 1.f;
          qk_scale = amax > 0.f ? qk_scale * ldexpf(1.f, ex - 15) : qk_scale;
#pragma unroll
          for (int w = 0; w < QW; ++w)
            qf[w] = pack2<false>(bf16_bits_to_float(raw[w] & 0xFFFFu) * qs,
                                 bf16_bits_to_float(raw[w] >> 16) * qs);
        } else {
#pragma unroll
          for (int w = 0; w < QW; ++w) qf[w] = raw[w];
        }
      }
      if constexpr (C::kQInSmem) {
#pragma unroll
        for (int i = 0; i < QW / 2; ++i) qsm[i * 32 + lane] = make_uint2(qf[2 * i], qf[2 * i + 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);  // the staged rows and descriptor may be replaced

      // ---- the unit's pages: warp w takes those whose CTA-local index is w mod 4
      const int len = have_q ? mine_d->len : 0;
      const int pg0 = mine_d->pg0, ctx = mine_d->ctx;
      float* score0 = nullptr;  // scored build: the scores of the unit's pages
      if constexpr (SC) {
        long long unit = (long long)mine_d->seq * a.Hkv + mine_d->h;
        if (pg0 == 0 && len == mine_d->npages) {
          if (area < 0) area = unit;
          unit = area;
        }
        score0 = a.scores + (size_t)unit * a.max_blocks * 16 * a.gs;
      }
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float vinv = INFINITY;  // block-scaled pools: 1 / the largest V scale seen (see decode_kernel)
      for (int k = kb + ((warp - kb) & (kConsumerWarps - 1)); k < kb + len; k += kConsumerWarps) {
        const int stage = k % C::kStages;
        if (!__all_sync(kFull, wait_or_abort(&full[stage], (k / C::kStages) & 1, abort_flag, a.err))) break;
        const uint8_t* Ks = ring + stage * C::kStageBytes;
        float* score = nullptr;
        if constexpr (SC) score = score0 + (size_t)(pg0 + k - kb) * 16 * a.gs;
        consume_page<KV, D, PSPLIT, SC>(Ks, Ks + C::kTile, (pg0 + k - kb) * 16, ctx, qk_scale, qf, qsm,
                                        &stage_scale[stage], m0, m1, l0, l1, o, vinv, score, SC ? a.gs : 0, SC ? a.G : 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, off);
        l1 += __shfl_xor_sync(kFull, l1, off);
      }
      if constexpr (BLK) {  // back to value units
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[i][0] *= 1.f / vinv;
          o[i][1] *= 1.f / vinv;
          o[i][2] *= 1.f / vinv;
          o[i][3] *= 1.f / vinv;
        }
      }

      // ---- merge of the four warps' states for this unit
      if (g == 0) {
        mlx[warp * 8 + 2 * t] = make_float2(m0, l0);
        mlx[warp * 8 + 2 * t + 1] = make_float2(m1, l1);
      }
      consumers_sync();  // every warp is past its last page (fragments dead); (m, l) published
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) {
        M0 = fmaxf(M0, mlx[w * 8 + 2 * t].x);
        M1 = fmaxf(M1, mlx[w * 8 + 2 * t + 1].x);
      }
      const float f0 = (m0 == -INFINITY) ? 0.f : fast_exp2(m0 - M0);
      const float f1 = (m1 == -INFINITY) ? 0.f : fast_exp2(m1 - M1);
      // A slot holds the accumulator fragments as the lanes hold them: value c
      // of m-tile i of lane L at (i * 4 + c) * 32 + L (stores without bank conflicts)
#pragma unroll
      for (int step = 0; step < kConsumerWarps / B::kMergeSlots; ++step) {
        if (warp / B::kMergeSlots == step) {
          float* sl = slot + (warp % B::kMergeSlots) * 8 * D + lane;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const float v[4] = {o[i][0] * f0, o[i][1] * f1, o[i][2] * f0, o[i][3] * f1};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (step == 0) sl[(i * 4 + c) * 32] = v[c];
              else sl[(i * 4 + c) * 32] += v[c];
            }
          }
        }
        consumers_sync();
      }
      // ---- the unit's output rows, or its partial
      const SegDesc sd = *mine_d;
      const bool direct = sd.pg0 == 0 && sd.len == sd.npages;
      const int pslot = 2 * blockIdx.x + (j == 0 ? 0 : 1);
      bool write = have_q && !*abort_flag;
      if constexpr (SC) write = __all_sync(kFull, write);  // one decision per warp: add_weights shuffles
      if (write && !direct && sd.pg0 == 0 && threadIdx.x == 0) s_job = make_int4(sd.seq, sd.h, sd.last_cta, pslot);
      const int tid = threadIdx.x;  // 0 .. 127
      for (int idx = tid; idx < a.G * D && write; idx += kConsumerWarps * 32) {
        const int head = idx / D, dim = idx - head * D;
        // where the fragments hold (head, dim): rows g (+ 8) of m-tile i for the
        // transposed-ldmatrix layouts, columns 2i (+ 1) of row g otherwise
        int i, gg, hi;
        if constexpr (LDT || LD16) {
          i = dim >> 4;
          gg = dim & 7;
          hi = (dim >> 3) & 1;
        } else {
          gg = dim / (D / 8);
          i = (dim % (D / 8)) >> 1;
          hi = dim & 1;
        }
        const int sidx = (i * 4 + 2 * hi + (head & 1)) * 32 + 4 * gg + (head >> 1);
        float O = slot[sidx];
        if constexpr (B::kMergeSlots == 2) O += slot[8 * D + sidx];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, mlx[w * 8 + head].x);
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) {
          const float2 ml = mlx[w * 8 + head];
          L += (ml.x == -INFINITY) ? 0.f : fast_exp2(ml.x - M) * ml.y;
        }
        if (direct) {
          const size_t row = (size_t)sd.seq * a.Hq + (size_t)sd.h * a.G + head;
          store_out<OUT>(a.out, row * D + dim, L > 0.f ? O / L * a.v_scale : 0.f);
          if constexpr (SC)
            if (dim == 0) s_unit_ml[head] = make_float2(M, 1.f / L);
        } else {
          const size_t prow = (size_t)pslot * a.G + head;
          a.ws_o[prow * D + dim] = O;
          if (dim == 0) {
            a.ws_ml[2 * prow] = M;
            a.ws_ml[2 * prow + 1] = L;
          }
        }
      }
      if constexpr (SC) {
        if (direct) {
          if (tid >= a.G && tid < a.gs) s_unit_ml[tid] = make_float2(0.f, 0.f);
          consumers_sync();  // (M, 1 / L), and every warp's scores
          const size_t row = ((size_t)sd.seq * a.Hkv + sd.h) * a.w_stride;
          if (write)
            add_weights<kConsumerWarps * 32, C::kFp8 ? 2 : 1>(score0, a.gs, s_unit_ml, a.w_in ? a.w_in + row : nullptr, a.w_out + row,
                                                a.decay, 0, totals_end(sd.ctx, a));
        }
      }
      if (tid == 0) s_go = !*abort_flag;  // one thread decides for all, read after the barrier
      consumers_sync();  // the slots and the (m, l) area are free again
      kb += len;
      if (!s_go) break;  // uniform: every warp reads the one decision
    }
    grid_dependents_launch();
    if (threadIdx.x == 0) a.jobs[blockIdx.x] = s_job;
  }
}

}  // namespace pa
