// pa_rope.cu -- rotary positions fused with the write into the paged KV pool.
//
// Pair i of a head turns by p f_i at position p.  The kernel needs that angle
// modulo a turn, for positions up to 2^31: an fp32 product would be off by a
// tenth of a radian at a million, and fp64 runs at a small fraction of the
// fp32 rate on this part.  So the speed is kept as a 64-bit binary fraction of
// a turn, F_i = f_i / (2 pi) * 2^64: p F_i modulo 2^64 is the angle's fraction
// of a turn, one integer multiply with no reduction step, and its upper bits as a
// signed fraction of half a turn are the argument of sincospi.  F_i comes from a
// double: off by at most 2^-53 of a turn per position (2^-33 of a turn at a million, 2^-22
// at 2^31); the argument's rounding to fp32 is 2^-26 of a turn.
//
// The work is a copy with some arithmetic in it, bound by HBM: 16-byte loads
// and stores, each thread owning both halves of eight pairs.  A warp makes its
// token's table of sin / cos in shared memory, for all the heads it takes, while its
// first loads are in flight; no warp waits for another.  8192 tokens of 64 / 8
// heads (320 MB) into FP8 pages: 56 us, 5.7 TB/s, 0.84 of a plain copy's rate;
// a block-wide table behind a barrier gave 67 us.  What holds it back is the
// arithmetic between loads and stores (issue slots 46% busy) and that the 1024
// CTAs take 1.7 waves.
//
// pa_norm_rope_and_cache adds, before the turn, x rsqrt(mean(x^2) + eps) (offset + w) per head:
// the D / 16 threads of a row sum their squares in fp32 with shuffles.  The same 8192 tokens:
// 67.7 us, 4.7 TB/s, with issue slots 67% and DRAM 50% busy: bound by neither, but by what a warp waits for (28% of its
// time loads, 28% shuffles and fixed latencies, at 6.7 warps a scheduler) and by 1.68 waves of CTAs.  64 tokens of
// 32 / 8 heads (bf16) 4.6 us; 2037 of 32 / 8 heads with a scale per tile 26.
// Weights held in fp32 registers or in shared memory, packed arithmetic and other
// warps per CTA were all slower.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"

namespace pa {
namespace {

// How a thread finds the partner of an element: HALF with rot_dim % 16 == 0
// (whole 16-byte vectors face each other), INTERLEAVED (pairs stay inside a
// vector), or HALF with any even rot_dim (partners read one by one).
enum RopeLayout { ROPE_HALF = 0, ROPE_INTER = 1, ROPE_HALF_ODD = 2 };

constexpr int kRopeWarps = 8;  // per CTA
// A token gets one warp, or up to eight while the call has fewer than this many
// warps: each warp makes its own table, so more warps a token cost instructions,
// fewer leave SMs idle.  64 tokens of 32 / 8 heads (bf16): 6.1 us with one warp a
// token, 3.7 with eight; 1024 of 64 / 8 (FP8): 17.3 with one, 12.6 with two, 13.8
// with eight; 8192: 56 us with one or two (5.7 TB/s), 83 with eight.
constexpr int kRopeFewWarps = 2048;

struct RopeArgs {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  const uint16_t* v;
  long long qs, ks, vs;  // token strides, elements
  const int32_t* pos;
  const int64_t* slots;
  int T, Hq, Hkv;
  int warps_per_token;     // 1, 2, 4 or 8
  unsigned parts;          // block-scaled pools
  long long num_slots;
  uint8_t* kpool;
  uint8_t* vpool;
  float k_scale, v_scale;  // PA_FP8_E4M3
  float* ksc;              // PA_FP8_E4M3_BLOCK
  float* vsc;
  unsigned int* err;
  pa_rope rope;
  // pa_norm_rope_and_cache (EXT builds): weights of the heads' norms (nullptr: that side
  // keeps its scale), the elements from one head's weights to the next's (0: shared),
  // and the axis whose positions a pair turns with (axis a's are pos[a T ..])
  const uint16_t* qw;
  const uint16_t* kw;
  int q_wstride, k_wstride;
  float eps, w_offset;
  uint8_t axis[64];
};

// cos and sin of pair i at position p, times gain.
__device__ __forceinline__ float2 turn(const pa_rope& r, int i, int p) {
  const int64_t phase = (int64_t)(r.step[i] * (uint64_t)(int64_t)p);
  float s, c;
  sincospif((float)phase * 0x1p-63f, &s, &c);  // phase / 2^64 of a turn = phase / 2^63 of half a turn
  return make_float2(c * r.gain, s * r.gain);
}

// A token's table of D / 2 (cos, sin) pairs in shared memory.  Unit u of a row
// uses pairs 8u .. 8u+7 two at a time: [j][u] of float4 spreads the units of a
// row over all banks.  (ROPE_HALF_ODD indexes single pairs.)
template <int D, int LAY>
__device__ __forceinline__ int cs_index(int i) {
  if constexpr (LAY == ROPE_HALF_ODD) return i;
  return 2 * (((i & 7) >> 1) * (D / 16) + (i >> 3)) + (i & 1);
}

// The two 16-byte vectors of a row that unit u owns.
template <int LAY>
__device__ __forceinline__ void unit_vecs(int u, int rot, int& v0, int& v1) {
  if constexpr (LAY == ROPE_HALF) {
    const int n = rot >> 4;  // units that turn
    v0 = u < n ? u : 2 * u;
    v1 = u < n ? u + n : 2 * u + 1;
  } else {
    v0 = 2 * u;
    v1 = 2 * u + 1;
  }
}

__device__ __forceinline__ void words(uint4 x, uint32_t (&w)[4]) {
  w[0] = x.x;
  w[1] = x.y;
  w[2] = x.z;
  w[3] = x.w;
}

// What a thread holds of one row: its two vectors, and for ROPE_HALF_ODD the
// partners of their elements.
template <int LAY>
struct UnitIn {
  uint4 x0, x1;
  uint16_t partner[LAY == ROPE_HALF_ODD ? 16 : 1];
};

template <int LAY, bool FULL>
__device__ __forceinline__ void load_unit(const uint16_t* row, int u, int rot, UnitIn<LAY>& in) {
  int v0, v1;
  unit_vecs<LAY>(u, rot, v0, v1);
  in.x0 = *reinterpret_cast<const uint4*>(row + 8 * v0);
  in.x1 = *reinterpret_cast<const uint4*>(row + 8 * v1);
  if constexpr (LAY == ROPE_HALF_ODD) {
    const int half = rot >> 1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int e = 16 * u + j;
      in.partner[j] = e < rot ? row[e < half ? e + half : e - half] : 0;
    }
  }
}

// The unit's 16 values as they are.
template <bool BF, int LAY>
__device__ __forceinline__ void plain_unit(const UnitIn<LAY>& in, float (&y)[16]) {
  uint32_t w0[4], w1[4];
  words(in.x0, w0);
  words(in.x1, w1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = unpack2<BF>(w0[j]), b = unpack2<BF>(w1[j]);
    y[2 * j] = a.x;
    y[2 * j + 1] = a.y;
    y[8 + 2 * j] = b.x;
    y[8 + 2 * j + 1] = b.y;
  }
}

// What a head's norm multiplies a unit with: rs = 1 / sqrt(mean x^2 + eps) and the
// weights of the unit's two vectors, in the pool's 16-bit type; w: the head's weights
// (for the partners of ROPE_HALF_ODD).
struct UnitNorm {
  float rs, offset;
  uint4 w0, w1;
  const uint16_t* w;
};

// x rs (offset + w), of two neighbours.
template <bool BF>
__device__ __forceinline__ float2 scaled2(float x0, float x1, uint32_t w, const UnitNorm& n) {
  const float2 v = unpack2<BF>(w);
  return make_float2(x0 * n.rs * (n.offset + v.x), x1 * n.rs * (n.offset + v.y));
}

template <bool BF>
__device__ __forceinline__ void scale_unit(const UnitNorm& n, float (&y)[16]) {
  uint32_t w0[4], w1[4];
  words(n.w0, w0);
  words(n.w1, w1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = scaled2<BF>(y[2 * j], y[2 * j + 1], w0[j], n), b = scaled2<BF>(y[8 + 2 * j], y[9 + 2 * j], w1[j], n);
    y[2 * j] = a.x;
    y[2 * j + 1] = a.y;
    y[8 + 2 * j] = b.x;
    y[9 + 2 * j] = b.y;
  }
}

// 1 / sqrt(mean x^2 + eps) of the rows that the warp's lanes hold, D / 16 lanes a row
// (every lane takes part).
template <bool BF, int D, int LAY>
__device__ __forceinline__ float row_rsqrt(const UnitIn<LAY>& in, float eps) {
  float y[16];
  plain_unit<BF, LAY>(in, y);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 16; ++j) s[j & 3] = fmaf(y[j], y[j], s[j & 3]);
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return rsqrtf(fmaf(sum, 1.f / D, eps));
}

// The unit's 16 values after the rotation.  FULL: all of the row turns.  norm: the
// head's norm, which comes first (nullptr: none).
template <bool BF, int D, int LAY, bool FULL>
__device__ __forceinline__ void turn_unit(const UnitIn<LAY>& in, int u, int rot, const float2* cs, float (&y)[16],
                                          const UnitNorm* norm = nullptr) {
  plain_unit<BF, LAY>(in, y);
  if (norm) scale_unit<BF>(*norm, y);
  if constexpr (LAY == ROPE_HALF) {
    if (!FULL && u >= (rot >> 4)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = reinterpret_cast<const float4*>(cs)[j * (D / 16) + u];
      const float a0 = y[2 * j], b0 = y[8 + 2 * j], a1 = y[2 * j + 1], b1 = y[9 + 2 * j];
      y[2 * j] = a0 * t.x - b0 * t.y;
      y[8 + 2 * j] = b0 * t.x + a0 * t.y;
      y[2 * j + 1] = a1 * t.z - b1 * t.w;
      y[9 + 2 * j] = b1 * t.z + a1 * t.w;
    }
  } else if constexpr (LAY == ROPE_INTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = reinterpret_cast<const float4*>(cs)[j * (D / 16) + u];
      const float a0 = y[4 * j], b0 = y[4 * j + 1], a1 = y[4 * j + 2], b1 = y[4 * j + 3];
      if (FULL || 16 * u + 4 * j < rot) {
        y[4 * j] = a0 * t.x - b0 * t.y;
        y[4 * j + 1] = b0 * t.x + a0 * t.y;
      }
      if (FULL || 16 * u + 4 * j + 2 < rot) {
        y[4 * j + 2] = a1 * t.z - b1 * t.w;
        y[4 * j + 3] = b1 * t.z + a1 * t.w;
      }
    }
  } else {
    const int half = rot >> 1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int e = 16 * u + j;
      if (e < rot) {
        const float2 t = cs[e < half ? e : e - half];
        float2 p2 = unpack2<BF>(in.partner[j]);
        if (norm) p2 = scaled2<BF>(p2.x, 0.f, norm->w[e < half ? e + half : e - half], *norm);
        y[j] = e < half ? y[j] * t.x - p2.x * t.y : y[j] * t.x + p2.x * t.y;
      }
    }
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(pack2<BF>(y[0], y[1]), pack2<BF>(y[2], y[3]), pack2<BF>(y[4], y[5]), pack2<BF>(y[6], y[7]));
}

// E4M3 codes of 8 values / s (code 0 when s = 0): the IEEE quotient, rounded
// to nearest even and saturated, as pa_reshape_and_cache stores values.
__device__ __forceinline__ uint2 codes8(const float* y, float s) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = make_float2(0.f, 0.f);
    if (s > 0.f) f = make_float2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
    q[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// Items [lt, items) of one token's heads, `nt` apart: item i is unit i % UNITS of
// head i / UNITS, IPT of them at a time, every load of a batch issued before the
// first use.  `first` runs behind the first batch's loads (the token's table);
// put(h, v0, v1, in, y) stores the turned unit.  The rounds are counted per warp,
// not per lane: in a last round with fewer than 32 items the lanes without one
// take part in the warp's barrier all the same.
// EXT: with the heads' norm where w, their weights, is given.
template <bool BF, int D, int LAY, bool FULL, bool EXT, typename First, typename Put>
__device__ __forceinline__ void turn_heads(const uint16_t* src, int items, int rot, int lt, int nt, const float2* cs,
                                           const uint16_t* w, int wstride, float eps, float w_offset, First first, Put put) {
  constexpr int UNITS = D / 16, IPT = LAY == ROPE_HALF_ODD ? 1 : 2;
  const int lane = lt & 31, warp0 = lt - lane;
  UnitNorm norm = {};
  auto weights = [&](int h) {  // (a lane's unit is the same in every round)
    int v0, v1;
    unit_vecs<LAY>(lane % UNITS, FULL ? D : rot, v0, v1);
    norm.w = w + (long long)h * wstride;
    norm.w0 = *reinterpret_cast<const uint4*>(norm.w + 8 * v0);
    norm.w1 = *reinterpret_cast<const uint4*>(norm.w + 8 * v1);
  };
  if constexpr (EXT) {
    norm.offset = w_offset;
    if (w) weights(0);
  }
  for (int base = warp0; base < items || base == warp0; base += nt * IPT) {
    UnitIn<LAY> in[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
      const int i = base + lane + j * nt;
      if constexpr (EXT) in[j] = {};
      if (i < items) load_unit<LAY, FULL>(src + (i / UNITS) * D, i % UNITS, FULL ? D : rot, in[j]);
    }
    if (base == warp0) first();
    // The table is complete; and with q_out == q a row's partners, which its own
    // warp reads (above), are read before any lane writes the row.
    __syncwarp();
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
      const int i = base + lane + j * nt;
      const bool normed = EXT && w;
      if (normed) norm.rs = row_rsqrt<BF, D, LAY>(in[j], eps);
      if (i < items) {
        if (normed && wstride) weights(i / UNITS);
        int v0, v1;
        unit_vecs<LAY>(i % UNITS, FULL ? D : rot, v0, v1);
        float y[16];
        turn_unit<BF, D, LAY, FULL>(in[j], i % UNITS, FULL ? D : rot, cs, y, normed ? &norm : nullptr);
        put(i / UNITS, v0, v1, y);
      }
    }
  }
}

// One token by `nt` threads (whole warps) of which this is `lt`: its query heads,
// then (KV) its key and value heads into their slot.  cs: this warp's table.
template <bool BF, bool FP8, bool KV, int D, int LAY, bool FULL, bool EXT>
__device__ __forceinline__ void rope_token(const RopeArgs& a, int t, int lt, int nt, float2* cs) {
  constexpr int UNITS = D / 16;
  const int rot = FULL ? D : a.rope.rot_dim;
  uint16_t* q_out = a.q_out + (long long)t * a.Hq * D;
  turn_heads<BF, D, LAY, FULL, EXT>(
      a.q + t * a.qs, a.Hq * UNITS, rot, lt, nt, cs, a.qw, a.q_wstride, a.eps, a.w_offset,
      [&] {
        int p = a.pos[t];
        for (int i = lt & 31; i < (rot >> 1); i += 32) {
          if constexpr (EXT) p = a.pos[(long long)a.axis[i] * a.T + t];
          cs[cs_index<D, LAY>(i)] = turn(a.rope, i, p);
        }
      },
      [&](int h, int v0, int v1, const float* y) {
        *reinterpret_cast<uint4*>(q_out + h * D + 8 * v0) = pack8<BF>(y);
        *reinterpret_cast<uint4*>(q_out + h * D + 8 * v1) = pack8<BF>(y + 8);
      });
  if constexpr (KV) {
    const int64_t slot = a.slots[t];
    if (slot >= a.num_slots && lt == 0) record_error(a.err, PA_ERR_BOUNDS);
    if (slot < 0 || slot >= a.num_slots) return;
    // element (h, offset, d) of the slot's block
    const long long e0 = ((slot >> 4) * a.Hkv * 16 + (slot & 15)) * (long long)D;
    constexpr int EB = FP8 ? 1 : 2;
    uint8_t* kp = a.kpool + EB * e0;
    uint8_t* vp = a.vpool + EB * e0;
    turn_heads<BF, D, LAY, FULL, EXT>(
        a.k + t * a.ks, a.Hkv * UNITS, rot, lt, nt, cs, a.kw, a.k_wstride, a.eps, a.w_offset, [] {},
        [&](int h, int v0, int v1, const float* y) {
          uint8_t* dst = kp + (long long)h * (16 * D * EB);
          if constexpr (FP8) {
            *reinterpret_cast<uint2*>(dst + 8 * v0) = codes8(y, a.k_scale);
            *reinterpret_cast<uint2*>(dst + 8 * v1) = codes8(y + 8, a.k_scale);
          } else {
            *reinterpret_cast<uint4*>(dst + 16 * v0) = pack8<BF>(y);
            *reinterpret_cast<uint4*>(dst + 16 * v1) = pack8<BF>(y + 8);
          }
        });
    // values: whole vectors, unchanged or encoded
    const uint16_t* v = a.v + t * a.vs;
    for (int i = lt; i < a.Hkv * (D / 8); i += nt) {
      const uint4 x = *reinterpret_cast<const uint4*>(v + 8 * i);
      uint8_t* dst = vp + (long long)(i / (D / 8)) * (16 * D * EB) + (i % (D / 8)) * (8 * EB);
      if constexpr (FP8) {
        uint32_t w[4];
        words(x, w);
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = unpack2<BF>(w[j]);
          y[2 * j] = u.x;
          y[2 * j + 1] = u.y;
        }
        *reinterpret_cast<uint2*>(dst) = codes8(y, a.v_scale);
      } else {
        *reinterpret_cast<uint4*>(dst) = x;
      }
    }
  }
}

// FULL: every dimension turns (ROPE_HALF and ROPE_INTER).  EXT: pa_norm_rope_and_cache.
template <bool BF, bool FP8, int D, int LAY, bool FULL, bool EXT>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_cache_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 cs[kRopeWarps][D / 2];
  grid_dependents_launch();  // a decode behind this kernel waits for its writes itself
  const int warp = threadIdx.x >> 5, wpt = a.warps_per_token, tok = warp / wpt;
  const int t = blockIdx.x * (kRopeWarps / wpt) + tok;
  if (t < a.T)
    rope_token<BF, FP8, true, D, LAY, FULL, EXT>(a, t, threadIdx.x - tok * wpt * 32, wpt * 32, cs[warp]);
}

// Block-scaled pools.  For each token come a.parts CTAs, K and V of eight heads
// each; those of a token that starts a run (see reshape_block_scaled_kernel) take the run, a warp per (K or V, head)
// tile, the others return at once.  The CTAs behind them turn queries as above: the
// runs are the longer chains, so they start first.  A run's rows of one tile, at most 16 x D values, stay in the warp's
// registers as they were loaded; they are turned twice, for the maximum and for
// the encoding, which costs less than the registers of the fp32 values would
// (four CTAs on an SM in the place of two).  2048 tokens of 64 / 8 heads (80 MB):
// 25 us; 29 with the queries first, 41 with the values kept in fp32.  Bound by
// the runs' latency: slots, rows, the table, the maximum, the division.
template <int D, int LAY, bool EXT>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_cache_block_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 cs[16][D / 2];
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned r = blockIdx.x, kv_ctas = (unsigned)a.T * a.parts;
  if (r >= kv_ctas) {
    const int wpt = a.warps_per_token, tok = warp / wpt;
    const int t = (r - kv_ctas) * (kRopeWarps / wpt) + tok;
    if (t < a.T)
      rope_token<true, true, false, D, LAY, false, EXT>(a, t, threadIdx.x - tok * wpt * 32, wpt * 32, cs[warp]);
    return;
  }
  const int t = r / a.parts, part = r % a.parts;
  // lane i reads the slot of token t - 1 + i: the run's length is one ballot away
  const long long ti = (long long)t - 1 + lane;
  const int64_t sl = lane <= 16 && ti >= 0 && ti < a.T ? a.slots[ti] : -2;
  const int64_t slot = __shfl_sync(0xffffffffu, sl, 1), prev = __shfl_sync(0xffffffffu, sl, 0);
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0 && part == 0) record_error(a.err, PA_ERR_BOUNDS);
    return;
  }
  const int off0 = (int)(slot & 15);
  if (off0 != 0 && prev == slot - 1) return;  // not the first token of its run
  const unsigned follows = __ballot_sync(0xffffffffu, sl == slot + lane - 1) >> 1;  // bit i: token t + i
  const int n = min(16 - off0, __ffs(~follows) - 1);
  const bool is_v = part & 1;
  const int h = (part >> 1) * kRopeWarps + warp;
  const bool live = h < a.Hkv;
  const int rot = a.rope.rot_dim;
  const uint16_t* src = (is_v ? a.v : a.k) + (long long)(live ? h : 0) * D;
  const long long stride = is_v ? a.vs : a.ks;
  const size_t sidx = (size_t)(slot >> 4) * a.Hkv + (live ? h : 0);
  float* scp = (is_v ? a.vsc : a.ksc) + sidx;
  constexpr int UNITS = D / 16, ROWS = 32 / UNITS, ITERS = 16 / ROWS;
  const int u = lane % UNITS, r0 = lane / UNITS;
  int v0, v1;
  unit_vecs<LAY>(u, rot, v0, v1);
  uint4 x[ITERS][2];
  auto row_at = [&](int i) { return src + (t + i * ROWS + r0) * stride; };
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (i * ROWS + r0 < n) {
      x[i][0] = *reinterpret_cast<const uint4*>(row_at(i) + 8 * v0);
      x[i][1] = *reinterpret_cast<const uint4*>(row_at(i) + 8 * v1);
    }
  }
  const float s_old = off0 > 0 ? *scp : 0.f;
  if (!is_v) {  // the run's tables, while the rows are in flight
    for (int i = threadIdx.x; i < n * (rot >> 1); i += blockDim.x) {
      const int tk = i / (rot >> 1), p = i - tk * (rot >> 1);
      const long long at = EXT ? (long long)a.axis[p] * a.T : 0;
      cs[tk][cs_index<D, LAY>(p)] = turn(a.rope, p, a.pos[at + t + tk]);
    }
    __syncthreads();
  }
  if (!live) return;
  uint32_t mb = 0;  // largest |y|: without the sign bit, magnitudes order like their bits (a NaN above all)
  auto widen = [&](int i, const float (&y)[16]) {
    if (i * ROWS + r0 < n) {
#pragma unroll
      for (int j = 0; j < 16; ++j) mb = max(mb, __float_as_uint(y[j]) & 0x7FFFFFFFu);
    }
  };
  // EXT: the norm makes values too dear to make twice, so they are kept, half of them in registers, half
  // in shared memory ([vector][lane], so without conflicts), which leaves room for four CTAs on an SM:
  // 2037 tokens of 32 / 8 heads 25.6 us, 30.4 made twice, 27.0 with three CTAs.
  constexpr bool ODD = LAY == ROPE_HALF_ODD;
  constexpr int IN_REGS = ITERS / 2, SLOTS = EXT ? ITERS - IN_REGS : 1;
  __shared__ float4 ys[EXT ? kRopeWarps : 1][SLOTS][4][EXT ? 32 : 1];
  float yr[IN_REGS][16];
  auto values = [&](int i, float (&y)[16]) {
    UnitIn<LAY> in;
    in.x0 = x[i][0];
    in.x1 = x[i][1];
    if (is_v) {
      plain_unit<true, LAY>(in, y);
    } else {
      if constexpr (ODD) load_unit<LAY, false>(row_at(i), u, rot, in);
      turn_unit<true, D, LAY, false>(in, u, rot, cs[i * ROWS + r0], y);
    }
  };
  if constexpr (EXT) {
    const bool normed = !is_v && a.kw;
    UnitNorm norm = {};
    if (normed) {
      norm.offset = a.w_offset;
      norm.w = a.kw + (long long)h * a.k_wstride;
      norm.w0 = *reinterpret_cast<const uint4*>(norm.w + 8 * v0);
      norm.w1 = *reinterpret_cast<const uint4*>(norm.w + 8 * v1);
    }
#pragma unroll
    for (int step = 0; step < ITERS; ++step) {
      const int i = ODD ? step : ITERS - 1 - step;
      if (i * ROWS >= n) continue;
      constexpr int L = ODD ? ROPE_INTER : LAY;  // (an odd row's partners are not read again)
      float y[16];
      UnitIn<L> in;
      in.x0 = x[i][0];
      in.x1 = x[i][1];
      const int slot_of = i < IN_REGS ? 0 : i - IN_REGS;
      if (is_v) {
        plain_unit<true, L>(in, y);
      } else {
        if (normed) norm.rs = row_rsqrt<true, D, L>(in, a.eps);
        if constexpr (ODD) {
          // partners through shared memory: the rows of this step
          plain_unit<true, L>(in, y);
          if (normed) scale_unit<true>(norm, y);
          float* row = reinterpret_cast<float*>(ys[warp][slot_of]) + r0 * D;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<float4*>(row + 16 * u)[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
          __syncwarp();
          const int half = rot >> 1;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int e = 16 * u + j;
            if (e < rot) {
              const float2 t = cs[i * ROWS + r0][e < half ? e : e - half];
              const float p = row[e < half ? e + half : e - half];
              y[j] = e < half ? y[j] * t.x - p * t.y : y[j] * t.x + p * t.y;
            }
          }
          __syncwarp();
        } else {
          turn_unit<true, D, L, false>(in, u, rot, cs[i * ROWS + r0], y, normed ? &norm : nullptr);
        }
      }
      widen(i, y);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (i < IN_REGS) yr[i < IN_REGS ? i : 0][j] = y[j];
      if (i >= IN_REGS) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ys[warp][slot_of][j][lane] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
      if (i * ROWS + r0 < n) {
        float y[16];
        values(i, y);
        widen(i, y);
      }
  }
  mb = __reduce_max_sync(0xffffffffu, mb);
  const float s_run = __fdiv_rn(__uint_as_float(mb), 448.f);
  const bool grow = off0 == 0 || s_run > s_old;
  const float s = grow ? s_run : s_old;
  uint8_t* tile = (is_v ? a.vpool : a.kpool) + sidx * 16 * D;
  if (off0 > 0 && grow) {  // the earlier rows' codes, to the larger scale
    for (int i = lane; i < off0 * D / 8; i += 32) {
      uint2* p = reinterpret_cast<uint2*>(tile) + i;
      const uint2 c = *p;
      uint32_t f[4];
      e4m3x4_to_f16x2x2(c.x, f[0], f[1]);
      e4m3x4_to_f16x2x2(c.y, f[2], f[3]);
      float z[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v2 = unpack2<false>(f[j]);
        z[2 * j] = __fmul_rn(v2.x, s_old);
        z[2 * j + 1] = __fmul_rn(v2.y, s_old);
      }
      *p = codes8(z, s);
    }
  }
#pragma unroll
  for (int i = 0; i < ITERS; ++i)
    if (i * ROWS + r0 < n) {
      float y[16];
      if constexpr (EXT) {
        if (i < IN_REGS) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = yr[i < IN_REGS ? i : 0][j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 f = ys[warp][i < IN_REGS ? 0 : i - IN_REGS][j][lane];
            y[4 * j] = f.x, y[4 * j + 1] = f.y, y[4 * j + 2] = f.z, y[4 * j + 3] = f.w;
          }
        }
      } else {
        values(i, y);
      }
      uint8_t* dst = tile + (size_t)(off0 + i * ROWS + r0) * D;
      *reinterpret_cast<uint2*>(dst + 8 * v0) = codes8(y, s);
      *reinterpret_cast<uint2*>(dst + 8 * v1) = codes8(y + 8, s);
    }
  if (lane == 0) *scp = s;
}

// ---------------------------------------------------------------- host side
typedef void (*RopeKernel)(RopeArgs);

template <bool BF, bool FP8, int D, bool EXT>
RopeKernel pick_lay(int lay, bool full) {
  if (lay == ROPE_HALF_ODD) return rope_cache_kernel<BF, FP8, D, ROPE_HALF_ODD, false, EXT>;
  if (lay == ROPE_HALF)
    return full ? rope_cache_kernel<BF, FP8, D, ROPE_HALF, true, EXT>
                : rope_cache_kernel<BF, FP8, D, ROPE_HALF, false, EXT>;
  return full ? rope_cache_kernel<BF, FP8, D, ROPE_INTER, true, EXT>
              : rope_cache_kernel<BF, FP8, D, ROPE_INTER, false, EXT>;
}

template <int D, bool EXT>
RopeKernel pick_kernel(int kv_dtype, int lay, bool full) {
  if (kv_dtype == PA_FP8_E4M3_BLOCK)
    return lay == ROPE_HALF    ? rope_cache_block_kernel<D, ROPE_HALF, EXT>
           : lay == ROPE_INTER ? rope_cache_block_kernel<D, ROPE_INTER, EXT>
                               : rope_cache_block_kernel<D, ROPE_HALF_ODD, EXT>;
  if (kv_dtype == PA_FP8_E4M3) return pick_lay<true, true, D, EXT>(lay, full);
  return kv_dtype == PA_BF16 ? pick_lay<true, false, D, EXT>(lay, full) : pick_lay<false, false, D, EXT>(lay, full);
}

template <bool EXT>
RopeKernel pick_kernel(int head_dim, int kv_dtype, int lay, bool full) {
  return head_dim == 64 ? pick_kernel<64, EXT>(kv_dtype, lay, full) : pick_kernel<128, EXT>(kv_dtype, lay, full);
}

int check_stride(const char* name, size_t stride, int heads, int head_dim) {
  if (stride < (size_t)heads * head_dim || stride % 8 != 0 || stride >= (size_t)1 << 40)
    return fail(PA_ERR_INVALID, "%s_stride %zu must be a multiple of 8, at least %zu and below 2^40", name, stride,
                (size_t)heads * head_dim);
  return PA_OK;
}

// What pa_norm_rope_and_cache adds to a call.
struct RopeExt {
  const void* q_weight;
  const void* k_weight;
  int weights_per_head;
  float eps, offset;
  const pa_rope_axes* axes;
};

// Both entry points.  ext: pa_norm_rope_and_cache's norms and axes, checked; nullptr for pa_rope_and_cache.
int rope_call(pa_pool* pool, int layer, const pa_rope* rope, const RopeExt* ext, const void* q, size_t q_stride,
              void* q_out, int n_q_heads, const void* k, size_t k_stride, const void* v, size_t v_stride,
              const int32_t* positions_dev, const int64_t* slot_mapping_dev, int T, void* stream) {
  int st = check_pool_layer(pool, layer);
  if (st) return st;
  const pa_pool_desc& d = pool->desc;
  if (!rope) return fail(PA_ERR_INVALID, "null rope");
  if ((rope->layout != PA_ROPE_HALF && rope->layout != PA_ROPE_INTERLEAVED) || rope->rot_dim < 2 ||
      rope->rot_dim % 2 != 0 || !std::isfinite(rope->gain))
    return fail(PA_ERR_INVALID, "the rope was not filled by pa_rope_init");
  if (rope->rot_dim > d.head_dim)
    return fail(PA_ERR_INVALID, "rot_dim %d above the pool's head_dim %d", rope->rot_dim, d.head_dim);
  if (T < 0) return fail(PA_ERR_INVALID, "T must be >= 0");
  if (n_q_heads < 1) return fail(PA_ERR_INVALID, "n_q_heads must be >= 1");
  // the items of a token are counted in 32 bits
  if ((long long)n_q_heads + 2ll * d.n_kv_heads > (1 << 20))
    return fail(PA_ERR_UNSUPPORTED, "at most 2^20 query, key and value heads together");
  if ((st = check_stride("q", q_stride, n_q_heads, d.head_dim))) return st;
  if ((st = check_stride("k", k_stride, d.n_kv_heads, d.head_dim))) return st;
  if ((st = check_stride("v", v_stride, d.n_kv_heads, d.head_dim))) return st;
  if (T == 0) return PA_OK;
  if (!q || !q_out || !k || !v || !positions_dev || !slot_mapping_dev) return fail(PA_ERR_INVALID, "null argument");
  if (((uintptr_t)q | (uintptr_t)q_out | (uintptr_t)k | (uintptr_t)v) & 15u)
    return fail(PA_ERR_INVALID, "q, q_out, k and v must be 16-byte aligned");
  if (q_out == q && q_stride != (size_t)n_q_heads * d.head_dim)
    return fail(PA_ERR_INVALID, "q_out may be q only when q is contiguous");
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  RopeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.qs = (long long)q_stride;
  a.ks = (long long)k_stride;
  a.vs = (long long)v_stride;
  a.pos = positions_dev;
  a.slots = slot_mapping_dev;
  a.T = T;
  a.Hq = n_q_heads;
  a.Hkv = d.n_kv_heads;
  a.num_slots = (long long)d.num_blocks * 16;
  a.kpool = pool->k + (size_t)layer * pool->layer_bytes;
  a.vpool = pool->v + (size_t)layer * pool->layer_bytes;
  a.k_scale = d.k_scale;
  a.v_scale = d.v_scale;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  a.err = err;
  a.rope = *rope;
  const int lay = rope->layout == PA_ROPE_INTERLEAVED ? ROPE_INTER : rope->rot_dim % 16 == 0 ? ROPE_HALF : ROPE_HALF_ODD;
  const bool full = rope->rot_dim == d.head_dim;
  if (ext) {
    a.qw = static_cast<const uint16_t*>(ext->q_weight);
    a.kw = static_cast<const uint16_t*>(ext->k_weight);
    a.q_wstride = a.k_wstride = ext->weights_per_head ? d.head_dim : 0;
    a.eps = ext->eps;
    a.w_offset = ext->offset;
    if (ext->axes) std::copy(ext->axes->axis, ext->axes->axis + 64, a.axis);
  }
  const RopeKernel kern =
      ext ? pick_kernel<true>(d.head_dim, d.kv_dtype, lay, full) : pick_kernel<false>(d.head_dim, d.kv_dtype, lay, full);
  a.warps_per_token = 1;
  while (a.warps_per_token < kRopeWarps && (long long)T * a.warps_per_token < kRopeFewWarps) a.warps_per_token *= 2;
  const unsigned q_ctas = (unsigned)((T - 1) / (kRopeWarps / a.warps_per_token) + 1);
  a.parts = 2u * (unsigned)((d.n_kv_heads + kRopeWarps - 1) / kRopeWarps);
  const long long ctas = q_ctas + (pool->block_scaled ? (long long)T * a.parts : 0);
  if (ctas > 0x7FFFFFFF) return fail(PA_ERR_UNSUPPORTED, "too many tokens and kv heads for one call");
  kern<<<(unsigned)ctas, kRopeWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "rope_and_cache launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_rope_init(const pa_rope_desc* d, const double* divisors, pa_rope* out) {
  if (!d || !out) return fail(PA_ERR_INVALID, "pa_rope_init: null argument");
  if (d->layout != PA_ROPE_HALF && d->layout != PA_ROPE_INTERLEAVED)
    return fail(PA_ERR_INVALID, "rotary layout %d is neither half nor interleaved", d->layout);
  if (d->rot_dim < 2 || d->rot_dim > 128 || d->rot_dim % 2 != 0)
    return fail(PA_ERR_INVALID, "rot_dim must be even, 2 to 128 (got %d)", d->rot_dim);
  if (d->scaling < PA_ROPE_SCALE_NONE || d->scaling > PA_ROPE_SCALE_YARN)
    return fail(PA_ERR_INVALID, "rotary scaling %d is not known", d->scaling);
  if (!(d->theta > 1.0) || !std::isfinite(d->theta)) return fail(PA_ERR_INVALID, "theta must be finite and above 1");
  if (!std::isfinite((float)d->gain)) return fail(PA_ERR_INVALID, "gain must be finite");
  if (d->scaling != PA_ROPE_SCALE_NONE && (!(d->factor > 0.0) || !std::isfinite(d->factor)))
    return fail(PA_ERR_INVALID, "the stretch factor must be finite and positive");
  if (d->scaling == PA_ROPE_SCALE_NTK && d->rot_dim == 2)
    return fail(PA_ERR_INVALID, "a raised base needs rot_dim > 2");
  const bool blend = d->scaling == PA_ROPE_SCALE_BANDS || d->scaling == PA_ROPE_SCALE_YARN;
  if (blend && (!(d->original_len > 0.0) || !std::isfinite(d->original_len) || !(d->low > 0.0) || !(d->high > d->low) ||
                !std::isfinite(d->high)))
    return fail(PA_ERR_INVALID, "need original_len > 0 and 0 < low < high, all finite");
  const int R = d->rot_dim;
  for (int i = 0; divisors && i < R / 2; ++i)
    if (!(divisors[i] > 0.0) || !std::isfinite(divisors[i]))
      return fail(PA_ERR_INVALID, "divisor %d must be finite and positive", i);
  const double two_pi = 6.283185307179586476925;
  const double theta = d->scaling == PA_ROPE_SCALE_NTK ? d->theta * std::pow(d->factor, (double)R / (R - 2)) : d->theta;
  // the (real-valued) index of the pair that makes `turns` turns over original_len
  auto index_of = [&](double turns) { return R * std::log(d->original_len / (two_pi * turns)) / (2.0 * std::log(theta)); };
  double lo = 0.0, hi = 0.0;
  if (d->scaling == PA_ROPE_SCALE_YARN) {
    lo = std::fmax(std::floor(index_of(d->high)), 0.0);
    hi = std::fmin(std::ceil(index_of(d->low)), (double)(R - 1));
  }
  pa_rope r = {};
  r.layout = d->layout;
  r.rot_dim = R;
  r.gain = (float)d->gain;
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / R);
    if (d->scaling == PA_ROPE_SCALE_LINEAR) f /= d->factor;
    if (blend) {
      double g = d->scaling == PA_ROPE_SCALE_BANDS ? (d->original_len * f / two_pi - d->low) / (d->high - d->low)
                                                   : 1.0 - (i - lo) / std::fmax(hi - lo, 0.001);
      g = std::fmin(std::fmax(g, 0.0), 1.0);
      f = f * g + f / d->factor * (1.0 - g);
    }
    if (divisors) f /= divisors[i];
    double turns = f / two_pi;
    if (!std::isfinite(turns)) return fail(PA_ERR_INVALID, "pair %d's speed is not finite", i);
    turns -= std::floor(turns);  // whole turns per position change nothing
    // 2^64 turns would not fit: the largest double below 1 gives 2^64 - 2^11
    r.step[i] = (uint64_t)std::ldexp(turns, 64);
  }
  *out = r;
  return PA_OK;
}

int pa_rope_and_cache(pa_pool* pool, int layer, const pa_rope* rope, const void* q, size_t q_stride, void* q_out,
                      int n_q_heads, const void* k, size_t k_stride, const void* v, size_t v_stride,
                      const int32_t* positions_dev, const int64_t* slot_mapping_dev, int T, void* stream) {
  pa::TraceRange trace_("pa_rope_and_cache");
  return rope_call(pool, layer, rope, nullptr, q, q_stride, q_out, n_q_heads, k, k_stride, v, v_stride, positions_dev,
                   slot_mapping_dev, T, stream);
}

int pa_norm_rope_and_cache(pa_pool* pool, int layer, const pa_rope* rope, const pa_rope_axes* axes, const void* q_weight,
                           const void* k_weight, int weights_per_head, float eps, float weight_offset, const void* q,
                           size_t q_stride, void* q_out, int n_q_heads, const void* k, size_t k_stride, const void* v,
                           size_t v_stride, const int32_t* positions_dev, const int64_t* slot_mapping_dev, int T,
                           void* stream) {
  pa::TraceRange trace_("pa_norm_rope_and_cache");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(PA_ERR_INVALID, "eps must be finite and at least 0");
  if (!std::isfinite(weight_offset)) return fail(PA_ERR_INVALID, "weight_offset must be finite");
  if (weights_per_head != 0 && weights_per_head != 1) return fail(PA_ERR_INVALID, "weights_per_head must be 0 or 1");
  if (((uintptr_t)q_weight | (uintptr_t)k_weight) & 15u)
    return fail(PA_ERR_INVALID, "the weights must be 16-byte aligned");
  if (axes) {
    if (axes->n_axes < 1 || axes->n_axes > PA_ROPE_MAX_AXES)
      return fail(PA_ERR_INVALID, "n_axes must be 1 to %d (got %d)", PA_ROPE_MAX_AXES, axes->n_axes);
    for (int i = 0; i < 64; ++i)
      if (axes->axis[i] >= axes->n_axes)
        return fail(PA_ERR_INVALID, "pair %d turns with axis %d of %d", i, (int)axes->axis[i], axes->n_axes);
  }
  const RopeExt ext = {q_weight, k_weight, weights_per_head, eps, weight_offset, axes};
  return rope_call(pool, layer, rope, &ext, q, q_stride, q_out, n_q_heads, k, k_stride, v, v_stride, positions_dev,
                   slot_mapping_dev, T, stream);
}

}  // extern "C"
