// pa_rope.cu -- rotary positions fused with the write into the paged KV pool.
//
// Pair i of a head turns by p f_i at position p.  The kernel needs that angle
// modulo a turn, for positions up to 2^31: an fp32 product would be off by a
// tenth of a radian at a million, and fp64 runs at a small fraction of the
// fp32 rate on this part.  So the speed is kept as a 64-bit binary fraction of
// a turn, F_i = f_i / (2 pi) * 2^64: p F_i modulo 2^64 is the angle's fraction
// of a turn, one integer multiply with no reduction step, and its upper bits as a
// signed fraction of half a turn are the argument of sincospi.
//
// The work is a copy with some arithmetic in it, bound by HBM: 16-byte loads
// and stores, each thread owning both halves of eight pairs, and the
// sin / cos of a token computed once per CTA, in shared memory, for all
// its heads.
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

constexpr int kRopeMaxTokens = 8;  // tokens per CTA when the heads are few

struct RopeArgs {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  const uint16_t* v;
  long long qs, ks, vs;  // token strides, elements
  const int32_t* pos;
  const int64_t* slots;
  int T, Hq, Hkv;
  int tokens_per_cta;
  long long num_slots;
  uint8_t* kpool;
  uint8_t* vpool;
  float k_scale, v_scale;  // PA_FP8_E4M3
  float* ksc;              // PA_FP8_E4M3_BLOCK
  float* vsc;
  unsigned int* err;
  pa_rope rope;
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

template <int LAY>
__device__ __forceinline__ void load_unit(const uint16_t* row, int u, int rot, bool turns, UnitIn<LAY>& in) {
  int v0, v1;
  unit_vecs<LAY>(u, rot, v0, v1);
  in.x0 = *reinterpret_cast<const uint4*>(row + 8 * v0);
  in.x1 = *reinterpret_cast<const uint4*>(row + 8 * v1);
  if constexpr (LAY == ROPE_HALF_ODD) {
    const int half = rot >> 1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int e = 16 * u + j;
      in.partner[j] = turns && e < rot ? row[e < half ? e + half : e - half] : 0;
    }
  }
}

// The unit's 16 values after the rotation (turns) or as they are.
template <bool BF, int D, int LAY>
__device__ __forceinline__ void turn_unit(const UnitIn<LAY>& in, int u, int rot, bool turns, const float2* cs,
                                          float (&y)[16]) {
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
  if (!turns) return;
  if constexpr (LAY == ROPE_HALF) {
    if (u >= (rot >> 4)) return;
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
      if (16 * u + 4 * j < rot) {
        y[4 * j] = a0 * t.x - b0 * t.y;
        y[4 * j + 1] = b0 * t.x + a0 * t.y;
      }
      if (16 * u + 4 * j + 2 < rot) {
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
        const float2 p2 = unpack2<BF>(in.partner[j]);
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

// Rows [0, rows) of `ntok` tokens from t0 on: row r < Hq is query head r, then
// the key and the value heads.  A CTA takes its items (token, row, unit)
// IPT at a time per thread, every load of a batch issued before the first use.
template <bool BF, bool FP8, int D, int LAY>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, int t0, int ntok, int rows, float2 (*cs)[D / 2]) {
  constexpr int UNITS = D / 16, IPT = LAY == ROPE_HALF_ODD ? 1 : 2;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int rot = a.rope.rot_dim;
  const int per_token = rows * UNITS, total = ntok * per_token;
  for (int base = 0; base < total; base += nt * IPT) {
    UnitIn<LAY> in[IPT];
    int tok[IPT], row[IPT], unit[IPT];
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
      const int item = base + k * nt + tid;
      row[k] = -1;
      if (item < total) {
        tok[k] = item / per_token;
        const int r = item - tok[k] * per_token;
        row[k] = r / UNITS;
        unit[k] = r % UNITS;
        const long long t = t0 + tok[k];
        const uint16_t* src = row[k] < a.Hq            ? a.q + t * a.qs + (long long)row[k] * D
                              : row[k] < a.Hq + a.Hkv ? a.k + t * a.ks + (long long)(row[k] - a.Hq) * D
                                                      : a.v + t * a.vs + (long long)(row[k] - a.Hq - a.Hkv) * D;
        load_unit<LAY>(src, unit[k], rot, row[k] < a.Hq + a.Hkv, in[k]);
      }
    }
    if (base == 0) {  // the tokens' tables, while the first loads are in flight
      for (int i = tid; i < ntok * (rot >> 1); i += nt) {
        const int tk = i / (rot >> 1), p = i - tk * (rot >> 1);
        cs[tk][cs_index<D, LAY>(p)] = turn(a.rope, p, a.pos[t0 + tk]);
      }
      __syncthreads();
    }
    // A row's units sit in one warp: with q_out == q its partners are read
    // (above) before any lane writes the row.
    __syncwarp();
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
      if (row[k] < 0) continue;
      int v0, v1;
      unit_vecs<LAY>(unit[k], rot, v0, v1);
      const long long t = t0 + tok[k];
      const bool is_v = row[k] >= a.Hq + a.Hkv;
      float y[16];
      turn_unit<BF, D, LAY>(in[k], unit[k], rot, !is_v, cs[tok[k]], y);
      if (row[k] < a.Hq) {
        uint16_t* dst = a.q_out + (t * a.Hq + row[k]) * D;
        *reinterpret_cast<uint4*>(dst + 8 * v0) = pack8<BF>(y);
        *reinterpret_cast<uint4*>(dst + 8 * v1) = pack8<BF>(y + 8);
        continue;
      }
      const int64_t slot = a.slots[t];
      if (slot < 0) continue;
      if (slot >= a.num_slots) {
        record_error(a.err, PA_ERR_BOUNDS);
        continue;
      }
      const int h = row[k] - a.Hq - (is_v ? a.Hkv : 0);
      const long long e = (((slot >> 4) * a.Hkv + h) * 16 + (slot & 15)) * (long long)D;
      uint8_t* pool = is_v ? a.vpool : a.kpool;
      if constexpr (FP8) {
        const float s = is_v ? a.v_scale : a.k_scale;
        *reinterpret_cast<uint2*>(pool + e + 8 * v0) = codes8(y, s);
        *reinterpret_cast<uint2*>(pool + e + 8 * v1) = codes8(y + 8, s);
      } else {
        *reinterpret_cast<uint4*>(pool + 2 * (e + 8 * v0)) = is_v ? in[k].x0 : pack8<BF>(y);
        *reinterpret_cast<uint4*>(pool + 2 * (e + 8 * v1)) = is_v ? in[k].x1 : pack8<BF>(y + 8);
      }
    }
  }
}

template <bool BF, bool FP8, int D, int LAY>
__global__ void __launch_bounds__(320) rope_cache_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 cs[kRopeMaxTokens][D / 2];
  grid_dependents_launch();  // a decode behind this kernel waits for its writes itself
  const int t0 = blockIdx.x * a.tokens_per_cta;
  rope_rows<BF, FP8, D, LAY>(a, t0, min(a.tokens_per_cta, a.T - t0), a.Hq + 2 * a.Hkv, cs);
}

// Block-scaled pools: CTA (t, 0) turns token t's queries; CTA (t, y > 0) takes,
// if t starts a run (see reshape_block_scaled_kernel), eight (K or V, head)
// tiles of the run, one per warp.  A run's rows of one tile, at most 16 x D
// values, stay in the warp's registers between the maximum and the encoding.
template <int D, int LAY>
__global__ void __launch_bounds__(256) rope_cache_block_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 cs[16][D / 2];
  grid_dependents_launch();
  const int t = blockIdx.x;
  if (blockIdx.y == 0) {
    rope_rows<true, true, D, LAY>(a, t, 1, a.Hq, cs);
    return;
  }
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 1) record_error(a.err, PA_ERR_BOUNDS);
    return;
  }
  const int off0 = (int)(slot & 15);
  if (t > 0 && off0 != 0 && a.slots[t - 1] == slot - 1) return;  // not the first token of its run
  int n = 1;
  while (n < 16 - off0 && t + n < a.T && a.slots[t + n] == slot + n) ++n;
  const int rot = a.rope.rot_dim;
  for (int i = threadIdx.x; i < n * (rot >> 1); i += blockDim.x) {
    const int tk = i / (rot >> 1), p = i - tk * (rot >> 1);
    cs[tk][cs_index<D, LAY>(p)] = turn(a.rope, p, a.pos[t + tk]);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit_id = (blockIdx.y - 1) * 8 + warp;
  if (unit_id >= 2 * a.Hkv) return;
  const bool is_v = unit_id >= a.Hkv;
  const int h = unit_id - (is_v ? a.Hkv : 0);
  const uint16_t* src = (is_v ? a.v : a.k) + (long long)h * D;
  const long long stride = is_v ? a.vs : a.ks;
  const size_t sidx = (size_t)(slot >> 4) * a.Hkv + h;
  float* scp = (is_v ? a.vsc : a.ksc) + sidx;
  const float s_old = off0 > 0 ? *scp : 0.f;
  constexpr int UNITS = D / 16, ROWS = 32 / UNITS, ITERS = 16 / ROWS;
  const int u = lane % UNITS, r0 = lane / UNITS;
  float y[ITERS][16];
  uint32_t mb = 0;  // largest |y|: without the sign bit, magnitudes order like their bits (a NaN above all)
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = i * ROWS + r0;
    if (r < n) {
      UnitIn<LAY> in;
      load_unit<LAY>(src + (t + r) * stride, u, rot, !is_v, in);
      turn_unit<true, D, LAY>(in, u, rot, !is_v, cs[r], y[i]);
#pragma unroll
      for (int j = 0; j < 16; ++j) mb = max(mb, __float_as_uint(y[i][j]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
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
  for (int i = 0; i < ITERS; ++i) {
    const int r = i * ROWS + r0;
    if (r < n) {
      int v0, v1;
      unit_vecs<LAY>(u, rot, v0, v1);
      uint8_t* dst = tile + (size_t)(off0 + r) * D;
      *reinterpret_cast<uint2*>(dst + 8 * v0) = codes8(y[i], s);
      *reinterpret_cast<uint2*>(dst + 8 * v1) = codes8(y[i] + 8, s);
    }
  }
  if (lane == 0) *scp = s;
}

// ---------------------------------------------------------------- host side
typedef void (*RopeKernel)(RopeArgs);

template <bool BF, bool FP8, int D>
RopeKernel pick_lay(int lay) {
  return lay == ROPE_HALF    ? rope_cache_kernel<BF, FP8, D, ROPE_HALF>
         : lay == ROPE_INTER ? rope_cache_kernel<BF, FP8, D, ROPE_INTER>
                             : rope_cache_kernel<BF, FP8, D, ROPE_HALF_ODD>;
}

template <int D>
RopeKernel pick_kernel(int kv_dtype, int lay) {
  if (kv_dtype == PA_FP8_E4M3_BLOCK)
    return lay == ROPE_HALF    ? rope_cache_block_kernel<D, ROPE_HALF>
           : lay == ROPE_INTER ? rope_cache_block_kernel<D, ROPE_INTER>
                               : rope_cache_block_kernel<D, ROPE_HALF_ODD>;
  if (kv_dtype == PA_FP8_E4M3) return pick_lay<true, true, D>(lay);
  return kv_dtype == PA_BF16 ? pick_lay<true, false, D>(lay) : pick_lay<false, false, D>(lay);
}

int check_stride(const char* name, size_t stride, int heads, int head_dim) {
  if (stride < (size_t)heads * head_dim || stride % 8 != 0 || stride >= (size_t)1 << 40)
    return fail(PA_ERR_INVALID, "%s_stride %zu must be a multiple of 8, at least %zu and below 2^40", name, stride,
                (size_t)heads * head_dim);
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
  RopeArgs a;
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
  const RopeKernel kern = d.head_dim == 64 ? pick_kernel<64>(d.kv_dtype, lay) : pick_kernel<128>(d.kv_dtype, lay);
  dim3 grid;
  int threads = 256;
  if (pool->block_scaled) {
    const int tiles = (2 * d.n_kv_heads + 7) / 8;
    if (tiles > 65534) return fail(PA_ERR_UNSUPPORTED, "too many kv heads for one call");
    a.tokens_per_cta = 1;
    grid = dim3(T, 1 + tiles);
  } else {
    // A CTA takes whole tokens, about 256 items at least; a token of more than
    // 320 items is taken in even rounds.
    const int items = (n_q_heads + 2 * d.n_kv_heads) * (d.head_dim / 16);
    a.tokens_per_cta = items >= 256 ? 1 : std::min(kRopeMaxTokens, 256 / items);
    const int all = items * a.tokens_per_cta, rounds = (all + 319) / 320;
    threads = (all + rounds * 32 - 1) / (rounds * 32) * 32;
    grid = dim3((T - 1) / a.tokens_per_cta + 1);
  }
  kern<<<grid, threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "rope_and_cache launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
