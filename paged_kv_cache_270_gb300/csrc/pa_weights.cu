// pa_weights.cu -- decode attention that also adds up the attention each cached
// token gets ("Capítulo 8 -- Gestión de caché KV de nueva generación", section
// 8.2: eviction by accumulated attention).
//
// With x the scaled scores (log2 units), M their maximum and L the sum of
// 2^(x - M) over a row, token t's weight is sum over the group's heads of
// 2^(x - M) / L.  M and L are known only once the whole row has been read, and
// K must not be read twice (it is half of all traffic): the scored build of the
// balanced decode kernel keeps every score, G floats per (kv head, token), in
// the workspace.  Rows that one CTA streams whole are weighed by it, from scores
// that are still in L2; rows split over CTAs by the kernel below.  For these each
// (kv head, token) costs 8 G bytes more than the 2 D e bytes of K and V (25% for
// FP8 at D = 128, G = 8; 6% for 16 bits, G = 4), where reading K again would
// cost D e (50%).
//
// Measured against pa_decode's balanced schedule: 256 x 4096 tokens of FP8, G =
// 8, 396 us against 326 (the totals' own bytes are 10 of the difference); 4 x
// 131072, 209 against 165; 64 ragged sequences of bf16, G = 4, 101 against 91.
// Other groups, 128 x 4096 tokens of FP8 (plain 164-171): G = 1 182, 2 199, 3 and 4
// 196, 5 and 6 233 (add_weights takes them two heads at a time), 7 and 8 211.
// Dropping used scores from L2 took 24 us off the first and 11 off the second (HBM
// writes of the decode kernel 220 -> 87 MB); the L2 hint on the stores another 9.
// Tried and slower, against 390 us: weighing a unit page by page inside the
// consumers' loop (539) or on the producer warp (544), for either becomes the pace
// of the stream.
#include <mutex>

#include "pa_decode_core.cuh"

namespace pa {
namespace {

// When a CTA takes whole units (one kernel) in the place of equal ranges (two):
// the pages of the busiest CTA are at most kWholeMost, and at most kWholeExtra
// more than an equal share, if every context is as long as its table.  Measured
// both ways (us, one kernel against two): 8 units of 7 pages 7.2 / 12.3, of 16
// 9.2 / 10.7, of 32 13.0 / 10.6; 256 units of 32 pages (14 extra) 19.8 / 22.6, of
// 64 (28) 32.3 / 31.8; 512 of 64 (10) 33.9 / 45.0, of 128 (20) 57.1 / 63.3 and
// 46.4 / 45.1 with most contexts half as long; 800 of 32 (22) 39.5 / 41.6.
constexpr int kWholeMost = 128, kWholeExtra = 20;
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;

// Scores kept per token: G, or an even number for the 8-byte stores.
int score_heads(int G) { return G == 1 ? 1 : (G + 1) & ~1; }

// One CTA per CTA of the decode kernel, over the same range of the schedule.
// For every unit (sequence, kv head) of which the range holds a part: the
// rows' (M, 1 / L) from all the unit's pieces, then the weights of the range's
// tokens.  The output rows of a unit that spans n CTAs are merged by those n
// CTAs, each a slice of the G x D values.  (Whole units are done.)  Of the 396 and
// 209 us above, 22 and 17 are this kernel: 8 of launch, dependent reads and merge, the
// rest the scores, most of them still in L2.  Bulk copies through shared memory,
// or one CTA per range end, were no faster.
template <int KV, int D, int OUT>
__global__ void __launch_bounds__(kFinishThreads, 4) weights_finish_kernel(const DecodeArgs a) {
  constexpr int kUnit = BalCfg<KV, D>::kUnitCostPages;
  __shared__ float2 s_ml[8];  // (M, 1 / L) of the unit's heads
  __shared__ float s_inv[8];  // 1 / L for the output rows: 0 where no score was finite
  __shared__ float s_red[kFinishWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  const RangeStart rs = a.ranges[blockIdx.x];
  if (rs.seq < 0) return;
  int seq = rs.seq;
  int ctx = clamp_ctx(a.ctx[seq], a.max_blocks);
  int npages = (ctx + 15) >> 4;
  if (npages == 0) return;  // the lengths changed under the kernel
  int h = (int)((rs.pos_begin - rs.cost) / (npages + kUnit));
  long long ucost = rs.cost + (long long)h * (npages + kUnit);  // position of the unit's start

  while (ucost < rs.pos_end && h < a.Hkv) {
    // the unit's pages in this range
    const long long first = ucost + kUnit;  // position of page 0
    const int pg0 = (int)max(0LL, rs.pos_begin - first), pg1 = (int)min((long long)npages, rs.pos_end - first);
    if (pg1 > pg0 && (pg0 > 0 || pg1 < npages)) {
      const size_t row0 = (size_t)seq * a.Hq + (size_t)h * a.G;
      // pieces: CTA c0's partial, in the slot it recorded, and the first
      // partials of CTAs c0 + 1 .. c1
      const int c0 = (int)(first / rs.T), c1 = min((int)((first + npages - 1) / rs.T), a.ctas - 1);
      const int n = c1 - c0 + 1, slot0 = 2 * c0 + (a.jobs[c0].w & 1);
      if (warp < a.gs) {
        float M = -INFINITY, L = 0.f;
        for (int i = lane; i < n && warp < a.G; i += 32) {
          const size_t p = (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * a.G + warp;
          const float m = a.ws_ml[2 * p], l = a.ws_ml[2 * p + 1];
          const float mn = fmaxf(M, m);
          if (mn != -INFINITY) {
            L = L * fast_exp2(M - mn) + l * fast_exp2(m - mn);
            M = mn;
          }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const float m = __shfl_xor_sync(kFull, M, off), l = __shfl_xor_sync(kFull, L, off);
          const float mn = fmaxf(M, m);
          if (mn != -INFINITY) {
            L = L * fast_exp2(M - mn) + l * fast_exp2(m - mn);
            M = mn;
          }
        }
        if (lane == 0) {
          s_ml[warp] = warp < a.G ? make_float2(M, 1.f / L) : make_float2(0.f, 0.f);
          s_inv[warp] = L > 0.f ? 1.f / L : 0.f;
        }
      }
      __syncthreads();
      // this CTA's slice of the output rows, 32 values at a time.  Few pieces: a
      // warp per 32 values adds them all up, its loads in flight together.  Many:
      // the warps take the pieces in turn and are added up in warp order.
      const int groups = a.G * D / 32, slices = min(n, groups), me = (int)blockIdx.x - c0;
      const int g0 = me * groups / slices, g1 = me < slices && me >= 0 ? (me + 1) * groups / slices : g0;
      auto piece = [&](int i) { return (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * a.G; };
      if (n <= kFinishWarps) {
        for (int gi = g0 + warp; gi < g1; gi += kFinishWarps) {
          const int head = gi * 32 / D, dim = gi * 32 % D + lane;
          float m[kFinishWarps], o[kFinishWarps];
#pragma unroll
          for (int i = 0; i < kFinishWarps; ++i) {
            m[i] = -INFINITY;
            o[i] = 0.f;
            if (i < n) {
              m[i] = a.ws_ml[2 * (piece(i) + head)];
              o[i] = a.ws_o[(piece(i) + head) * D + dim];
            }
          }
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < kFinishWarps; ++i) sum += m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - s_ml[head].x) * o[i];
          store_out<OUT>(a.out, (row0 + head) * D + dim, s_inv[head] > 0.f ? sum * s_inv[head] * a.v_scale : 0.f);
        }
      } else {
        for (int gi = g0; gi < g1; ++gi) {
          const int head = gi * 32 / D, dim = gi * 32 % D + lane;
          float O = 0.f;
          for (int i0 = warp; i0 < n; i0 += 4 * kFinishWarps) {
            float m[4], o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int i = i0 + j * kFinishWarps;
              m[j] = -INFINITY;
              o[j] = 0.f;
              if (i < n) {
                m[j] = a.ws_ml[2 * (piece(i) + head)];
                o[j] = a.ws_o[(piece(i) + head) * D + dim];
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) O += m[j] == -INFINITY ? 0.f : fast_exp2(m[j] - s_ml[head].x) * o[j];
          }
          s_red[warp][lane] = O;
          __syncthreads();
          if (warp == 0) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kFinishWarps; ++w) sum += s_red[w][lane];
            store_out<OUT>(a.out, (row0 + head) * D + dim, s_inv[head] > 0.f ? sum * s_inv[head] * a.v_scale : 0.f);
          }
          __syncthreads();
        }
      }
      // ---- the weights of tokens [16 pg0, min(ctx, 16 pg1))
      const size_t unit = (size_t)seq * a.Hkv + h, row = unit * a.w_stride;
      add_weights<kFinishThreads, 2>(a.scores + unit * a.max_blocks * 16 * a.gs, a.gs, s_ml,
                                     a.w_in ? a.w_in + row : nullptr, a.w_out + row, a.decay, 16 * pg0,
                                     totals_end(min(ctx, 16 * pg1), a));
      __syncthreads();  // s_ml is free again
    }
    ucost += npages + kUnit;
    if (++h == a.Hkv) {
      h = 0;
      do {
        if (++seq >= a.S) return;
        ctx = clamp_ctx(a.ctx[seq], a.max_blocks);
      } while (ctx == 0);
      npages = (ctx + 15) >> 4;
    }
  }
}

// ---------------------------------------------------------------- host side
struct Kernels {
  const void* decode;
  int smem;
  cudaError_t (*launch)(const DecodeArgs&, const CUtensorMap*, const CUtensorMap*, cudaStream_t);
  int* occupancy;  // [128], per device; 0 = not yet configured
};

template <int KV, int D, int OUT>
struct Build {
  // The weights keep their precision in the product with V, also for 16-bit outputs (a
  // second product with what rounding them to 16 bits drops).  With one product the
  // bf16 output of FP8 pages is off from a value rounded once by 7e-4 of its norm, with
  // two by 1e-4.  The second one costs 256 x 4096 tokens of FP8 390 -> 395 us, with a
  // scale per tile 406 -> 414, 4 x 131072 nothing that shows (208).
  static constexpr bool kPsplit = true;
  static constexpr int kMinB = std::min(Cfg<KV, D>::kMinBlocks, 4);  // the schedule puts at most four CTAs on an SM
  static constexpr auto kDecode = &decode_bal_kernel<KV, D, OUT, kPsplit, kMinB, true>;
  static cudaError_t launch(const DecodeArgs& a, const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = BalCfg<KV, D>::kLaunchSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kDecode, a, *tk, *tv);
    if (e != cudaSuccess || a.whole) return e;
    cfg.blockDim = dim3(kFinishThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, weights_finish_kernel<KV, D, OUT>, a);
  }
  static Kernels get() {
    static int occupancy[128];
    return {reinterpret_cast<const void*>(kDecode), BalCfg<KV, D>::kLaunchSmem, &launch, occupancy};
  }
};

template <int KV>
Kernels pick(int head_dim, int out_dtype) {
  constexpr int kOut16 = KV == KV_F16 ? OUT_F16 : OUT_BF16;
  if (head_dim == 64) return out_dtype == PA_FP32 ? Build<KV, 64, OUT_F32>::get() : Build<KV, 64, kOut16>::get();
  return out_dtype == PA_FP32 ? Build<KV, 128, OUT_F32>::get() : Build<KV, 128, kOut16>::get();
}

Kernels pick(int kv_dtype, int head_dim, int out_dtype) {
  switch (kv_dtype) {
    case PA_FP16:
      return pick<KV_F16>(head_dim, out_dtype);
    case PA_BF16:
      return pick<KV_BF16>(head_dim, out_dtype);
    case PA_FP8_E4M3_BLOCK:
      return pick<KV_E4M3B>(head_dim, out_dtype);
    default:
      return pick<KV_E4M3>(head_dim, out_dtype);
  }
}

// Sets the shared-memory opt-in once per device; the CTAs of a launch: one per
// resident slot, at most four per SM.
int configure(const Kernels& k, int* ctas) {
  static std::mutex mu;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess || dev < 0 || dev >= 128) return fail(PA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  std::lock_guard<std::mutex> lock(mu);
  if (k.occupancy[dev] == 0) {
    int occ = 0;
    e = cudaFuncSetAttribute(k.decode, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k.decode, kThreads, k.smem);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "decode kernel configuration: %s", cudaGetErrorString(e));
    k.occupancy[dev] = std::max(occ, 1);
  }
  *ctas = std::min(k.occupancy[dev], 4) * sms;
  return PA_OK;
}

// Parts of the workspace, in floats.
struct Workspace {
  size_t ml, jobs, ranges, scores, total;
};

Workspace layout(int ctas, int S, int Hq, int Hkv, int D, int max_blocks) {
  const size_t G = Hq / Hkv;
  auto up = [](size_t n) { return (n + 3) / 4 * 4; };  // 16-byte parts
  Workspace w;
  w.ml = up(2 * (size_t)ctas * G * D);
  w.jobs = w.ml + up(2 * (size_t)ctas * G * 2);
  w.ranges = w.jobs + 4 * (size_t)ctas;
  w.scores = w.ranges + up(sizeof(RangeStart) / 4 * (size_t)ctas) + 28;  // room to start on a 128-byte line
  w.total = w.scores + (size_t)S * Hkv * max_blocks * 16 * score_heads((int)G);
  return w;
}

// Tokens are indexed in 32 bits, up to 4096 past the last one of a row (a round of
// the weighing).
int check_width(int max_blocks) {
  if (max_blocks > (1 << 27) - 256)
    return fail(PA_ERR_UNSUPPORTED, "tables of at most 2^27 - 256 blocks (got %d)", max_blocks);
  return PA_OK;
}

}  // namespace

int weights_set_wait_limit(unsigned long long ns) { return (int)set_pipe_wait_limit_here(ns); }

}  // namespace pa

using namespace pa;

extern "C" {

int pa_decode_weights_workspace_bytes(const pa_pool* pool, int S, int n_q_heads, int max_blocks_per_seq,
                                      size_t* bytes) {
  int st = check_shape(pool, S, n_q_heads, max_blocks_per_seq);
  if (st) return st;
  if ((st = check_width(max_blocks_per_seq))) return st;
  if (!bytes) return fail(PA_ERR_INVALID, "null output");
  const pa_pool_desc& d = pool->desc;
  // the size does not depend on the output dtype: that of the query dtype's build
  int ctas = 0;
  st = configure(pick(d.kv_dtype, d.head_dim, in_dtype_of(d.kv_dtype)), &ctas);
  if (st) return st;
  *bytes = layout(ctas, std::min(S, kBalancedMaxSeqs), n_q_heads, d.n_kv_heads, d.head_dim, max_blocks_per_seq).total *
           sizeof(float);
  return PA_OK;
}

int pa_decode_weights(pa_pool* pool, int layer, void* out, int out_dtype, const void* q,
                      const int32_t* block_tables_dev, int max_blocks_per_seq, const int32_t* ctx_lens_dev, int S,
                      int n_q_heads, float softmax_scale, const float* weights_in, float* weights_out,
                      size_t weights_stride, float decay, void* workspace, size_t workspace_bytes, void* stream) {
  pa::TraceRange trace_("pa_decode_weights");
  int st = check_decode_args(pool, layer, out_dtype, S, n_q_heads, max_blocks_per_seq, softmax_scale);
  if (st) return st;
  if ((st = check_width(max_blocks_per_seq))) return st;
  if (!std::isfinite(decay)) return fail(PA_ERR_INVALID, "decay must be finite");
  if (weights_stride < 1 || weights_stride >= (size_t)1 << 40)
    return fail(PA_ERR_INVALID, "weights_stride must be at least 1 and below 2^40");
  if (S == 0) return PA_OK;
  st = check_decode_ptrs(out, q, block_tables_dev, ctx_lens_dev);
  if (st) return st;
  if (!weights_out) return fail(PA_ERR_INVALID, "null weights_out");
  if (((uintptr_t)weights_in | (uintptr_t)weights_out) & 15u)
    return fail(PA_ERR_INVALID, "the weights must be 16-byte aligned");
  if (!workspace || ((uintptr_t)workspace & 15u))
    return fail(PA_ERR_INVALID, "a 16-byte aligned workspace is needed");
  const pa_pool_desc& d = pool->desc;
  const int Hkv = d.n_kv_heads, D = d.head_dim;
  int ctas = 0, own_ctas = 0;
  st = configure(pick(d.kv_dtype, D, in_dtype_of(d.kv_dtype)), &ctas);
  if (st) return st;
  const Kernels k = pick(d.kv_dtype, D, out_dtype);
  st = configure(k, &own_ctas);
  if (st) return st;
  const Workspace ws = layout(ctas, std::min(S, kBalancedMaxSeqs), n_q_heads, Hkv, D, max_blocks_per_seq);
  if (workspace_bytes < ws.total * sizeof(float))
    return fail(PA_ERR_INVALID, "workspace of %zu bytes needed, %zu given", ws.total * sizeof(float), workspace_bytes);
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  const CUtensorMap *tk = nullptr, *tv = nullptr;
  try {
    st = layer_maps(pool, layer, &tk, &tv);
  } catch (...) {  // (the pool's first use of a layer allocates its map on the host)
    return fail(PA_ERR_NO_MEMORY, "host allocation failed");
  }
  if (st) return st;

  DecodeArgs a = {};
  float* base = static_cast<float*>(workspace);
  a.ws_o = base;
  a.ws_ml = base + ws.ml;
  a.jobs = reinterpret_cast<int4*>(base + ws.jobs);
  a.ranges = reinterpret_cast<RangeStart*>(base + ws.ranges);
  a.scores = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(base + ws.scores) & ~(uintptr_t)127);
  a.G = n_q_heads / Hkv;
  a.gs = score_heads(a.G);
  a.max_blocks = max_blocks_per_seq;
  a.Hq = n_q_heads;
  a.Hkv = Hkv;
  a.num_blocks = d.num_blocks;
  a.ctas = ctas;
  a.qk_scale_log2 = softmax_scale * 1.4426950408889634f * (d.kv_dtype == PA_FP8_E4M3 ? d.k_scale : 1.f);
  a.v_scale = d.kv_dtype == PA_FP8_E4M3 ? d.v_scale : 1.f;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  a.err = err;
  a.w_stride = (long long)weights_stride;
  a.decay = decay;
  const long long units = (long long)std::min(S, kBalancedMaxSeqs) * Hkv;
  const long long most = (units + ctas - 1) / ctas * max_blocks_per_seq, share = units * max_blocks_per_seq / ctas;
  a.whole = most <= kWholeMost && most - share <= kWholeExtra;
  // one schedule holds at most kBalancedMaxSeqs sequences: larger batches in turn
  for (int s = 0; s < S; s += kBalancedMaxSeqs) {
    a.S = std::min(S - s, kBalancedMaxSeqs);
    a.q = static_cast<const uint16_t*>(q) + (size_t)s * n_q_heads * D;
    a.out = static_cast<uint8_t*>(out) + (size_t)s * n_q_heads * D * (out_dtype == PA_FP32 ? 4 : 2);
    a.tables = block_tables_dev + (size_t)s * max_blocks_per_seq;
    a.ctx = ctx_lens_dev + s;
    const size_t at = (size_t)s * Hkv * weights_stride;
    a.w_in = weights_in ? weights_in + at : nullptr;
    a.w_out = weights_out + at;
    const cudaError_t e = k.launch(a, tk, tv, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "decode_weights launch: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

}  // extern "C"
