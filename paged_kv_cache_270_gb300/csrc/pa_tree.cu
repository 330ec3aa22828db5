// pa_tree.cu -- attention of a tree of drafted tokens per sequence over the paged KV cache.
//
// A node's result is softmax(scale q K^T) V over its sequence's history and the nodes whose
// bits its mask row has.  All the nodes of a sequence read the same pages, so per kv
// head their queries are the rows of one matrix product with K and one with V:
// nodes x G rows, up to 128 of them (a tile) on the tcgen05 tensor cores, and the pages
// are read once per tile.  K and V are the bytes that the work cannot do without, and up
// to about 128 rows the products take no longer than HBM does to deliver them.
//
// The pipeline of a CTA is that of the chunked prefill (pa_prefill_tc.cu: operand layouts, the
// two E4M3 terms of a query, V converted to binary16, the two threads of a row, S and P in
// one buffer).  What differs:
//  * one CTA per SM for the whole call, and a schedule made on the device: the blocks of 128
//    keys of all (sequence, kv head, tile) units, in order, are cut into ranges of equal
//    cost, one per CTA (a unit costs kUnitCost blocks besides its own).  A range goes from
//    unit to unit without draining: the copies, the products and the softmax run on over
//    its pieces (segments), whose descriptions the copying warp hands to the other roles.
//  * a unit that spans several CTAs leaves partial states (O, m, l) per piece, which
//    tree_merge_kernel joins.  A long history is thus read by the whole GPU.
//  * the queries of the next segment are put into the second of two places in tensor memory
//    while this one runs.
//  * a mask: blocks that reach the tree take 64 bits per thread from the node's row.
//  * what a row does not see must not touch it.  A masked key's weight is 0, but 0 times an
//    infinity or a NaN among V is not: such values of nodes are taken out of the block in shared
//    memory, and put back for the rows that see them when the output is written.
//  * with a scale per tile, O's weights follow a reference of the row's own, the largest score plus log2 of its
//    tile's V scale among the keys that it sees: a tile that it does not see, or whose weight is small,
//    takes no bits from the others (24 sequences of 1000-9001 tokens, 40 / 8 heads: 166 us and 8).
//
// What bounds it: 16-bit pools HBM (64 sequences of 512-4096 tokens, 16 nodes of 32 / 8 heads, bf16:
// 104 us and 6 of the merge, 6.0 TB/s); FP8 pools the chain of hand-offs of a block (scores, maximum, weights, the
// second product), 2200-2450 cycles where HBM takes 1400 and the products 1030 (128 sequences of
// 4096, 16 nodes of 64 / 8 heads: 267 us and 8, 4.2 TB/s).  Trees above 128 rows read their pages once
// per tile and are bound by the same chain (4 of 131072, 32 nodes of 64 / 8 heads, two tiles: 490 us
// and 8, 0.60 of the products' rate, HBM at 55%).  Calls with little to read take their latency: 8 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "pa_tc.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kRows = 128;     // MMA rows of a tile: nodes x the G heads of a kv head
// 16 warps, four on each scheduler: 0 issues MMAs, 1 copies, 2 and 3 fetch masks, 4-11 softmax, 12-15
// take V, the queries of the segment ahead and the output of the one behind.  A warp reaches the 32 tensor-memory lanes of its
// number modulo 4, so a tile's rows are put into the highest lanes: with 96 rows or fewer the MMA
// warp's scheduler has no softmax warp at work.
constexpr int kThreads = 512;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kTmemCols = 512;
// TMEM columns (one lane per row): S in buffers of 128 at 0 and 128 by block parity, overwritten by
// P as in the prefill; O at 256; the queries of even segments at 384, of odd ones at 448 (FP8
// pools: the two E4M3 terms 32 columns apart).
constexpr uint32_t kOCol = 256, kQCol = 384;
constexpr int kScaleRing = 8;  // block-scaled pools: blocks whose scales are held
// Segments whose descriptions are held.  The copying warp hands out number c + 3 before it
// issues the copies of segment c, and the MMA warp gives up number s only once it has issued
// Q K^T of a block behind s, so c + 3 - kSegRing must lie two segments before c.
constexpr int kSegRing = 8;
constexpr int kRowRing = 4;  // segments whose masks and score factors are held
// The largest weight is kept near 2^7 and below 2^15, so that small ones stay normal
// binary16 numbers; the reference point moves when the maximum has grown by 2^8.
constexpr float kTop = 7.f, kGrow = 15.f;
constexpr float kMinFactor = 1.17549435e-38f;  // the smallest normal number

// Tables of at most this many pages are not split, which saves the merge and its launch: 16 sequences of 512 tokens
// 13.5 us, 18.0 split; 64 of 256 26.6, 29.9 split.  Of 2048 tokens 92 whole, 74 split.
constexpr int kWholePages = 32;

enum Kind { K_E4M3 = 0, K_E4M3B = 1, K_BF16 = 2, K_F16 = 3 };

template <int KIND, int D>
struct Lay {
  static constexpr bool kF8 = KIND == K_E4M3 || KIND == K_E4M3B;
  static constexpr bool kBlk = KIND == K_E4M3B;
  static constexpr bool kBf = KIND == K_BF16;
  static constexpr int kRow = D * (kF8 ? 1 : 2);       // bytes of a key
  static constexpr int kHalves = kRow == 256 ? 2 : 1;  // 128-byte parts, loaded and laid out apart
  static constexpr int kPart = kRow / kHalves;
  static constexpr int kSlot = 128 * kRow;  // a block of K, or of V
  static constexpr int kRing = kF8 || kSlot == 32768 ? 3 : 4;  // blocks of K, and of V
  static constexpr int kVT = 2 * kRing * kSlot;  // FP8: two blocks of V in binary16
  static constexpr int kVTBlock = 128 * D * 2;
  static constexpr int kQ = kVT + (kF8 ? 2 * kVTBlock : 0);  // FP8: the next segment's queries as they are
  static constexpr int kData = kQ + (kF8 ? kRows * D * 2 : 0);
  // a block needs kUnitCost more for its unit's queries and output rows
  static constexpr int kUnitCost = kF8 ? 3 : 2;
};

// A segment: blocks [b0, b1) of a unit; b1 == b0 ends the list.
struct Seg {
  int seq, h, tile, b0;
  int b1, n, base, q0;
  int nblk, last_cta, pad0, pad1;
};

struct Ctrl {
  Seg seg[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], vt_empty[2];
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing];
  uint64_t q_ready[2], q_free[2], row_free[kRowRing], o_full, o_free, drain;
  uint64_t tail_ready[2], tail_done[2];  // 16-bit pools: blocks that reach the tree, by their parity
  uint64_t mask[kRowRing][128][PA_TREE_MAX_NODES / 64];  // a tile's nodes' mask words
  float row_scale[kRowRing][128];        // each row's score factor
  float4 fin[kRowRing][128];             // each row's (m, 2^(r - m), the two threads' l) at the segment's end
  // block-scaled pools, each page of a block: K scale, log2 of the V scale, and the exponent and factor that the
  // weights take for it (16-bit outputs: all of the log2, and 1; fp32 outputs: a whole number, and what is left)
  float4 sc[kScaleRing][8];
  float2 xbuf[2][2][128];                // the two half-row threads' maxima (one scale: of floats)
  long long warp_sums[kThreads / 32];
  long long start_off;
  int start_seq;
  int bad[kScaleRing];  // segment j has infinities or NaN in its nodes' V or a tile without a finite scale: bad[j % 8] == j + 1
  uint32_t tmem;
  int abort;
};

template <int KIND, int D>
constexpr int smem_bytes() {
  // (at least 116 KiB: two CTAs on an SM would wait for each other's tensor memory)
  constexpr int n = 1024 + Lay<KIND, D>::kData + (int)sizeof(Ctrl);
  static_assert(n <= 232448, "shared memory budget");
  return n > 118784 ? n : 118784;
}

struct TreeArgs {
  const uint16_t* q;
  void* out;
  const uint64_t* mask;  // nullptr: chains
  const int32_t* q_start;
  const int32_t* tables;
  const int32_t* ctx;
  const uint8_t* v;  // this layer's V, for the values put back
  const float* ksc;  // block-scaled pools: this layer's scales [num_blocks][Hkv]
  const float* vsc;
  float* ws_o;       // [2 ctas][128][D]
  float2* ws_ml;     // [2 ctas][128] (m in log2 units, l)
  int4* jobs;        // [ctas] units to merge: (sequence, kv head and tile, last CTA, slot)
  int whole;         // CTAs take whole units
  int T, S, Hq, Hkv, G, tile_nodes, max_nodes, words, max_blocks, num_blocks, ctas;
  float qk_scale_log2;  // softmax_scale * log2(e) (* k_scale of a static FP8 pool)
  float v_scale;        // static FP8 pool's V scale, else 1
  int wide;             // out is 32-byte aligned
  unsigned int* err;
};

// A sequence's place in the schedule, from its lengths (loaded apart, so that the loads of the next
// one can be under way).
struct SeqRaw {
  int q0, q1, ctx;
};

__device__ __forceinline__ SeqRaw seq_raw(const TreeArgs& a, int s) {
  return s < a.S ? SeqRaw{a.q_start[s], a.q_start[s + 1], a.ctx[s]} : SeqRaw{0, 0, 0};
}

struct SeqInfo {
  int q0, n, ctx, tiles, nblk;
  bool bad;
  __device__ long long units(int Hkv) const { return (long long)tiles * Hkv; }
};

__device__ __forceinline__ SeqInfo seq_info(const TreeArgs& a, const SeqRaw& r) {
  SeqInfo i;
  i.q0 = r.q0;
  const long long n = (long long)r.q1 - r.q0;
  i.n = i.ctx = i.tiles = i.nblk = 0;
  i.bad = false;
  if (n == 0) return i;
  if (r.q0 < 0 || n < 0 || r.q1 > a.T || n > a.max_nodes || r.ctx < n || r.ctx > 16 * a.max_blocks) {
    i.bad = true;
    return i;
  }
  i.ctx = r.ctx;
  i.n = (int)n;
  i.tiles = (i.n + a.tile_nodes - 1) / a.tile_nodes;
  i.nblk = (i.ctx + 127) >> 7;
  return i;
}

// The tensor-memory lane of a tile's first row (a multiple of 32, so that warps are whole).
__device__ __forceinline__ int first_lane(int rows) { return (kRows - rows) & ~31; }

// The mask of a row over the 64 nodes from j0 on (bits of nodes below 0, history, are set).
// w: its words (nullptr: a chain, whose node `own` sees those up to itself).
__device__ __forceinline__ uint64_t sees64(const uint64_t* w, int words, int own, int n, int j0) {
  if (j0 <= -64) return ~0ull;
  if (!w) {
    const int last = own - j0;  // the last bit set
    return last < 0 ? 0ull : last >= 63 ? ~0ull : (2ull << last) - 1;
  }
  uint64_t v;
  if (j0 < 0) {
    v = (w[0] << -j0) | ((1ull << -j0) - 1);
  } else {
    const int i = j0 >> 6, sh = j0 & 63;
    const uint64_t lo = i < words ? w[i] : 0, hi = i + 1 < words ? w[i + 1] : 0;
    v = sh ? (lo >> sh) | (hi << (64 - sh)) : lo;
  }
  const int valid = n - j0;
  return valid <= 0 ? 0ull : valid >= 64 ? v : v & ((1ull << valid) - 1);
}

__device__ __forceinline__ bool sees(const TreeArgs& a, long long row, int own, int j) {
  return a.mask ? a.mask[row * a.words + (j >> 6)] >> (j & 63) & 1 : j <= own;
}

// Eight words, 32-byte aligned: a whole sector by one lane.  (A warp's lanes write rows that lie apart, and L1
// takes a cycle for each line of an instruction.)
__device__ __forceinline__ void store8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// The infinities and NaN among 16 bytes of V, taken out (true if there were any).
template <int KIND>
__device__ __forceinline__ bool take_out(uint4& x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m;
    if constexpr (KIND == K_BF16) m = __vcmpeq2(w[i] & 0x7F807F80u, 0x7F807F80u);
    else if constexpr (KIND == K_F16) m = __vcmpeq2(w[i] & 0x7C007C00u, 0x7C007C00u);
    else m = __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    any |= m;
    w[i] &= ~m;
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
  return any != 0;
}

// Adds to o (32 columns from dim d0) the infinities and NaN of V of the nodes that the row sees in the
// segment, and NaN for a seen token whose tile has no finite scale.
template <int KIND, int D>
__device__ __noinline__ void put_back(const TreeArgs& a, const Seg& sg, long long row, int own, int d0, float* o) {
  using L = Lay<KIND, D>;
  const int first = max(0, 128 * sg.b0 - sg.base);
  const int end = min(sg.n, 128 * sg.b1 - sg.base);
  auto tile_of = [&](int t) -> long long {
    const int blk = a.tables[(size_t)sg.seq * a.max_blocks + (t >> 4)];
    return blk < 0 || blk >= a.num_blocks ? -1 : (long long)blk * a.Hkv + sg.h;
  };
  auto lost = [&](long long tile) { return L::kBlk && !(fabsf(a.ksc[tile]) < INFINITY && fabsf(a.vsc[tile]) < INFINITY); };
  bool nan = false;
  if (L::kBlk)  // tiles of the history
#pragma unroll 1
    for (int t = 128 * sg.b0; t < min(sg.base, 128 * sg.b1); t += 16) {
      const long long tile = tile_of(t);
      nan = nan || (tile >= 0 && lost(tile));
    }
#pragma unroll 1
  for (int j = first; j < end; ++j) {
    if (!sees(a, row, own, j)) continue;
    const int t = sg.base + j;
    const long long tile = tile_of(t);
    if (tile < 0) continue;
    nan = nan || lost(tile);
    const uint8_t* v = a.v + ((size_t)tile * 16 + (t & 15)) * L::kRow;
#pragma unroll 1
    for (int e = 0; e < 32; ++e) {
      float x;
      if constexpr (KIND == K_BF16) x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(v)[d0 + e]);
      else if constexpr (KIND == K_F16) x = __half2float(reinterpret_cast<const __half*>(v)[d0 + e]);
      else x = (v[d0 + e] & 0x7F) == 0x7F ? NAN : 0.f;
      if (!(fabsf(x) < INFINITY)) o[e] += x;
    }
  }
  if (nan)
#pragma unroll 1
    for (int e = 0; e < 32; ++e) o[e] = NAN;
}

// Whether the phase of the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return done != 0;
}

// D (TMEM) = A x B (+ D) with A in tensor memory; lo: the low word of B's descriptor, whose high one is a
// constant of its layout.
template <bool F8>
__device__ __forceinline__ void mma_lo(uint32_t d, uint32_t a_tmem, uint32_t lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  if constexpr (F8)
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n\t}"
                 ::"r"(d), "r"(a_tmem), "r"(lo), "r"(hi), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
                 ::"r"(d), "r"(a_tmem), "r"(lo), "r"(hi), "r"(idesc), "r"(acc) : "memory");
}

// As tc::wait_or_abort, whose retries are kept out of line: inlined at every wait they make up most of the code.
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  return wait_or_abort(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(bar)), parity, abort_flag, err);
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  return mbar_try_wait(bar, parity) || wait_more(smem_addr(bar), parity, abort_flag, err);
}

template <int KIND, int D, int OUT, bool PSPLIT>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmk,
                                                           const __grid_constant__ CUtensorMap tmv) {
  using L = Lay<KIND, D>;
  constexpr bool F8 = L::kF8, BLK = L::kBlk, BF = L::kBf;
  constexpr int R = L::kRing;
  constexpr int DH = D / 2;  // a half-row thread's share of the head dim
  constexpr uint32_t kIdescQK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24) | (BF ? (1u << 7) | (1u << 10) : 0u);
  constexpr uint32_t kIdescPV =
      (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24) | (BF ? (1u << 7) | (1u << 10) : 0u);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl* ctl = reinterpret_cast<Ctrl*>(sm + L::kData);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 3) {  // a barrier of each kind per lane
    const int i = lane;
    if (i < kSegRing) {
      mbar_init(&ctl->seg_full[i], 1);
      mbar_init(&ctl->seg_empty[i], 15);  // MMA, 2 for masks, 8 softmax, 4 for V
    }
    if (i < kScaleRing) {
      mbar_init(&ctl->sc_full[i], 1);
      mbar_init(&ctl->sc_empty[i], 8);
      ctl->bad[i] = 0;
    }
    if (i < kRowRing) mbar_init(&ctl->row_free[i], 8);
    if (i < R) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);           // the Q K MMAs
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], F8 ? 4 : 1);  // FP8: the warps that convert it; 16-bit: the P V MMAs
    }
    if (i < 2) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], F8 ? 12 : 8);  // softmax; FP8: and the four warps that convert V
      mbar_init(&ctl->vt_empty[i], 1);
      mbar_init(&ctl->q_ready[i], 6);
      mbar_init(&ctl->q_free[i], 1);
      mbar_init(&ctl->tail_ready[i], 1);
      mbar_init(&ctl->tail_done[i], 4);
    }
    if (i == 0) {
      mbar_init(&ctl->o_full, 1);
      mbar_init(&ctl->o_free, 4);
      mbar_init(&ctl->drain, 1);
      ctl->abort = 0;
      ctl->start_seq = -1;
    }
    fence_barrier_init();
  }
  if (warp == 1 && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&ctl->tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();  // the kernel before may still write lengths, tables, queries and pages

  // ---------------------------------------------------------------- schedule
  // Positions: a unit of nblk blocks takes kUnitCost + nblk of them, its blocks behind; units in
  // (sequence, kv head, tile) order.  Each CTA takes T positions.
  // (For short tables, a.whole: a unit takes one position.)
  constexpr int kUnit = L::kUnitCost;
  auto span_of = [&](const SeqInfo& i) { return a.whole ? 1 : i.nblk + kUnit; };
  const int per = (a.S + kThreads - 1) / kThreads;
  const int s0 = min(a.S, (int)threadIdx.x * per), s1 = min(a.S, s0 + per);
  long long mine = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const SeqInfo i = seq_info(a, seq_raw(a, s));
    if (i.bad) record_error(a.err, PA_ERR_BOUNDS);
    mine += i.units(a.Hkv) * span_of(i);
  }
  long long before, total = 0;
  {
    long long x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(kAll, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) ctl->warp_sums[warp] = x;
    __syncthreads();
    long long ahead = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      ahead += w < warp ? ctl->warp_sums[w] : 0;
      total += ctl->warp_sums[w];
    }
    before = ahead + x - mine;
  }
  const long long T = max((total + a.ctas - 1) / a.ctas, a.whole ? 1ll : (long long)kUnit + 1);
  const long long pos0 = (long long)blockIdx.x * T, pos_end = min(total, pos0 + T);
  if (pos0 < total && before <= pos0 && pos0 < before + mine) {
    long long cum = before;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const SeqInfo i = seq_info(a, seq_raw(a, s));
      const long long c = i.units(a.Hkv) * span_of(i);
      if (pos0 < cum + c) {
        ctl->start_seq = s;
        ctl->start_off = pos0 - cum;
        break;
      }
      cum += c;
    }
  }
  if (threadIdx.x == 32) a.jobs[blockIdx.x] = make_int4(-1, 0, 0, 0);  // (the copying warp's lane 0 may set it)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // A 512-column allocation spans the whole tensor memory, so its base is 0, and taken as the constant:
  // every tensor-memory operand of the MMA warp is then an immediate.
  constexpr uint32_t tmem = 0;

  if (pos0 >= total || ctl->start_seq < 0) {
    // no work for this CTA
  } else if (ctl->tmem != 0) {
    if (threadIdx.x == 0) record_error(a.err, PA_ERR_UNSUPPORTED);
  } else if (warp == 1) {
    // ---------------------------------------------------------- schedule and TMA producer
    const uint64_t policy = l2_evict_first_policy();
    int seq = ctl->start_seq;
    SeqInfo info = seq_info(a, seq_raw(a, seq));
    SeqRaw ahead = seq_raw(a, seq + 1);
    int span = span_of(info);
    long long u = ctl->start_off / span;
    int v = (int)(ctl->start_off - u * span);
    long long pos = pos0;
    bool ok = true;
    int made = 0;  // descriptions handed out
    bool last = false;
    auto produce = [&]() {  // the next segment's description, empty behind the last one
      Seg sg = {};
      while (pos < pos_end) {
        while (u >= info.units(a.Hkv)) {
          if (++seq >= a.S) break;
          info = seq_info(a, ahead);
          ahead = seq_raw(a, seq + 1);
          span = span_of(info);
          u = 0;
          v = 0;
        }
        if (seq >= a.S) {  // (the lengths changed under the kernel)
          pos = pos_end;
          break;
        }
        const int take = (int)min((long long)(span - v), pos_end - pos);
        const int b0 = a.whole ? 0 : max(0, v - kUnit), b1 = a.whole ? info.nblk : max(0, v + take - kUnit);
        const long long ustart = pos - v;
        const int unit = (int)u, nblk = info.nblk;
        pos += take;
        v += take;
        if (v == span) {
          v = 0;
          ++u;
        }
        if (b1 > b0) {
          sg.seq = seq;
          sg.h = unit / info.tiles;
          sg.tile = unit - sg.h * info.tiles;
          sg.b0 = b0;
          sg.b1 = b1;
          sg.n = info.n;
          sg.base = info.ctx - info.n;
          sg.q0 = info.q0;
          sg.nblk = nblk;
          sg.last_cta = (int)((ustart + span - 1) / T);
          if (b0 == 0 && b1 < nblk && lane == 0)
            a.jobs[blockIdx.x] = make_int4(seq, unit, sg.last_cta, 2 * blockIdx.x + (made > 0));
          break;
        }
      }
      const int e = made % kSegRing;
      if (made >= kSegRing)
        ok = ok && __all_sync(kAll, wait_for(&ctl->seg_empty[e], ((made / kSegRing) - 1) & 1, abort_flag, a.err));
      if (ok && lane == 0) {
        ctl->seg[e] = sg;
        mbar_arrive(&ctl->seg_full[e]);
      }
      ++made;
      last = sg.b1 == sg.b0;
    };
    // Batches of up to four blocks of a segment: the table entries of a batch are loaded two
    // batches ahead (lane i: page i), its tile scales one ahead, for while the copies keep HBM
    // busy such a load takes some microseconds.
    struct Batch {
      int j, seq, h, b, nb, page_end, raw;  // j: the segment's number
    };
    float sk = 1.f, sv = 0.f;
    auto scales = [&](Batch& x) {  // checks the entries; block-scaled pools: loads their scales
      const bool live = 8 * x.b + lane < x.page_end;
      if (live && (x.raw < 0 || x.raw >= a.num_blocks)) {
        record_error(a.err, PA_ERR_BOUNDS);
        x.raw = 0;
      }
      if constexpr (BLK) {
        sk = 1.f;
        sv = 0.f;
        if (live) {
          sk = a.ksc[(size_t)x.raw * a.Hkv + x.h];
          sv = a.vsc[(size_t)x.raw * a.Hkv + x.h];
        }
      }
    };
    int g = 0, gk = 0;    // blocks issued: whole, and their K
    int fj = -1, fb = 0;  // the segment that batches are fetched from, and the next one's first block
    Seg front = {};
    bool more = true;
    Batch cur = {}, nxt = {};
#pragma unroll 1
    while (ok) {
      Batch far = {};
      if (more && fb == front.b1) {
        // A segment is described before the first copies of the one in front of it, as the queries' warps look
        // one segment ahead.
        ++fj;
#pragma unroll 1
        while (ok && !last && made < fj + 2) produce();
        if (!ok) break;
        __syncwarp();
        front = ctl->seg[fj % kSegRing];
        fb = front.b0;
        more = front.b1 > front.b0;
      }
      if (more) {
        far.j = fj;
        far.seq = front.seq;
        far.h = front.h;
        far.b = fb;
        far.nb = min(4, front.b1 - fb);
        far.page_end = min(8 * (fb + far.nb), (front.base + front.n + 15) >> 4);
        const int page = 8 * fb + lane;
        if (page < far.page_end) far.raw = a.tables[(size_t)far.seq * a.max_blocks + page];
        fb += far.nb;
      }
      // a tile without a finite scale holds NaN, for the rows that see it (put_back); here it counts for nothing
      float csk = sk, csv = sv;
      if (BLK && !(fabsf(sk) < INFINITY && fabsf(sv) < INFINITY)) {
        csk = 1.f;
        csv = 0.f;
        ctl->bad[cur.j & 7] = cur.j + 1;
      }
      float lgv = 0.f, ev = 0.f, fv = 1.f;
      if constexpr (BLK) {
        csv = csv >= kMinFactor ? csv : 0.f;  // (subnormal scales count as 0)
        ev = lgv = log2f(csv);
        if constexpr (PSPLIT) {
          ev = floorf(lgv);
          fv = csv > 0.f ? ldexpf(csv, -(int)ev) : 0.f;
        }
      }
      scales(nxt);
#pragma unroll 1
      for (int j = 0; j < cur.nb; ++j, ++g) {
        const int slot = g % R, pb = 8 * j, b = cur.b + j;
        const int cnt = min(8, cur.page_end - 8 * b);
        if constexpr (BLK) {
          const int e = g % kScaleRing;
          if (g >= kScaleRing)
            ok = __all_sync(kAll, wait_for(&ctl->sc_empty[e], ((g / kScaleRing) - 1) & 1, abort_flag, a.err));
          if (!ok) break;
          if (lane >= pb && lane < pb + 8) ctl->sc[e][lane - pb] = make_float4(csk, lgv, ev, fv);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->sc_full[e]);
        }
        const int i = lane - pb;  // this lane's page of the block
        const int row0 = (cur.raw * a.Hkv + cur.h) * 16;
        auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full, uint64_t* empty) {
          if (g >= R) ok = __all_sync(kAll, ok && wait_for(empty, ((g / R) - 1) & 1, abort_flag, a.err));
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)cnt * 16u * L::kRow);
          if (i >= 0 && i < cnt) {
#pragma unroll
            for (int hh = 0; hh < L::kHalves; ++hh)
              tma_load_2d(dst + i * 16 * L::kPart + hh * 16384, map, 128 * hh, row0, full, policy);
          }
        };
        load(&tmk, sm + slot * L::kSlot, &ctl->k_full[slot], &ctl->k_empty[slot]);
        if (ok) ++gk;
        load(&tmv, sm + (R + slot) * L::kSlot, &ctl->v_full[slot], &ctl->v_empty[slot]);
        if (!ok) break;
      }
      cur = nxt;
      nxt = far;
      if (!more && cur.nb == 0 && nxt.nb == 0) break;
    }
    // no copy may still target shared memory when the CTA exits
    if (lane == 0) {
#pragma unroll 1
      for (int j = max(0, gk - R); j < gk; ++j)
        if (!mbar_wait(&ctl->k_full[j % R], (j / R) & 1)) record_error(a.err, PA_ERR_TIMEOUT);
#pragma unroll 1
      for (int j = max(0, g - R); j < g; ++j)
        if (!mbar_wait(&ctl->v_full[j % R], (j / R) & 1)) record_error(a.err, PA_ERR_TIMEOUT);
    }
  } else if (warp == 0) {
    // ---------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t kHi128 = (1024u >> 4) | (1u << 14) | (2u << 29);  // 128-byte swizzle, 8 rows 1024 bytes apart
      constexpr uint32_t kHiK = L::kPart == 64 ? (512u >> 4) | (1u << 14) | (4u << 29) : kHi128;
      const uint32_t k_lo = ((smem_addr(sm) & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t v_lo = ((smem_addr(sm + (F8 ? L::kVT : R * L::kSlot)) & 0x3FFFFu) >> 4) | ((16384u >> 4) << 16);
      // cursors over the blocks: Q K^T, two blocks ahead of P V
      // (a block's place in the ring of three and that round's parity are counted along: a remainder by three costs
      // this thread some 50 cycles)
      int kslot = 0, kpar = 0, vslot = 0, vpar = 0;
      int gq = 0, jq = -1, bq = 0, bq1 = 0, qbase = 0, tq = 0;
      bool q_end = false;
      int gp = 0, jp = -1, bp = 0, bp0 = 0, bp1 = 0, pbase = 0, tp = 0;
      // A wait costs this thread some 150 cycles even when its phase is complete.  So the next one's barrier
      // is tested while the MMAs in between are issued.  (The phase in front of the tested one is known to be
      // complete: this thread has waited for it.)
      bool k_ready = false, p_ready = false, v_ready = false;
      auto seg_wait = [&](int j) { return wait_for(&ctl->seg_full[j % kSegRing], (j / kSegRing) & 1, abort_flag, a.err); };
      auto issue_qk = [&]() -> bool {
        if (bq == bq1) {
          if (q_end) return true;
          ++jq;
          if (!seg_wait(jq)) return false;
          const Seg& sg = ctl->seg[jq % kSegRing];
          bq = sg.b0;
          bq1 = sg.b1;
          qbase = sg.base;
          if (bq == bq1) {
            q_end = true;
            return true;
          }
          if (!wait_for(&ctl->q_ready[jq & 1], (jq >> 1) & 1, abort_flag, a.err)) return false;
        }
        const int slot = kslot, sb = gq & 1;
        if (!k_ready && !wait_for(&ctl->k_full[slot], kpar, abort_flag, a.err)) return false;
        k_ready = false;
        tc_fence_after();
        if constexpr (!F8)
          if (128 * bq + 127 >= qbase) {  // V of a block that reaches the tree is looked through first
            mbar_arrive(&ctl->tail_ready[tq & 1]);
            ++tq;
          }
        const uint32_t lo = k_lo + (uint32_t)(slot * (L::kSlot >> 4));
        const uint32_t qcol = tmem + kQCol + 64 * (jq & 1), scol = tmem + sb * 128;
        if constexpr (F8) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_lo<true>(scol, qcol + 32 * t + 8 * k, lo + 2 * k, kHiK, kIdescQK, (uint32_t)(t | k));
        } else {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_lo<false>(scol, qcol + 32 * h + 8 * k, lo + h * (16384 >> 4) + k * 2, kHiK, kIdescQK, (uint32_t)(h | k));
        }
        mma_commit(&ctl->s_full[sb]);
        mma_commit(&ctl->k_empty[slot]);
        ++gq;
        if (++kslot == R) {
          kslot = 0;
          kpar ^= 1;
        }
        if (++bq == bq1) mma_commit(&ctl->q_free[jq & 1]);  // the segment's queries are read
        return true;
      };
#pragma unroll 1
      for (int lead = 0;; ++lead) {
        if (lead >= 2) {
          if (bp == bp1) {
            ++jp;
            if (!seg_wait(jp)) break;
            const Seg& sg = ctl->seg[jp % kSegRing];
            bp = bp0 = sg.b0;
            bp1 = sg.b1;
            pbase = sg.base;
            mbar_arrive(&ctl->seg_empty[jp % kSegRing]);
            if (bp == bp1) break;
            if (jp > 0 && !wait_for(&ctl->o_free, (jp - 1) & 1, abort_flag, a.err)) break;  // O is read out
          }
          const int vb = gp & 1;
          if (!p_ready && !wait_for(&ctl->p_full[vb], (gp >> 1) & 1, abort_flag, a.err)) break;
          if constexpr (!F8) {
            if (!v_ready && !wait_for(&ctl->v_full[vslot], vpar, abort_flag, a.err)) break;
            if (128 * bp + 127 >= pbase) {
              if (!wait_for(&ctl->tail_done[tp & 1], (tp >> 1) & 1, abort_flag, a.err)) break;
              ++tp;
            }
          }
          k_ready = mbar_test(&ctl->k_full[kslot], kpar);
          tc_fence_after();
          const uint32_t lo = v_lo + (uint32_t)(F8 ? vb * (L::kVTBlock >> 4) : vslot * (L::kSlot >> 4));
          const uint32_t pcol = tmem + vb * 128, add = bp > bp0;
#pragma unroll
          for (int part = 0; part < (PSPLIT ? 2 : 1); ++part)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_lo<false>(tmem + kOCol, pcol + 32 * (k >> 1) + 16 * part + 8 * (k & 1), lo + k * (2048 >> 4), kHi128, kIdescPV,
                            part | k ? 1u : add);
          if constexpr (F8) mma_commit(&ctl->vt_empty[vb]);
          else mma_commit(&ctl->v_empty[vslot]);
          ++gp;
          if (++vslot == R) {
            vslot = 0;
            vpar ^= 1;
          }
          if (++bp == bp1) mma_commit(&ctl->o_full);
          p_ready = mbar_test(&ctl->p_full[gp & 1], (gp >> 1) & 1);
          if constexpr (!F8) v_ready = mbar_test(&ctl->v_full[vslot], vpar);
        }
        if (!issue_qk()) break;
      }
      // every MMA issued above has finished before TMEM is released
      mma_commit(&ctl->drain);
      if (!mbar_wait(&ctl->drain, 0)) record_error(a.err, PA_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------- masks
    bool ok = true;
    for (int j = 0; ok; ++j) {
      const int e = j % kSegRing, rr = j % kRowRing;
      ok = __all_sync(kAll, wait_for(&ctl->seg_full[e], (j / kSegRing) & 1, abort_flag, a.err));
      if (!ok) break;
      const Seg sg = ctl->seg[e];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->seg_empty[e]);
      if (sg.b1 == sg.b0) break;
      // segment j - 2's phase of q_ready is over, and the rows of segment j - kRowRing are done
      if (j >= 2) ok = __all_sync(kAll, wait_for(&ctl->q_free[j & 1], ((j >> 1) - 1) & 1, abort_flag, a.err));
      if (j >= kRowRing) ok = __all_sync(kAll, ok && wait_for(&ctl->row_free[rr], ((j / kRowRing) - 1) & 1, abort_flag, a.err));
      if (!ok) break;
      if (a.mask && 128 * sg.b1 > sg.base) {
        const int node0 = sg.tile * a.tile_nodes, nodes = min(a.tile_nodes, sg.n - node0);
        const uint64_t* src = a.mask + (size_t)(sg.q0 + node0) * a.words;
#pragma unroll 1
        for (int i = threadIdx.x - 64; i < nodes * a.words; i += 64) ctl->mask[rr][i / a.words][i % a.words] = src[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_ready[j & 1]);
    }
  } else if (warp >= 12) {
    // ---------------------------------------------------------- V, queries and output
    const int ct = threadIdx.x - 12 * 32;  // 0 .. 127: a key of V, a row of Q and O
    const int qr = ct;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    bool ok = true;
    // A thread's own row of queries of segment j.  FP8: the warps are busy with V, so the row is copied to shared
    // memory in the background (chunk c at place c ^ (row mod 16): no bank conflicts) and taken up
    // some blocks later.  16-bit pools: loaded where it is stored; the warps have little else to do.
    uint8_t* stage = sm + L::kQ + ct * (D * 2);
    const int turn = ct & (D / 8 - 1);
    auto query_row = [&](int j) -> const uint4* {
      const Seg& sg = ctl->seg[j % kSegRing];
      const int rows = min(a.tile_nodes, sg.n - sg.tile * a.tile_nodes) * a.G;
      const int row = qr - first_lane(rows), tl = row / a.G, hh = row - tl * a.G;
      if (row < 0 || row >= rows) return nullptr;
      return reinterpret_cast<const uint4*>(
          a.q + ((long long)(sg.q0 + sg.tile * a.tile_nodes + tl) * a.Hq + (long long)sg.h * a.G + hh) * D);
    };
    auto load_rows = [&](int j) {
      if constexpr (F8) {
        const uint4* src = query_row(j);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint8_t* to = stage + ((c ^ turn) << 4);
          if (src) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(src + c) : "memory");
          else *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
        }
      }
    };
    auto store_rows = [&](int j) {
      // segment j - 2's queries are read, and the rows of segment j - kRowRing are done
      if (j >= 2) ok = __all_sync(kAll, ok && wait_for(&ctl->q_free[j & 1], ((j >> 1) - 1) & 1, abort_flag, a.err));
      if (j >= kRowRing)
        ok = __all_sync(kAll, ok && wait_for(&ctl->row_free[j % kRowRing], ((j / kRowRing) - 1) & 1, abort_flag, a.err));
      if constexpr (F8) asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok) return;
      tc_fence_after();
      const uint32_t qcol = trow + kQCol + 64 * (j & 1);
      float row_scale = fabsf(a.qk_scale_log2);
      if constexpr (!F8) {
        const uint4* src = query_row(j);
        const uint32_t flip = a.qk_scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale flips the queries' signs
#pragma unroll 1
        for (int part = 0; part < D / 64; ++part) {
          uint32_t qw[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = src ? src[8 * part + c] : make_uint4(0, 0, 0, 0);
            qw[4 * c] = x.x ^ flip;
            qw[4 * c + 1] = x.y ^ flip;
            qw[4 * c + 2] = x.z ^ flip;
            qw[4 * c + 3] = x.w ^ flip;
          }
          tmem_st32u(qcol + 32 * part, qw);
        }
      } else {
        // scaled by a power of two (the largest |q| in [128, 256)) and split into two E4M3 terms
        uint32_t top = 0;  // the largest magnitude's bits, of either half of a word
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = lds128(stage + ((c ^ turn) << 4));
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
        }
        const float amax = bf16_bits_to_float(max(top & 0xFFFFu, top >> 16));
        int ex = 8;
        if (amax > 0.f && amax < INFINITY) frexpf(amax, &ex);
        ex = max(ex, -118);  // (2^(8 - ex) and its inverse are normal numbers; of rows below 2^-118 the last bits are lost)
        // (E4M3 has no infinity: a row that holds one, or a NaN, becomes NaN, as its scores would)
        const float qs = amax < INFINITY ? copysignf(ldexpf(1.f, 8 - ex), a.qk_scale_log2) : NAN;
        row_scale *= ldexpf(1.f, ex - 8);
#pragma unroll 1
        for (int part = 0; part < D / 32; ++part) {
          uint32_t qhi[8], qlo[8];  // 4 dims per word
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 x = lds128(stage + (((4 * part + c) ^ turn) << 4));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w0 = w[2 * h], w1 = w[2 * h + 1];
              const float2 x01 = make_float2(bf16_bits_to_float(w0 & 0xFFFFu) * qs, bf16_bits_to_float(w0 >> 16) * qs);
              const float2 x23 = make_float2(bf16_bits_to_float(w1 & 0xFFFFu) * qs, bf16_bits_to_float(w1 >> 16) * qs);
              const uint32_t h01 = __nv_cvt_float2_to_fp8x2(x01, __NV_SATFINITE, __NV_E4M3);
              const uint32_t h23 = __nv_cvt_float2_to_fp8x2(x23, __NV_SATFINITE, __NV_E4M3);
              const float2 d01 = unpack2<false>(e4m3x2_to_f16x2(h01));
              const float2 d23 = unpack2<false>(e4m3x2_to_f16x2(h23));
              const uint32_t l01 = __nv_cvt_float2_to_fp8x2(make_float2(x01.x - d01.x, x01.y - d01.y), __NV_SATFINITE, __NV_E4M3);
              const uint32_t l23 = __nv_cvt_float2_to_fp8x2(make_float2(x23.x - d23.x, x23.y - d23.y), __NV_SATFINITE, __NV_E4M3);
              qhi[2 * c + h] = (h01 & 0xFFFFu) | (h23 << 16);
              qlo[2 * c + h] = (l01 & 0xFFFFu) | (l23 << 16);
            }
          }
          tmem_st8u(qcol + 8 * part, qhi);
          tmem_st8u(qcol + 32 + 8 * part, qlo);
        }
      }
      // (a zero factor would turn a masked -inf into NaN; with scales of tiles it is bounded with the tile's)
      ctl->row_scale[j % kRowRing][qr] = BLK ? row_scale : fmaxf(row_scale, kMinFactor);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_ready[j & 1]);
    };
    // The rows of segment j: the output, or a partial state.
    auto write_rows = [&](int j) {
      const Seg& sg = ctl->seg[j % kSegRing];
      ok = __all_sync(kAll, ok && wait_for(&ctl->row_free[j % kRowRing], (j / kRowRing) & 1, abort_flag, a.err));
      ok = __all_sync(kAll, ok && wait_for(&ctl->o_full, j & 1, abort_flag, a.err));
      if (!ok) return;
      tc_fence_after();
      const int rows = min(a.tile_nodes, sg.n - sg.tile * a.tile_nodes) * a.G;
      const int r = qr - first_lane(rows), tl = r / a.G, hh = r - tl * a.G;
      if ((qr | 31) >= first_lane(rows)) {  // (whole warps)
        const bool live = r >= 0 && r < rows, whole = sg.b0 == 0 && sg.b1 == sg.nblk;
        const bool odd = *(volatile int*)&ctl->bad[j % kScaleRing] == j + 1;
        const float4 fin = ctl->fin[j % kRowRing][qr];
        const float Ls = fin.z + fin.w;
        const float inv = whole ? (Ls > 0.f ? (BLK ? fin.y : a.v_scale) / Ls : 0.f) : BLK ? fin.y : 1.f;
        const int own = sg.tile * a.tile_nodes + tl;
        const long long qrow = (long long)sg.q0 + own;
        const long long orow = (qrow * a.Hq + (long long)sg.h * a.G + hh) * D;
        const long long prow = (long long)(2 * blockIdx.x + (j > 0)) * kRows + r;
        const uint32_t oc = trow + kOCol;
        // (A loop, though O is free only behind it: straight code that reads all of O first, run once a
        // segment, is 1-2% slower over the measured batches.)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(oc + 32 * c, o);
          tmem_wait_ld();
          if (!live) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (odd) {
            float x[32];  // (a copy: o stays in registers where nothing is put back)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = o[e];
            put_back<KIND, D>(a, sg, qrow, own, 32 * c, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = x[e];
          }
          uint32_t w[32];
          if (OUT != PA_FP32 && whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2<OUT == PA_BF16>(o[2 * e], o[2 * e + 1]);
            uint16_t* to = static_cast<uint16_t*>(a.out) + orow + 32 * c;
            if (a.wide) {
              store8(to, w);
              store8(to + 16, w + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(to)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          } else {
            float* to = whole ? static_cast<float*>(a.out) + orow + 32 * c : a.ws_o + prow * D + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e]);
            if (a.wide || !whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) store8(to + e, w + e);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<uint4*>(to)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          }
        }
        if (live && !whole) a.ws_ml[prow] = make_float2(fin.x, Ls);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_free);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_free);
      }
    };
    // Segment j's first block of V, then the output of j - 1 (whose last products are done about then), and
    // between j's other blocks the queries of j + 1.  A description is given back with its output.
    int g = 0, t = 0, vs = 0, vp = 0;  // (vs, vp: the block's place in its ring, that round's parity)
    for (int j = -1; ok; ++j) {
      int b0 = 0, b1 = 0, base = 0, ctx = 0;
      if (j >= 0) {
        const Seg& sg = ctl->seg[j % kSegRing];
        b0 = sg.b0;
        b1 = sg.b1;
        base = sg.base;
        ctx = base + sg.n;
      }
      const bool end = j >= 0 && b1 == b0;
      bool rows_ahead = false;
      if (!end) {
        ok = __all_sync(kAll, wait_for(&ctl->seg_full[(j + 1) % kSegRing], ((j + 1) / kSegRing) & 1, abort_flag, a.err));
        if (!ok) break;
        rows_ahead = ctl->seg[(j + 1) % kSegRing].b1 > ctl->seg[(j + 1) % kSegRing].b0;
        if (rows_ahead) load_rows(j + 1);
      }
      for (int b = b0;; ++b) {
        if (b < b1) {
          const int slot = vs;
          const int nvalid = min(128, ctx - 128 * b);  // keys behind the context: zero
          const int nplain = base - 128 * b;           // keys from here on are nodes
          bool odd = false;                            // infinities or NaN among them
          if constexpr (F8) {
            const int half = g & 1;
            ok = __all_sync(kAll, wait_for(&ctl->v_full[slot], vp, abort_flag, a.err));
            if (ok && g >= 2) ok = __all_sync(kAll, wait_for(&ctl->vt_empty[half], ((g >> 1) - 1) & 1, abort_flag, a.err));
            if (!ok) break;
            const uint8_t* vr = sm + (R + slot) * L::kSlot;
            uint8_t* vt = sm + L::kVT + half * L::kVTBlock;
            // consecutive lanes take consecutive keys of one 16-byte chunk
#pragma unroll 4
            for (int ch = 0; ch < D / 16; ++ch) {
              const int key = ct;
              uint4 w = make_uint4(0, 0, 0, 0);
              // a row's chunks are permuted by its line's place: 128-byte lines, or 64-byte rows two to a line
              const uint32_t off = L::kPart == 64 ? key * 64 + ((ch ^ ((key >> 1) & 3)) << 4) : key * 128 + ((ch ^ (key & 7)) << 4);
              if (key < nvalid) w = lds128(vr + off);
              if (nplain < 128 && key >= nplain) odd |= take_out<KIND>(w);
              const uint32_t cw[4] = {w.x, w.y, w.z, w.w};
              uint32_t hv[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) e4m3x4_to_f16x2x2(cw[q], hv[2 * q], hv[2 * q + 1]);
              uint8_t* row = vt + (ch >> 2) * 16384 + key * 128;
              const int c0 = (ch & 3) * 2;
              *reinterpret_cast<uint4*>(row + ((c0 ^ (key & 7)) << 4)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
              *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (key & 7)) << 4)) = make_uint4(hv[4], hv[5], hv[6], hv[7]);
            }
            if (odd) ctl->bad[j % kScaleRing] = j + 1;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&ctl->p_full[half]);
              mbar_arrive(&ctl->v_empty[slot]);
            }
          } else if (nplain < 128) {
            // read in place: rows behind the context are zeroed, nodes' rows looked through
            ok = __all_sync(kAll, wait_for(&ctl->tail_ready[t & 1], (t >> 1) & 1, abort_flag, a.err));
            ok = ok && __all_sync(kAll, wait_for(&ctl->v_full[slot], vp, abort_flag, a.err));
            if (!ok) break;
            uint8_t* vr = sm + (R + slot) * L::kSlot;
            constexpr int CH = D / 8;  // 16-byte chunks per key
            const int first = max(0, nplain);
#pragma unroll 1
            for (int idx = ct; idx < (128 - first) * CH; idx += 128) {
              const int key = first + idx / CH, c = idx % CH;
              uint4* p = reinterpret_cast<uint4*>(vr + (c >> 3) * 16384 + key * 128 + (c & 7) * 16);
              if (key >= nvalid) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                uint4 w = *p;
                if (take_out<KIND>(w)) {
                  *p = w;
                  odd = true;
                }
              }
            }
            if (odd) ctl->bad[j % kScaleRing] = j + 1;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tail_done[t & 1]);
            ++t;
          }
          ++g;
          if (++vs == R) {
            vs = 0;
            vp ^= 1;
          }
        }
        // The next queries: between the blocks of a long segment (their loads take some microseconds while the copies
        // keep HBM busy), at once in a short one, whose end needs them soon.
        if (rows_ahead && b == (b1 - b0 < 4 ? b0 : b0 + 3)) store_rows(j + 1);
        if (b == b0 && j > 0) {
          write_rows(j - 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->seg_empty[(j - 1) % kSegRing]);
        }
        if (!ok || b + 1 >= b1) break;
      }
      if (end) break;
    }
    if constexpr (F8) asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that ran out)
  } else {
    // ---------------------------------------------------------- softmax rows
    // Two threads per row, as in the prefill; half hf takes keys 64 hf ..
    // 64 hf + 63 of every block and the head dim's half hf of Q and O.  The two warps of 32
    // rows exchange partials through shared memory (one phase of their barrier each).  Warps whose
    // lanes hold no row only keep the barriers in step.
    const int sw = warp - 4, hf = sw >> 2, quad = sw & 3;
    const int ln = quad * 32 + lane;  // the row's lane
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    int xk = 0;  // next exchange phase
    bool ok = true;
    // The two warps of 32 rows tell each other their halves' maxima, and whether all is well (a NaN says that it
    // is not; a maximum of NaN alone counts for nothing).  They meet at a hardware barrier, which has no
    // time limit: so both leave at a meeting that says so, and a warp that leaves for any other reason, its
    // list's end among them, comes to one more meeting, which is the other's next one.
    bool parted = false;
    auto exchange = [&](float2 mine) -> float2 {  // (.y: block-scaled pools; a NaN there counts for nothing by itself)
      using X = std::conditional_t<BLK, float2, float>;
      X* x = reinterpret_cast<X*>(ctl->xbuf[xk & 1]);
      mine.x = !ok ? NAN : mine.x == mine.x ? mine.x : -INFINITY;
      if constexpr (BLK) x[128 * hf + ln] = mine;
      else x[128 * hf + ln] = mine.x;
      __syncwarp();
      asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
      float2 other = make_float2(0.f, 0.f);
      if constexpr (BLK) other = x[128 * (hf ^ 1) + ln];
      else other.x = x[128 * (hf ^ 1) + ln];
      ok = __all_sync(kAll, ok && other.x == other.x);
      parted = !ok;
      ++xk;
      return other;
    };
    auto read_seg = [&](int j, Seg& sg) {
      const int e = j % kSegRing;
      ok = __all_sync(kAll, ok && wait_for(&ctl->seg_full[e], (j / kSegRing) & 1, abort_flag, a.err));
      sg = {};
      if (ok) sg = ctl->seg[e];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->seg_empty[e]);
    };
    int g = 0;
    for (int j = 0; ok; ++j) {
      Seg cur;
      read_seg(j, cur);
      if (!ok || cur.b1 == cur.b0) break;  // (behind the loop: the last meeting)
      const int rows = min(a.tile_nodes, cur.n - cur.tile * a.tile_nodes) * a.G;
      const int lane0 = first_lane(rows), r = max(ln - lane0, 0);
      const bool active = quad * 32 >= lane0;
      const int tl = min(r / a.G, rows / a.G - 1), own = cur.tile * a.tile_nodes + tl;  // this row's node
      const uint64_t* words = a.mask ? ctl->mask[j % kRowRing][tl] : nullptr;
      // l is relative to 2^m and O to 2^r.  Block-scaled pools: m follows the largest score, r the largest score
      // plus log2 of its tile's V scale, so O's weights are as large as 16 bits hold whatever the tiles' scales are, and
      // only seen keys move either.  One scale: r is m.
      float m = -INFINITY, l = 0.f, r_o = -INFINITY, row_scale = 1.f;
      for (int b = cur.b0; b < cur.b1; ++b, ++g) {
        const int sb = g & 1, se = g % kScaleRing;
        const bool first = b == cur.b0;
        float ov = 1.f;  // factor for this row's O
        if constexpr (BLK)
          ok = __all_sync(kAll, ok && wait_for(&ctl->sc_full[se], (g / kScaleRing) & 1, abort_flag, a.err));
        const int j0 = 128 * b + 64 * hf - cur.base;  // this thread's first key, as a node
        const bool masked = j0 + 63 >= 0;
        ok = __all_sync(kAll, ok && wait_for(&ctl->s_full[sb], (g >> 1) & 1, abort_flag, a.err));
        // (S was made from the segment's queries, so its masks and factors are there too)
        if (first) row_scale = ctl->row_scale[j % kRowRing][ln];
        const uint64_t vis = active && masked ? sees64(words, a.words, own, cur.n, j0) : ~0ull;
        const uint32_t sbase = trow + sb * 128;
        if (active) {
          float mh = -INFINITY, mo = -INFINITY;
          float sv[2][32];  // this thread's 64 scores of the block, read from TMEM once
          float pf[2][2];   // the score factor of each of the thread's four pages
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int hp = 0; hp < 2; ++hp)
              pf[cc][hp] = BLK ? fmaxf(row_scale * ctl->sc[se][2 * (2 * hf + cc) + hp].x, kMinFactor) : row_scale;
          if (ok) {
            tc_fence_after();
            tmem_ld32(sbase + 64 * hf, sv[0]);
            tmem_ld32(sbase + 64 * hf + 32, sv[1]);
            tmem_wait_ld();
            float pm[2][2];  // each page's largest raw score
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              float* v = sv[cc];
              if (masked) {
                const uint32_t w = (uint32_t)(vis >> (32 * cc));
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(w >> e & 1)) v[e] = -INFINITY;
              }
              pm[cc][0] = max16(v);
              pm[cc][1] = max16(v + 16);
            }
            if constexpr (BLK) {
              float po[2][2];
#pragma unroll
              for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                for (int hp = 0; hp < 2; ++hp) {
                  pm[cc][hp] *= pf[cc][hp];
                  po[cc][hp] = pm[cc][hp] + ctl->sc[se][2 * (2 * hf + cc) + hp].y;
                }
              mh = fmaxf(fmax3f(pm[0][0], pm[0][1], pm[1][0]), pm[1][1]);
              mo = fmaxf(fmax3f(po[0][0], po[0][1], po[1][0]), po[1][1]);
            } else {  // one positive factor: the largest product is the largest score times it
              mh = fmaxf(fmax3f(pm[0][0], pm[0][1], pm[1][0]), pm[1][1]) * row_scale;
            }
          }
          const float2 other = exchange(make_float2(mh, mo));
          const float mx = fmaxf(mh, other.x);
          if (!ok) break;
          // The first seen keys, or a maximum that grew.  (fp32 outputs with scales of tiles: whole numbers, so that the
          // exponents below are exact.)
          if (mx > m + kGrow) {
            const float to = (BLK && PSPLIT ? ceilf(mx) : mx) - kTop, alpha = fast_exp2(m - to);
            l *= alpha;
            if constexpr (!BLK) ov = alpha;
            m = to;
          }
          if constexpr (BLK) {
            const float mxo = fmaxf(mo, other.y);
            if (mxo > r_o + kGrow) {
              const float to = (PSPLIT ? ceilf(mxo) : mxo) - kTop;
              ov = fast_exp2(r_o - to);
              r_o = to;
            }
          }
          // (nothing seen yet, or nothing but values of 0: every weight is 0, or counts in l alone)
          const float mref = m == -INFINITY ? 0.f : m;
          const float dref = (BLK && r_o != -INFINITY ? r_o : 0.f) - mref;  // (block-scaled pools) O's reference, from m
          // O is rescaled once the previous block's P V is done (see the prefill for why this phase
          // of its barrier is never mistaken)
          if (ok && !first && __any_sync(kAll, ov != 1.f)) {
            const int gl = g - 1;
            ok = __all_sync(kAll, F8 ? wait_for(&ctl->vt_empty[gl & 1], (gl >> 1) & 1, abort_flag, a.err)
                                     : wait_for(&ctl->v_empty[gl % R], (gl / R) & 1, abort_flag, a.err));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < DH / 16; ++cc) {  // 16 columns at a time (the scores are live)
                uint32_t o[16];
                const uint32_t oc = trow + kOCol + DH * hf + 16 * cc;
                tmem_ld16u(oc, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ov);
                tmem_st16u(oc, o);
              }
              tmem_wait_st();
            }
          }
          // P in 16 bits over the chunk's own S columns (the low part 16 columns on)
          if (ok) {
            float rs = 0.f;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const int c = 2 * hf + cc;
              float* v = sv[cc];
#pragma unroll
              for (int hp = 0; hp < 2; ++hp) {
                // Block-scaled pools: a weight times its V scale is 2^(score + log2 scale - r); most of the scale goes
                // into the exponent, so that it costs a product per page in the place of one per weight.  l takes
                // the page's sum back to 2^(score - m) by what went into the exponent before its rounding at the
                // score's size, so that this rounding cancels where one page has the weight.  The exponent is kept
                // above what l needs (2^-64 of the largest score's weight); where that bound holds, O gets what is 0 in
                // 16 bits.
                float nmp = -mref, back = 1.f, vm = 1.f;
                if constexpr (BLK) {
                  const float4 sp = ctl->sc[se][2 * c + hp];
                  const float shift = fmaxf(sp.z - dref, -64.f);
                  nmp = shift - mref;
                  back = fast_exp2(-shift);
                  vm = sp.w;
                }
                const float2 f2 = make_float2(pf[cc][hp], pf[cc][hp]), nm = make_float2(nmp, nmp);
                const float2 vm2 = make_float2(vm, vm);
                float2 t01 = make_float2(0.f, 0.f), t23 = t01;
                float* x = v + 16 * hp;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float2 za = __ffma2_rn(make_float2(x[e], x[e + 1]), f2, nm);
                  const float2 zb = __ffma2_rn(make_float2(x[e + 2], x[e + 3]), f2, nm);
                  float2 pa = make_float2(fast_exp2(za.x), fast_exp2(za.y));
                  float2 pb = make_float2(fast_exp2(zb.x), fast_exp2(zb.y));
                  t01 = __fadd2_rn(t01, pa);
                  t23 = __fadd2_rn(t23, pb);
                  if constexpr (BLK && PSPLIT) {
                    pa = __fmul2_rn(pa, vm2);
                    pb = __fmul2_rn(pb, vm2);
                  }
                  x[e] = pa.x;
                  x[e + 1] = pa.y;
                  x[e + 2] = pb.x;
                  x[e + 3] = pb.y;
                }
                rs += ((t01.x + t01.y) + (t23.x + t23.y)) * back;
              }
              uint32_t ph[16], pl[16];  // in V's type: bfloat16 for bfloat16 pools, else binary16
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                ph[e] = pack2<BF>(v[2 * e], v[2 * e + 1]);
                if constexpr (PSPLIT) {
                  const float2 hv = unpack2<BF>(ph[e]);
                  pl[e] = pack2<BF>(v[2 * e] - hv.x, v[2 * e + 1] - hv.y);
                }
              }
              tmem_st16u(sbase + 32 * c, ph);
              if constexpr (PSPLIT) tmem_st16u(sbase + 32 * c + 16, pl);
            }
            l += rs;
            tmem_wait_st();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (BLK) mbar_arrive(&ctl->sc_empty[se]);
          mbar_arrive(&ctl->p_full[sb]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // what the output takes besides O
      if (hf == 0) {
        const float y = !BLK ? 1.f : r_o == -INFINITY ? 0.f : fast_exp2(r_o - m);
        ctl->fin[j % kRowRing][ln].x = m, ctl->fin[j % kRowRing][ln].y = y, ctl->fin[j % kRowRing][ln].z = l;
      }
      else ctl->fin[j % kRowRing][ln].w = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->row_free[j % kRowRing]);
    }
    if (!parted) exchange(make_float2(0.f, 0.f));
  }

  tc_fence_before();
  __syncthreads();
  grid_dependents_launch();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(ctl->tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the pieces of units that several CTAs shared: out = sum_i 2^(m_i - M) O_i / sum_i
// 2^(m_i - M) l_i.  Piece i > 0 of CTA c's unit is the first segment of CTA c + i.  A warp
// per row: a lane per piece for the weights, then the pieces' rows, whose loads do not
// wait for each other (one sequence of 131072 tokens, one kv head, 152 pieces: 50 us with both
// kernels; a running maximum from piece to piece 179).
template <int D, int OUT>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a) {
  grid_dependency_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 job = a.jobs[c0];
  if (job.x < 0) return;
  const SeqInfo info = seq_info(a, seq_raw(a, job.x));
  if (info.tiles == 0) return;
  const int h = job.y / info.tiles, tile = job.y - h * info.tiles;
  const int rows = min(a.tile_nodes, info.n - tile * a.tile_nodes) * a.G;
  const int pieces = job.z - c0 + 1;
  constexpr int LPR = D / 4, PPW = 32 / LPR;  // lanes of a row; pieces that a warp reads at once
  const int sub = lane / LPR, d4 = lane % LPR;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 4) {
    auto prow = [&](int i) { return (size_t)(i == 0 ? job.w : 2 * (c0 + i)) * kRows + r; };
    float2 ml = make_float2(-INFINITY, 0.f);  // of the piece whose number is the lane's
    if (lane < pieces) ml = a.ws_ml[prow(lane)];
    float M = ml.x;
    for (int i = lane + 32; i < pieces; i += 32) M = fmaxf(M, a.ws_ml[prow(i)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, off));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float Ls = 0.f;
    for (int base = 0; base < pieces; base += 32) {
      float w = 0.f;
      if (base + lane < pieces) {
        if (base > 0) ml = a.ws_ml[prow(base + lane)];
        // a piece without any seen key holds zeros, or the NaN of a score
        w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : fast_exp2(ml.x - M);
        if (w != 0.f) Ls += w * ml.y;
      }
      const int cnt = min(32, pieces - base);
#pragma unroll 8
      for (int i = 0; i < cnt; i += PPW) {
        const float wi = __shfl_sync(kAll, w, (i + sub) & 31);
        const float4 x = reinterpret_cast<const float4*>(a.ws_o)[prow(base + min(i + sub, cnt - 1)) * (D / 4) + d4];
        if (i + sub < cnt) {
          // a piece whose weight is below fp32's range leaves its infinities and NaN (one without seen keys has none)
          auto part = [&](float v) { return wi != 0.f ? wi * v : fabsf(v) < INFINITY ? 0.f : v; };
          o.x += part(x.x);
          o.y += part(x.y);
          o.z += part(x.z);
          o.w += part(x.w);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) Ls += __shfl_xor_sync(kAll, Ls, off);
    if constexpr (PPW == 2) {
      o.x += __shfl_xor_sync(kAll, o.x, 16);
      o.y += __shfl_xor_sync(kAll, o.y, 16);
      o.z += __shfl_xor_sync(kAll, o.z, 16);
      o.w += __shfl_xor_sync(kAll, o.w, 16);
      if (sub) continue;
    }
    const float f = Ls > 0.f ? a.v_scale / Ls : Ls == 0.f ? 0.f : NAN;
    const int node = r / a.G, hh = r - node * a.G;
    const size_t at = ((size_t)(info.q0 + tile * a.tile_nodes + node) * a.Hq + (size_t)h * a.G + hh) * D + 4 * d4;
    if constexpr (OUT == PA_FP32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    } else {
      constexpr bool BF = OUT == PA_BF16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(pack2<BF>(o.x * f, o.y * f), pack2<BF>(o.z * f, o.w * f));
    }
  }
}

// ---------------------------------------------------------------- host side
struct Build {
  const void* fn;
  int smem;
  cudaError_t (*launch)(const TreeArgs&, const CUtensorMap*, const CUtensorMap*, cudaStream_t);
  bool* configured;  // per device
};

template <int KIND, int D, int OUT, bool PSPLIT>
struct Launch {
  static cudaError_t go(const TreeArgs& a, const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<KIND, D>();
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_kernel<KIND, D, OUT, PSPLIT>, a, *tk, *tv);
    if (e != cudaSuccess || a.whole) return e;
    // Units of eight pieces and more have a warp per row; otherwise a warp takes two, as the CTAs that find
    // no unit cost more (one sequence of 131072 tokens and one kv head 50 us, 73 with 16; 64 x 2048 74.5, 75.4 with 32).
    cfg.gridDim = dim3(a.ctas, 8ll * a.S * a.Hkv <= a.ctas ? kRows / 4 : kRows / 8);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, OUT>, a);
  }
  static Build get() {
    static bool configured[128];
    return {reinterpret_cast<const void*>(&tree_kernel<KIND, D, OUT, PSPLIT>), smem_bytes<KIND, D>(), &go, configured};
  }
};

template <int D>
Build pick(int kv_dtype, bool f32) {
  switch (kv_dtype) {
    case PA_FP8_E4M3:
      return f32 ? Launch<K_E4M3, D, PA_FP32, true>::get() : Launch<K_E4M3, D, PA_BF16, false>::get();
    case PA_FP8_E4M3_BLOCK:
      return f32 ? Launch<K_E4M3B, D, PA_FP32, true>::get() : Launch<K_E4M3B, D, PA_BF16, false>::get();
    case PA_BF16:  // 16-bit pools: P's low part too, or the weights would lose what the output can hold
      return f32 ? Launch<K_BF16, D, PA_FP32, true>::get() : Launch<K_BF16, D, PA_BF16, true>::get();
    default:
      return f32 ? Launch<K_F16, D, PA_FP32, true>::get() : Launch<K_F16, D, PA_FP16, true>::get();
  }
}

// Maps of a layer's K and V regions in rows of 64 bytes, 64-byte swizzled: 128 of them
// are the K-major operand layout of that width.
int layer_row64_maps(pa_pool* pool, int layer, const CUtensorMap** tk, const CUtensorMap** tv) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const pa_pool_desc& d = pool->desc;
  if (pool->tmaps_half.size() != 2u * d.n_layers) {
    pool->tmaps_half.assign(2u * d.n_layers, pa_tmap_blob{});
    pool->tmap_half_ready.assign(d.n_layers, 0);
  }
  CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(pool->tmaps_half.data()) + 2 * layer;
  if (!pool->tmap_half_ready[layer]) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {64, (cuuint64_t)d.num_blocks * d.n_kv_heads * d.block_size}, strides[1] = {64};
    const cuuint32_t box[2] = {64, 16}, es[2] = {1, 1};
    for (int which = 0; which < 2; ++which) {
      uint8_t* base = (which ? pool->v : pool->k) + (size_t)layer * pool->layer_bytes;
      const CUresult r = reinterpret_cast<Encode>(p)(
          &maps[which], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    }
    pool->tmap_half_ready[layer] = 1;
  }
  *tk = &maps[0];
  *tv = &maps[1];
  return PA_OK;
}

int sm_count(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e != cudaSuccess || *dev < 0 || *dev >= 128) return fail(PA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  return PA_OK;
}

int configure(const Build& b, int dev) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (!b.configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(b.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, b.smem);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "decode_tree configuration: %s", cudaGetErrorString(e));
    b.configured[dev] = true;
  }
  return PA_OK;
}

// Bytes of the workspace's parts: partial O, (m, l), jobs.
struct Workspace {
  size_t ml, jobs, total;
};

Workspace layout(int ctas, int D) {
  Workspace w;
  w.ml = 2 * (size_t)ctas * kRows * D * 4;
  w.jobs = w.ml + 2 * (size_t)ctas * kRows * 8;
  w.total = w.jobs + (size_t)ctas * 16 + 16;  // (room to start on 32 bytes)
  return w;
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

int tree_set_wait_limit(unsigned long long ns) { return (int)set_pipe_wait_limit_here(ns); }

}  // namespace pa

using namespace pa;

extern "C" {

int pa_decode_tree_workspace_bytes(const pa_pool* pool, int n_q_heads, int max_nodes, size_t* bytes) {
  int st = check_tree(pool, n_q_heads, max_nodes);
  if (st) return st;
  if (!bytes) return fail(PA_ERR_INVALID, "null output");
  int dev = 0, sms = 0;
  if ((st = sm_count(&dev, &sms))) return st;
  *bytes = layout(sms, pool->desc.head_dim).total;
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
  const size_t elems = (size_t)T * n_q_heads * pool->desc.head_dim;
  if (overlap(out, elems * (out_dtype == PA_FP32 ? 4 : 2), q, elems * 2))
    return fail(PA_ERR_INVALID, "out must not overlap q");
  if ((uintptr_t)tree_mask_dev & 7u) return fail(PA_ERR_INVALID, "tree_mask must be 8-byte aligned");
  if (!workspace || ((uintptr_t)workspace & 15u))
    return fail(PA_ERR_INVALID, "a 16-byte aligned workspace is needed");
  const pa_pool_desc& d = pool->desc;
  const int D = d.head_dim;
  int dev = 0, sms = 0;
  if ((st = sm_count(&dev, &sms))) return st;
  const Workspace ws = layout(sms, D);
  if (workspace_bytes < ws.total)
    return fail(PA_ERR_INVALID, "workspace of %zu bytes needed, %zu given", ws.total, workspace_bytes);
  const Build b = D == 64 ? pick<64>(d.kv_dtype, out_dtype == PA_FP32) : pick<128>(d.kv_dtype, out_dtype == PA_FP32);
  if ((st = configure(b, dev))) return st;
  unsigned int* err = device_error_word();
  if (!err) return PA_ERR_CUDA;
  const CUtensorMap *tk = nullptr, *tv = nullptr;
  try {
    const int row = D * pool->elem_bytes;
    st = row == 128   ? layer_maps(pool, layer, &tk, &tv)
         : row == 256 ? layer_half_maps(pool, layer, &tk, &tv)
                      : layer_row64_maps(pool, layer, &tk, &tv);
  } catch (...) {  // (the pool's first use of a layer allocates its map on the host)
    return fail(PA_ERR_NO_MEMORY, "host allocation failed");
  }
  if (st) return st;
  TreeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.out = out;
  a.mask = tree_mask_dev;
  a.v = pool->v + (size_t)layer * pool->layer_bytes;
  a.ksc = pool->block_scaled ? layer_scales(pool, pool->k, layer) : nullptr;
  a.vsc = pool->block_scaled ? layer_scales(pool, pool->v, layer) : nullptr;
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)workspace + 31) & ~(uintptr_t)31);
  a.ws_o = reinterpret_cast<float*>(base);
  a.ws_ml = reinterpret_cast<float2*>(base + ws.ml);
  a.jobs = reinterpret_cast<int4*>(base + ws.jobs);
  a.T = T;
  a.Hq = n_q_heads;
  a.Hkv = d.n_kv_heads;
  a.G = n_q_heads / d.n_kv_heads;
  a.tile_nodes = kRows / a.G;
  a.max_nodes = max_nodes;
  a.words = (max_nodes + 63) / 64;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = d.num_blocks;
  a.ctas = sms;
  const bool f8 = d.kv_dtype == PA_FP8_E4M3;
  a.qk_scale_log2 = softmax_scale * 1.4426950408889634f * (f8 ? d.k_scale : 1.f);
  a.v_scale = f8 ? d.v_scale : 1.f;
  a.wide = ((uintptr_t)out & 31u) == 0;
  a.whole = max_blocks_per_seq <= kWholePages;
  a.err = err;
  // one schedule holds at most kBalancedMaxSeqs sequences: larger batches in turn
  for (int s = 0; s < S; s += kBalancedMaxSeqs) {
    a.S = std::min(S - s, kBalancedMaxSeqs);
    a.q_start = q_start_dev + s;
    a.tables = block_tables_dev + (size_t)s * max_blocks_per_seq;
    a.ctx = ctx_lens_dev + s;
    const cudaError_t e = b.launch(a, tk, tv, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "decode_tree launch: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

}  // extern "C"
