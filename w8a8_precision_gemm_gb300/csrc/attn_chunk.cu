// attn_chunk.cu -- causal attention of several new tokens per sequence over the
// paged FP8 key/value cache: prompts, chunks of prompts behind cached tokens, draft
// tokens, and single tokens beside them.
//
//   s_ij = scale * ks_j * sum_d q_id k_jd,   p_i = softmax(s_i),   o_i = sum_j p_ij vs_j v_jd
//
// over the cached tokens j at or before query i's own position (its last `window`
// ones, or all).
//
// Bound by the tensor cores for long chunks, 4 head_dim operations per visible pair of
// a query head and a token, and by HBM for a few tokens behind a long cache.
//   * Scores: kind::f8f6f4 on the cache's own codes, so keys go into shared memory as they are. A query
//     row, scaled by a power of two so that its largest value is in [2^7, 2^8), is split in two: e4m3, and what is left as
//     e5m2.  A bf16 value has 8 significant bits: 4 and a rest of 4 units of the last place, which 3 bits hold, so values
//     down to 2^-13 of the largest are exact; smaller ones are off by at most 2^-21 of it.
//     Products are exact, sums fp32, the keys' scales are applied to them in fp32.
//   * Outputs: kind::f16, an e4m3 code being an fp16 number.  The weights w_ij = exp2(x_ij - R_i) vs_j (x: scores in
//     log2 units) are rounded to fp16, half a step: 2^-11 of a value of 2^-14 or more, 2^-25 below.  The reference
//     R_i, a whole number, puts the largest weight of the first tokens it is taken from between 2^2.1 and 2^3.2, and moves when
//     one grows past 2^15 (in blocks that are masked, past 2^11.1): what is lost of a row is below 2^-27 of its largest weight
//     for every token.  What was summed before is then scaled by a power of two, exactly, and so are the weights of the same tile that
//     are rounded already.  So the softmax need not look for a maximum: one pass, and the largest
//     weight, which every block yields, says whether it may stand.
//
// Rows of the MMAs are (token, query head of the group) pairs in a row, so a group of any
// size fills them: 256 rows in two tiles of 128 (one for head_dim above 128) against tiles of 128
// (64) tokens.  16 warps:
//   * four gather a tile's codes through the block table with cp.async, the keys into their swizzled place, the values
//     into each thread's own bytes, from which they are widened to fp16 and stored swizzled (read transposed);
//   * two issue the MMAs, one for each row tile, in turns: the scores of a tile, which are its weights' place in TMEM,
//     behind the outputs of the tile before.  (MMAs of both in one another's midst end together, both softmaxes then
//     run side by side and the tensor core waits for both: 1630 us for 1586.)  A unit of one row tile takes the two score
//     buffers in turn instead;
//   * four per row tile do the softmax, a row a thread, 64 tokens at a time, beside the other tile's MMAs; the next unit's
//     queries are copied and turned, and its scores computed, while the outputs are stored;
//   * one hands out the segments.
// The outputs stay in TMEM and are rescaled when a reference moves.
//
// A unit of work is (row tiles of a sequence, KV head).  The token tiles of all units in a
// row, each unit with a fixed amount for its start and end, are cut into equal
// ranges, one per CTA, whatever the lengths (units of few tiles stay whole); a unit that lies in several ranges leaves
// partial sums in the workspace, and the CTA that is done with it last joins
// them in order: one launch, the same result every run.  The tiles of a segment are taken from its end, so that the
// masked tile and the one that sets the reference are the same.
//
// Measured (GB300, 40 query and 8 KV heads of 128): 2048 tokens behind 30720, 1335 us, 1000 TFLOP/s (dense, as the formula
// counts), 53% of a cuBLAS bf16 GEMM: a tile of 256 rows takes 5000 cycles.  The softmax of a row
// tile takes 2700 of them and its MMAs, two fp8 passes and one in fp16, 1500 (1024 if nothing held them up), in turn with the
// other's.  Tensor pipe 34% busy, issue slots 45%, shared memory two thirds (operands, the codes on their way, the scales
// that every row reads).  Eight prompts of 1000 tokens: 234 us.  64 sequences
// of 4 tokens behind 8192 or fewer: 232 us, 2.5 TB/s: a tile of tokens is 3200 cycles of one row tile's chain from scores to
// weights to outputs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"

namespace qurl {
namespace {

constexpr int kSoftmax = 256;     // threads 0..255: two groups of 128, a row a thread
constexpr int kConverters = 128;  // threads 256..383
constexpr int kThreads = 512;     // and two warps that issue the MMAs, one that hands out the segments, one without work
// Registers a thread: 128 at launch (512 threads), moved between the warpgroups: the softmax threads' loop over 64
// scores at a time needs room to overlap its loads, products and exponentials.
constexpr int kRegsSoftmax = 168, kRegsConvert = 88, kRegsMma = 88;
static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsMma <= 4 * 128, "registers at launch");
constexpr int kRing = 8;          // tiles whose scales are kept
constexpr int kSegments = 4;      // segments handed out ahead
// Costs: a tile of one row tile 2, of two 3 (3200 and 5000 cycles: the tensor core has more to do, the loads are the same), a
// unit beside its tiles 12 (eight prompts of 1000 tokens 236 us, at 14 242),
// the least that a range gets 8 (with more, up to 48, calls of few units take longer: 4 tokens behind 4096 27 us, 57 at 48).
// Units of kWhole tiles or fewer are not cut: to start, store and join a part costs more (one prompt of 300 tokens 25 us,
// cut 35; of 1000 tokens 49, cut 62; eight of them 236, cut 249; at 10 a batch with a window of 1000 takes 89 us, at 8 76).
constexpr int kUnitCost = 12;
constexpr int kMinRange = 8;
constexpr int kWhole = 8;
constexpr float kWide = 0x1p24f;  // scores from here on are not told apart from their neighbours
constexpr float kFar = 100.0f;    // a reference lies no further than this below the largest score
constexpr float kHeavy = 0x1p15f; // weights above this move the reference, and so do exponentials whose sum is above
constexpr float kMuch = 0x1p110f;

// PANELS: 64-column panels of a head's values as fp16.
template <int PANELS_>
struct ChunkCfg {
  static constexpr int PANELS = PANELS_;
  static constexpr int CODE_PANELS = (PANELS + 1) / 2; // 128-column panels of a head in 8 bits
  static constexpr int TILES = PANELS <= 2 ? 2 : 1;    // row tiles
  static constexpr int ROWS = 128 * TILES;
  static constexpr int BN = PANELS <= 2 ? 128 : 64;    // tokens per tile
  static constexpr int K_STAGES = 3, V_STAGES = 2, RAW_STAGES = 2;
  static constexpr int Q_PIECE = CODE_PANELS * 128 * 128;  // a row tile of queries, one of the two pieces
  static constexpr int K_BYTES = CODE_PANELS * BN * 128;   // a tile of keys
  static constexpr int V_BYTES = PANELS * BN * 128;        // a tile of values as fp16
  static constexpr int Q_LANES = PANELS == 1 ? 8 : PANELS == 2 ? 16 : 32;  // lanes that copy a row of queries, 16 bytes each
  static constexpr int LANES = PANELS == 1 ? 4 : PANELS == 2 ? 8 : 16;  // lanes per token row in the gather
  static constexpr int WARP_ROWS = BN / 4;             // token rows of a tile per converter warp
  static constexpr int LOADS = WARP_ROWS * LANES / 32; // 16-byte pieces per lane, keys and values each
  static constexpr int RAW_BYTES = LOADS * kConverters * 16;  // a tile of value codes as they come
  static constexpr int OFF_K = TILES * 2 * Q_PIECE;
  static constexpr int OFF_V = OFF_K + K_STAGES * K_BYTES;
  static constexpr int OFF_RAW = OFF_V + V_STAGES * V_BYTES;
  static constexpr int SMEM = OFF_RAW + RAW_STAGES * RAW_BYTES + 1024;
  static constexpr int TM_S = BN;                      // columns between the two score buffers
  static constexpr int TM_O = 256;                     // first column of the outputs (64 PANELS per row tile)
  static_assert(2 * TM_S <= TM_O && TM_O + TILES * 64 * PANELS <= 512, "TMEM columns");
  static_assert(SMEM <= 212 * 1024, "shared memory");
};

struct ChunkPlan {
  float* partial;     // [2 grid][head_dim / 4][ROWS][4], then [2 grid][ROWS][2] of (reference, sum)
  float* partial_ml;
  unsigned* counter;  // [grid]
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));  // (subnormal scales too)
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One arrival on `bar` once this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// 2^n, n in [-126, 127], and floor(log2 x) of a normal x > 0 (-127 for zero and subnormals).
__device__ __forceinline__ float pow2(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }

// A wait that ends as soon as the phase does: without a hint of how long it may take the thread is suspended by the
// barrier itself, with one it sleeps in between.
__device__ __forceinline__ bool try_wait_now(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait (ptx.cuh) that gives up for a timeout only: a page out of range latched by
// this kernel leaves the other sequences' results alone.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* status) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait_now(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(status) == kDevTimeout) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* status) {
  if (try_wait_now(bar, parity)) return true;
  return wait_long(bar, parity, status);
}
// The same for MMAs that this thread has issued itself, whatever the status says:
// none may still be writing TMEM when it is released.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, int* status) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(status, kDevTimeout);
      return;
    }
  }
}

// MMAs issued by the lane of a warp that `lead` marks, from values that are the same in all of it: what forms them then stays in
// uniform registers.  (In a branch that one lane takes they are moved there for each MMA, 125 cycles of an MMA's 64.)
__device__ __forceinline__ void umma_scores(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc,
                                            uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// A (128 x 16 fp16) in TMEM.
__device__ __forceinline__ void umma_outputs(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t hi, uint32_t idesc,
                                             uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// Matrix descriptor of a value tile: its rows (tokens) are the MMA's K, its columns (dimensions) the
// MMA's N, 64 of them (128 bytes) in a swizzle row.  Groups of 8 rows lie 1024 bytes apart (the stride
// along K), the panels of 64 columns `panel` bytes (the stride along N).
__device__ __forceinline__ uint64_t desc_transposed(uint32_t saddr, uint32_t panel) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(panel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// A sequence: its rows of q, the tokens it has and those of them that are new.
struct Seq {
  int row0, fresh, len;
};
__device__ __forceinline__ Seq seq_of(const AttnChunkArgs& a, int b, bool* bad = nullptr) {
  const int c0 = __ldg(a.cu_new + b), c1 = __ldg(a.cu_new + b + 1), n = __ldg(a.seq_lens + b);
  const int room = a.max_blocks * a.block_size;
  const int r0 = min(max(c0, 0), a.M), r1 = min(max(c1, r0), a.M);
  if (bad && (c0 != r0 || c1 != r1 || n > room)) *bad = true;
  return {r0, r1 - r0, min(max(n, 0), room)};
}

// A unit's rows [row, row + rows) of (token, head) pairs, and the tiles of tokens they see.
struct Unit {
  int row, rows, tile0, tiles;
  int low;     // the first token that a row sees
  int weight;  // the cost of a tile
  __device__ int cost() const { return tiles == 0 ? 0 : kUnitCost + tiles * weight; }
};

template <class C>
__device__ __forceinline__ int units_of(const AttnChunkArgs& a, const Seq& s, int group) {
  return static_cast<int>((static_cast<long long>(s.fresh) * group + C::ROWS - 1) / C::ROWS);
}
template <class C>
__device__ __forceinline__ Unit unit_of(const AttnChunkArgs& a, const Seq& s, int group, int u) {
  Unit w;
  w.row = u * C::ROWS;
  w.rows = min(C::ROWS, s.fresh * group - w.row);
  const int first = s.len - s.fresh + w.row / group, last = s.len - s.fresh + (w.row + w.rows - 1) / group;
  // (first is below zero for rows that stand before the first token, and a window may be as large as an int)
  const int lo = a.window > 0 && first >= a.window ? first - a.window + 1 : 0;
  w.low = lo;
  w.tile0 = lo / C::BN;
  w.tiles = last < 0 ? 0 : last / C::BN + 1 - w.tile0;
  w.weight = w.rows > 128 ? 3 : 2;
  return w;
}

// One unit's tiles inside this CTA's range, as the roles take it from shared memory.
struct Segment {
  int n;       // tiles (0: no more segments)
  int b;       // sequence
  int head;    // KV head
  int qrow;    // row of q of the sequence's first new token, and
  int pos;     // its position
  int row;     // the unit's first (token, head) pair of the sequence, and
  int rows;    // how many
  int first;   // first token of the first tile, and
  int low;     // the first that a row of the unit sees
  int stop;    // tokens that the unit's last row sees
  int part;    // the whole unit: -1; else the place of these partial sums,
  int r0, r1;  // the first and last range with tiles of the unit
};

struct Shared {
  uint64_t kfull[3], kempty[3], vfull[2], vempty[2];  // a stage of keys, of values
  uint64_t scfull[kRing];                             // the scales of a tile
  uint64_t sgfull[kSegments], sgempty[kSegments];     // a segment
  uint64_t qfull;                                     // a segment's queries, and the scores of the one before have been used
  uint64_t sfull[2], pfull[2], ofull[2];              // scores, weights (per score buffer), outputs (per row tile)
  uint64_t turn[2];                                   // a row tile's MMAs of a step are issued
  uint64_t meet;                                      // the softmax threads
  uint64_t drain[2];
  uint32_t tmem;
  int ranges;                 // ranges in use
  long long total;            // the cost of all units
  long long before[kThreads + 1];  // cost before each thread's sequences
  // where this CTA's range begins
  int b, u, head;
  long long at;               // cost before that unit
  Segment segment[kSegments];
  alignas(16) float ks[kRing][128];
  alignas(16) float vs[kRing][128];
  uint32_t valid[kRing][4];   // tokens whose page exists
  int last;
  int nan;                    // a value code that is no number has been met
};

// The cost of a sequence's units for one KV head; sequences of many units are summed by
// the whole warp.  Every lane of the warp calls this, with its own sequence (fresh = 0: none).
template <class C>
__device__ __forceinline__ long long cost_of(const AttnChunkArgs& a, const Seq& s, int group) {
  const int n = units_of<C>(a, s, group);
  long long sum = 0;
  if (n <= 8)
    for (int u = 0; u < n; ++u) sum += unit_of<C>(a, s, group, u).cost();
  uint32_t big = __ballot_sync(0xFFFFFFFFu, n > 8);
  while (big != 0) {
    const int l = __ffs(big) - 1;
    big &= big - 1;
    const Seq t = {__shfl_sync(0xFFFFFFFFu, s.row0, l), __shfl_sync(0xFFFFFFFFu, s.fresh, l), __shfl_sync(0xFFFFFFFFu, s.len, l)};
    const int m = units_of<C>(a, t, group), lane = threadIdx.x & 31;
    long long part = 0;
    for (int u = lane; u < m; u += 32) part += unit_of<C>(a, t, group, u).cost();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
    if (lane == l) sum = part;
  }
  return sum;
}

// Walks the segments of this CTA's range in order.
template <class C>
struct Walk {
  const AttnChunkArgs& a;
  const Shared& sh;
  int group, b, u, head;
  long long at, end;
  Seq s;
  Unit w;
  int t0, t1;  // the unit's tiles in this segment

  __device__ static long long range_start(const Shared& sh, int r) { return sh.total * r / sh.ranges; }

  __device__ Walk(const AttnChunkArgs& a_, const Shared& sh_) : a(a_), sh(sh_) {
    group = a.q_heads / a.kv_heads;
    b = sh.b, u = sh.u, head = sh.head - 1, at = sh.at;
    t0 = t1 = 0;
    w = {};
    s = {0, 0, 0};
    end = static_cast<int>(blockIdx.x) < sh.ranges ? range_start(sh, blockIdx.x + 1) : -1;
    if (end < 0) at = 0;
    else {
      s = seq_of(a, b);
      w = unit_of<C>(a, s, group, u);
      at -= w.cost();
    }
  }
  // The tiles of this unit before a border at cost x (tile t costs [at + kUnitCost + t weight, + weight)); a unit of
  // few tiles stays whole, in the range that has more of it.
  __device__ int cut(long long x) const {
    const long long cost = x - at - kUnitCost;
    if (cost <= 0) return 0;
    const long long t = w.weight == 2 ? (cost + 1) / 2 : (cost + 2) / 3;
    if (t >= w.tiles) return w.tiles;
    return w.tiles > kWhole ? static_cast<int>(t) : 2 * t <= w.tiles ? 0 : w.tiles;
  }
  __device__ bool next() {
    const long long start = end < 0 ? 0 : range_start(sh, blockIdx.x);
    while (true) {
      at += w.cost();
      if (at >= end) return false;
      if (++head == a.kv_heads) {
        head = 0;
        do {  // the next unit that sees any token
          if (++u >= units_of<C>(a, s, group)) {
            u = 0;
            do {
              s = seq_of(a, ++b);
            } while (s.fresh == 0);
          }
          w = unit_of<C>(a, s, group, u);
        } while (w.tiles == 0);
      }
      t0 = cut(start);
      t1 = cut(end);
      if (t1 > t0) return true;
    }
  }
  // the first and the last range that hold tiles of this unit
  __device__ int first_range() const {
    int r = static_cast<int>(((at + kUnitCost + 1) * sh.ranges - 1) / sh.total);  // (of its first tile's border)
    while (cut(range_start(sh, r + 1)) == 0) ++r;
    return r;
  }
  __device__ int last_range() const {
    int r = static_cast<int>(((at + w.cost()) * sh.ranges - 1) / sh.total);
    while (cut(range_start(sh, r)) == w.tiles) --r;
    return r;
  }
};

// 16 codes -> 32 bytes of fp16.
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=&r"(lo), "=&r"(hi)
      : "r"(c));
}
__device__ __forceinline__ void widen16(const uint4 c, uint4& lo, uint4& hi) {
  widen4(c.x, lo.x, lo.y);
  widen4(c.y, lo.z, lo.w);
  widen4(c.z, hi.x, hi.y);
  widen4(c.w, hi.z, hi.w);
}

// NaN in a half of `acc` once one of the values is; no finite values make one: a product is exact (below 2^18) within
// the operation, and the sum never below zero.
__device__ __forceinline__ void note_nan(const uint4 v, uint32_t& acc) {
  asm("fma.rn.relu.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(v.x), "r"(v.y));
  asm("fma.rn.relu.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(v.z), "r"(v.w));
}
__device__ __forceinline__ bool has_nan(uint32_t f16x2) { return (((f16x2 & 0x7FFF7FFFu) + 0x03FF03FFu) & 0x80008000u) != 0; }
// The codes that are no number (magnitude 0x7F): the top bit of their bytes, and the codes with 0 in their place.
__device__ __forceinline__ uint32_t no_numbers(uint32_t c) { return ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool no_numbers(const uint4 c) {
  return (no_numbers(c.x) | no_numbers(c.y) | no_numbers(c.z) | no_numbers(c.w)) != 0;
}
__device__ __forceinline__ uint32_t numbers_only(uint32_t c) { return c & ~((no_numbers(c) >> 7) * 0xFFu); }

__device__ __forceinline__ void st_shared(uint32_t at, const uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Of 32 tokens from column `at` of a tile on, those a row sees (columns [lo, hi)) that are valid (`valid`: a bit for each).
__device__ __forceinline__ uint32_t seen32(int lo, int hi, int at, uint32_t valid) {
  const int l = min(max(lo - at, 0), 32), h = min(max(hi - at, 0), 32);
  const uint32_t below_l = l == 32 ? 0xFFFFFFFFu : (1u << l) - 1, below_h = h == 32 ? 0xFFFFFFFFu : (1u << h) - 1;
  return below_h & ~below_l & valid;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}
// 32 columns of this thread's TMEM lane, on their way until tmem_wait_ld; `landed` keeps what uses them behind it.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void landed(float* r) {
  asm volatile(""
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
          "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
          "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
          "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_row32(uint32_t taddr, float (&r)[32]) {
  tmem_ld32_start(taddr, r);
  tmem_wait_ld();
  landed(r);
}
__device__ __forceinline__ void tmem_row64(uint32_t taddr, float (&r)[64]) {
  tmem_ld32_start(taddr, r);
  tmem_ld32_start(taddr + 32, r + 32);
  tmem_wait_ld();
  landed(r);
  landed(r + 32);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The weights of 64 tokens from their scores s, as fp16 pairs: w = exp2(s ks f - R) vs.  Returns the largest |w|
// and adds the exponentials to `sum`.
__device__ __forceinline__ float weights64(const float (&s)[64], uint32_t ks, uint32_t vs, float f, float R, float2& sum,
                                           uint32_t (&w)[32]) {
  float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
  const float2 f2 = make_float2(f, f), r2 = make_float2(-R, -R);
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float4 k = ld_shared_f4(ks + 16 * i), v = ld_shared_f4(vs + 16 * i);
    const float2 z0 = __ffma2_rn(__fmul2_rn(make_float2(s[4 * i], s[4 * i + 1]), make_float2(k.x, k.y)), f2, r2);
    const float2 z1 = __ffma2_rn(__fmul2_rn(make_float2(s[4 * i + 2], s[4 * i + 3]), make_float2(k.z, k.w)), f2, r2);
    const float2 p0 = make_float2(ex2(z0.x), ex2(z0.y)), p1 = make_float2(ex2(z1.x), ex2(z1.y));
    const float2 w0 = __fmul2_rn(p0, make_float2(v.x, v.y)), w1 = __fmul2_rn(p1, make_float2(v.z, v.w));
    sum0 = __fadd2_rn(sum0, p0);
    sum1 = __fadd2_rn(sum1, p1);
    m0 = max3(m0, fabsf(w0.x), fabsf(w0.y));
    m1 = max3(m1, fabsf(w1.x), fabsf(w1.y));
    w[2 * i] = half2_bits(w0.x, w0.y);
    w[2 * i + 1] = half2_bits(w1.x, w1.y);
  }
  sum = __fadd2_rn(sum0, sum1);
  return fmaxf(m0, m1);
}

// The same, stored, for tokens of which some do not count (those a row does not see, below `lo` or from `hi` on in the tile,
// or not in `valid`), or whose scores are so large that a product rounded apart from the difference decides (kWide).
// Returns the sum of the exponentials.  A loop over short code, as reference64: what runs once or twice in a unit is fetched
// each time, at several cycles an instruction.  at: the first token in the tile; the weights lie where no score is
// still to be read.
__device__ __forceinline__ float weights64_slow(uint32_t taddr, uint32_t to, uint32_t ks, uint32_t vs, float f, float R, int at, int lo,
                                                int hi, const uint32_t* valid) {
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float s[32];
    uint32_t w[16];
    tmem_row32(taddr + 32 * h, s);
    const uint32_t bits = seen32(lo, hi, at + 32 * h, valid[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 k = ld_shared_f4(ks + 128 * h + 16 * i), v = ld_shared_f4(vs + 128 * h + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 y = __fmul2_rn(make_float2(s[4 * i + e], s[4 * i + e + 1]), e == 0 ? make_float2(k.x, k.y) : make_float2(k.z, k.w));
        const float2 z = __fadd2_rn(__fmul2_rn(y, make_float2(f, f)), make_float2(-R, -R));
        const bool b0 = bits >> (4 * i + e) & 1, b1 = bits >> (4 * i + e + 1) & 1;
        const float2 p = make_float2(b0 ? ex2(z.x) : 0.0f, b1 ? ex2(z.y) : 0.0f);
        sum = __fadd2_rn(sum, p);
        // (a scale of a token that does not count is nothing to multiply by)
        w[2 * i + e / 2] = half2_bits(p.x * (b0 ? (e == 0 ? v.x : v.z) : 0.0f), p.y * (b1 ? (e == 0 ? v.y : v.w) : 0.0f));
      }
    }
    tmem_st16(to + 16 * h, w);
  }
  return sum.x + sum.y;
}

// The whole number that, as a reference, puts the largest weight of the same tokens between 2^2.1 and 2^3.2 (see kWide and kFar
// for its limits), from their scores; -infinity if none counts.
__device__ __forceinline__ float reference64(uint32_t taddr, uint32_t ks, uint32_t vs, float f, int at, int lo, int hi,
                                             const uint32_t* valid) {
  float most[4], heavy[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) most[e] = heavy[e] = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float s[32];
    tmem_row32(taddr + 32 * h, s);
    const uint32_t bits = seen32(lo, hi, at + 32 * h, valid[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 k = ld_shared_f4(ks + 128 * h + 16 * i), v = ld_shared_f4(vs + 128 * h + 16 * i);
      const float kk[4] = {k.x, k.y, k.z, k.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = bits >> (4 * i + e) & 1 ? __fmul_rn(__fmul_rn(s[4 * i + e], kk[e]), f) : -INFINITY;
        most[e] = fmaxf(most[e], x);
        heavy[e] = fmaxf(heavy[e], x > -INFINITY ? x + lg2(fabsf(vv[e])) : x);
      }
    }
  }
  most[0] = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
  heavy[0] = fmaxf(fmaxf(heavy[0], heavy[1]), fmaxf(heavy[2], heavy[3]));
  // (The scores are whole numbers from kWide on.  Rounded down, or to the nearest, references move more often: one prompt of
  // 1000 tokens 57 or 51 us, up 48.)
  // (An infinite scale is no measure for the exponentials: it makes its weights infinite by any reference.)
  const float heaviest = heavy[0] < INFINITY ? heavy[0] - 3.125f : most[0];
  return fabsf(most[0]) < kWide ? ceilf(fmaxf(heaviest, most[0] - kFar)) : most[0];
}

// 2^d as a product, for the difference d <= 0 of two references: a sum of exponentials may be as large as 2^kFar by the
// one and still count by the other, where 2^d itself is 0 in fp32.  (-infinity: 2^-252.)
__device__ __forceinline__ float2 factors(float d) {
  const int n = max(static_cast<int>(d), -252);
  return make_float2(pow2(n / 2), pow2(n - n / 2));
}

// The natural logarithm of a row's sum of exponentials, from its reference and its sum by it (the reference may
// lie far from the largest score).
__device__ __forceinline__ float log_sum(float R, float l) {
  if (l == 0.0f) return -INFINITY;  // (no token)
  const int e = exponent(l);
  return ((R + static_cast<float>(e)) + log2f(l * pow2(-e))) * 0.693147180559945309f;
}

template <int REGS>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// Segment `seg`, by a warp whose lanes all call this; false behind the last one, or if a wait has run out (then
// `ok` is false too).
__device__ __forceinline__ bool next_segment(Shared& sh, int seg, Segment& g, bool& ok, int* status) {
  ok = wait_phase(&sh.sgfull[seg % kSegments], (seg / kSegments) & 1, status);
  ok = __all_sync(0xFFFFFFFFu, ok);
  if (!ok) return false;
  g = sh.segment[seg % kSegments];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.sgempty[seg % kSegments]);
  return g.n > 0;
}

// Whether any of the segment's tokens that a row sees, those in (pos - reach, pos], has a value that is no number.  Called by
// whole warps, once converters have met such a value: the codes are read again, 32 tokens at a time.
template <class C>
__device__ __forceinline__ bool sees_nan(const AttnChunkArgs& a, const Segment& k, bool mine, int pos, int reach) {
  const int stop = min(k.first + k.n * C::BN, k.stop), lane = threadIdx.x & 31;
  bool found = false;
#pragma unroll 1
  for (int j0 = max(k.first, k.low); j0 < stop; j0 += 32) {
    bool bad = false;
    const int j = j0 + lane;
    if (j < stop) {
      const int blk = j / a.block_size, page = __ldg(a.block_table + static_cast<long long>(k.b) * a.ld_table + blk);
      const long long slot = static_cast<long long>(page) * a.block_size + (j - blk * a.block_size);
      if (page >= 0 && slot < a.num_slots) {
        const uint4* v = reinterpret_cast<const uint4*>(a.v_cache + (slot * a.kv_heads + k.head) * a.head_dim);
#pragma unroll 1
        for (int c = 0; c < a.head_dim >> 4; ++c) bad |= no_numbers(__ldg(v + c));
      }
    }
    const uint32_t tokens = __ballot_sync(0xFFFFFFFFu, bad);
    const int hi = mine ? pos + 1 - j0 : 0;
    found |= seen32(max(hi, 0) - reach, hi, 0, tokens) != 0;
  }
  return found;
}

template <int PANELS>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_chunk_kernel(const AttnChunkArgs a, const ChunkPlan p) {
  using C = ChunkCfg<PANELS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hd = a.head_dim, group = a.q_heads / a.kv_heads;

  if (tid == 0) {
    sh.nan = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.vfull[i], kConverters);
      mbar_init(&sh.vempty[i], 2);
      mbar_init(&sh.drain[i], 1);
      mbar_init(&sh.turn[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i], 128);
      mbar_init(&sh.ofull[i], 1);
    }
    for (int i = 0; i < C::K_STAGES; ++i) {
      mbar_init(&sh.kfull[i], kConverters);
      mbar_init(&sh.kempty[i], 2);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(&sh.scfull[i], 2 * kConverters);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&sh.sgfull[i], 1);
      mbar_init(&sh.sgempty[i], 14);  // the warps of the softmax, the converters and the MMAs
    }
    mbar_init(&sh.qfull, kSoftmax);
    mbar_init(&sh.meet, kSoftmax);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  // head_dim an odd multiple of 16: the MMA's last 32 columns of a score reach past the head, into bytes that no
  // copy writes; they are zero in keys (never NaN; the queries' are written as zeros)
  if (hd & 16) {
    const int col = hd & 127, panel = hd >> 7;
    for (int i = tid; i < C::K_STAGES * C::BN; i += kThreads) {
      const int st = i / C::BN, row = i % C::BN;
      *reinterpret_cast<uint4*>(smem + C::OFF_K + st * C::K_BYTES + panel * C::BN * 128 + row * 128 + (col ^ ((row & 7) << 4))) =
          make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_wait();
  griddep_launch_dependents();

  // the cost of all sequences, and where this CTA's range begins
  {
    const int chunk = (a.B + kThreads - 1) / kThreads;
    long long n = 0;
    bool bad = false;
    for (int i = 0; i < chunk; ++i) {
      const int b = tid * chunk + i;
      Seq s = {0, 0, 0};
      if (b < a.B) s = seq_of(a, b, &bad);
      n += cost_of<C>(a, s, group);
    }
    if (bad && blockIdx.x == 0) latch_bad_index(a.status);
    long long c = n * a.kv_heads;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    sh.before[tid + 1] = c;
    if (tid == 0) sh.before[0] = 0;
    __syncthreads();
    long long add = 0;
    for (int w = 0; w < warp; ++w) add += sh.before[32 * (w + 1)];
    __syncthreads();  // (the warps' sums are read before any is changed)
    sh.before[tid + 1] = c + add;
    __syncthreads();
    if (warp == 0) {
      const long long total = sh.before[kThreads];
      const long long most = (total + kMinRange - 1) / kMinRange;
      const int ranges = static_cast<int>(most < gridDim.x ? most : gridDim.x);
      if (lane == 0) {
        sh.total = total;
        sh.ranges = ranges;
      }
      if (static_cast<int>(blockIdx.x) < ranges) {
        const long long start = total * blockIdx.x / ranges;
        int lo = 0, hi = kThreads;  // the thread whose sequences hold it
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sh.before[mid] <= start) lo = mid;
          else hi = mid;
        }
        long long at = sh.before[lo];
        for (int b = lo * chunk; b < a.B; ++b) {
          const Seq s = seq_of(a, b);
          const int units = units_of<C>(a, s, group);
          bool found = false;
          for (int u0 = 0; u0 < units; u0 += 32) {  // 32 units at a time
            const int u = u0 + lane;
            const long long mine = u < units ? static_cast<long long>(unit_of<C>(a, s, group, u).cost()) * a.kv_heads : 0;
            long long inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
              if (lane >= o) inc += v;
            }
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, mine > 0 && at + inc > start);
            if (hit != 0) {
              if (lane == __ffs(hit) - 1) {
                const long long first = at + inc - mine, per = mine / a.kv_heads;
                const int head = static_cast<int>((start - first) / per);
                sh.b = b;
                sh.u = u;
                sh.head = head;
                sh.at = first + head * per;
              }
              found = true;
              break;
            }
            at += __shfl_sync(0xFFFFFFFFu, inc, 31);
          }
          if (found) break;
        }
      }
    }
    __syncthreads();
  }

  bool ok = true;
  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ converters: lane = token row for the lookups
    // (Loops of 8 copies and 4 conversions: with 2 and 2, which chain their latencies, 64 x 4 tokens take 282 us for 252; with
    // 8 and 8 prompts take 242 for 236, straight-line code of several KB running at the rate at which it is fetched.)
    fewer_regs<kRegsConvert>();
    const int w = warp - 8, chunks = hd >> 4;  // 16-byte pieces of a head
    const int sub = lane / C::LANES, piece = lane % C::LANES;
    const bool loads = piece < chunks;
    const uint32_t s_k = smem_addr(smem + C::OFF_K), s_v = smem_addr(smem + C::OFF_V);
    const uint32_t raw = smem_addr(smem + C::OFF_RAW) + (tid - kSoftmax) * 16;  // this thread's pieces
    Segment k;
    int seg = 0, t = 0, page = -1, in_page = 0, head = 0;
    bool more = next_segment(sh, 0, k, ok, a.status);
    auto look_up = [&]() {  // the page of this lane's token in tile t of the segment, from its end
      const int j = k.first + (k.n - 1 - t) * C::BN + w * C::WARP_ROWS + lane, blk = j / a.block_size;
      // (nor the pages before the unit's windows: they may have been given back)
      in_page = lane < C::WARP_ROWS && j >= k.low && j < k.stop ? j - blk * a.block_size : -1;
      if (in_page >= 0) page = __ldg(a.block_table + static_cast<long long>(k.b) * a.ld_table + blk);
      head = k.head;
    };
    if (more) look_up();
    bool have = false;
    for (int g = 0; ok && (have || more); ++g) {
      // gathers tile g (its page has been looked up) and looks up the next one's
      const bool gathers = more;
      if (gathers) {
        const int st = g % C::K_STAGES, ring = g % kRing;
        long long at = -1;
        if (in_page >= 0) {
          const long long slot = static_cast<long long>(page) * a.block_size + in_page;
          if (page < 0 || slot >= a.num_slots) latch_bad_index(a.status);
          else at = slot * a.kv_heads + head;
        }
        if (g >= C::K_STAGES) ok = wait_phase(&sh.kempty[st], (g / C::K_STAGES + 1) & 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, at >= 0);
        if (lane < C::WARP_ROWS) {
          const uint32_t n = at >= 0 ? 4 : 0;
          const long long i = at >= 0 ? at : 0;
          cp_async4(smem_addr(&sh.ks[ring][w * C::WARP_ROWS + lane]), a.k_scale + i, n);
          cp_async4(smem_addr(&sh.vs[ring][w * C::WARP_ROWS + lane]), a.v_scale + i, n);
        }
        const long long byte = at >= 0 ? at * hd : -1;
        const uint32_t k_st = s_k + st * C::K_BYTES + (piece >> 3) * (C::BN * 128), raw_st = raw + (g & 1) * C::RAW_BYTES;
#pragma unroll 8
        for (int i = 0; i < C::LOADS; ++i) {
          const int r = i * (32 / C::LANES) + sub, row = w * C::WARP_ROWS + r;
          const long long off = __shfl_sync(0xFFFFFFFFu, byte, r);
          if (loads) {
            const uint32_t n = off >= 0 ? 16 : 0;
            const long long from = off >= 0 ? off + piece * 16 : 0;
            cp_async16(k_st + row * 128 + (((piece & 7) ^ (row & 7)) << 4), a.k_cache + from, n);
            cp_async16(raw_st + i * (kConverters * 16), a.v_cache + from, n);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (a.fault == 0 || g != 0) cp_async_arrive(&sh.kfull[st]);
        cp_async_arrive(&sh.scfull[ring]);
        if (lane == 0) {
          if (C::WARP_ROWS == 32) sh.valid[ring][w] = valid;
          else reinterpret_cast<uint16_t*>(&sh.valid[ring][0])[w] = static_cast<uint16_t>(valid);
        }
        mbar_arrive(&sh.scfull[ring]);
        if (++t == k.n) {
          more = next_segment(sh, ++seg, k, ok, a.status);
          if (!ok) break;
          t = 0;
        }
        if (more) look_up();
      }
      if (have) {  // tile g - 1: the thread's own pieces as fp16 (lanes of a row write the halves of theirs in turn: no bank twice)
        if (gathers) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        const int h = g - 1;
        if (h >= 2) ok = wait_phase(&sh.vempty[h & 1], ((h >> 1) & 1) ^ 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t base = s_v + (h & 1) * C::V_BYTES + (piece >> 2) * (C::BN * 128), from = raw + (h & 1) * C::RAW_BYTES;
        const bool swap = (piece & 4) != 0;
        uint32_t nan = 0;
        auto widen = [&](int i, const uint4 codes) {
          const int row = w * C::WARP_ROWS + i * (32 / C::LANES) + sub;
          uint4 lo, hi;
          widen16(codes, lo, hi);
          note_nan(lo, nan);
          note_nan(hi, nan);
          const uint32_t c0 = ((2 * piece) & 7) ^ (row & 7);
          st_shared(base + row * 128 + ((swap ? c0 ^ 1 : c0) << 4), swap ? hi : lo);
          st_shared(base + row * 128 + ((swap ? c0 : c0 ^ 1) << 4), swap ? lo : hi);
        };
        // A value that is no number must not meet the weights of zero of the rows that do not see its token: its code becomes 0 and
        // the pieces are widened again; the rows that see it are found once the segment is done (sees_nan).  Watching for it, two
        // instructions per 8 codes in place of a minimum that would hide it, costs 3% (eight prompts of 1000 tokens 235 us, 228).
#pragma unroll 1
        for (int clean = 0; clean < 2; ++clean) {
          nan = 0;
#pragma unroll 4
          for (int i = 0; i < C::LOADS; ++i)
            if (loads) widen(i, ld_shared(from + i * (kConverters * 16)));
          if (__builtin_expect(!has_nan(nan), 1)) break;
          sh.nan = 1;
#pragma unroll 1
          for (int i = 0; i < C::LOADS; ++i) {
            const uint4 c = ld_shared(from + i * (kConverters * 16));
            st_shared(from + i * (kConverters * 16), make_uint4(numbers_only(c.x), numbers_only(c.y), numbers_only(c.z), numbers_only(c.w)));
          }
        }
        mbar_arrive(&sh.vfull[h & 1]);
      }
      have = gathers;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 12) {
    // ------------------------------------------------------------ MMA issuers, one for each row tile
    fewer_regs<kRegsMma>();
    if (warp < 14) {
      // the whole warp goes through the steps, its first lane issues
      const int mma = __shfl_sync(0xFFFFFFFFu, warp, 0) - 12;  // the row tile whose MMAs this warp issues
      const uint32_t lead = lane == 0 ? 1 : 0, tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, a.status)) != 0; };
      auto commit = [&](uint64_t* bar) {
        if (lead) umma_commit(bar);
      };
      constexpr uint32_t id_hi = umma_idesc_f32acc(0, 0, 128, C::BN), id_lo = umma_idesc_f32acc(1, 0, 128, C::BN);  // e4m3, e5m2
      const uint32_t id_o = umma_idesc_f32acc(0, 0, 128, hd) | (1u << 16);  // B (values) transposed
      const uint64_t q0 = umma_desc_sw128(smem_addr(smem)), k0 = umma_desc_sw128(smem_addr(smem) + C::OFF_K),
                     v0 = desc_transposed(smem_addr(smem) + C::OFF_V, C::BN * 128);
      const int ksteps = (hd + 31) >> 5;
      int g = 0, seg = 0, steps = 0;
      uint32_t before = 0;  // bit b: parity of the tiles that went through score buffer b before this segment
      auto scores = [&](int tile, int buf, int st) {
        const uint32_t qd = static_cast<uint32_t>(q0) + tile * (2 * C::Q_PIECE / 16), kd = static_cast<uint32_t>(k0) + st * (C::K_BYTES / 16);
        const uint32_t at = tm + buf * C::TM_S;
#pragma unroll(PANELS <= 2 ? 2 : 1)
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int kk = 0; kk < 2 * PANELS; ++kk)
            umma_scores(at, qd + (half * C::Q_PIECE + (kk >> 2) * (128 * 128) + (kk & 3) * 32) / 16,
                        kd + ((kk >> 2) * (C::BN * 128) + (kk & 3) * 32) / 16, static_cast<uint32_t>(q0 >> 32), half != 0 ? id_lo : id_hi, half | kk, kk < ksteps ? lead : 0);
        commit(&sh.sfull[buf]);
      };
      auto outputs = [&](int tile, int buf, int st, int use, bool first) {
        if (!wait(&sh.pfull[buf], ((before >> buf) + use) & 1)) return false;
        tc_fence_after();
        const uint32_t vd = static_cast<uint32_t>(v0) + st * (C::V_BYTES / 16);
        const uint32_t p_at = tm + buf * C::TM_S, o_at = tm + C::TM_O + tile * 64 * PANELS;
#pragma unroll
        for (int kk = 0; kk < C::BN / 16; ++kk) umma_outputs(o_at, p_at + kk * 8, vd + kk * (16 * 128 / 16), static_cast<uint32_t>(v0 >> 32), id_o, kk > 0 || !first ? 1 : 0, lead);
        commit(&sh.ofull[tile]);
        return true;
      };
      auto keys = [&](int i) {
        // (the converters' copies and stores are fenced here, where nothing is on its way: a fence waits for loads)
        if (!wait(&sh.kfull[i % C::K_STAGES], (i / C::K_STAGES) & 1)) return false;
        fence_proxy_async_smem();
        tc_fence_after();
        return true;
      };
      auto values = [&](int i) {
        if (!wait(&sh.vfull[i & 1], (i >> 1) & 1)) return false;
        fence_proxy_async_smem();
        return true;
      };
      for (; ok; ++seg) {
        ok = wait(&sh.sgfull[seg % kSegments], (seg / kSegments) & 1);
        if (!ok) break;
        const int n = __shfl_sync(0xFFFFFFFFu, sh.segment[seg % kSegments].n, 0);
        const bool two = __shfl_sync(0xFFFFFFFFu, sh.segment[seg % kSegments].rows, 0) > 128;
        __syncwarp();
        if (lead) mbar_arrive(&sh.sgempty[seg % kSegments]);
        if (n == 0) break;
        ok = wait(&sh.qfull, seg & 1);
        if (!ok) break;
        tc_fence_after();
        if (two) {  // the outputs of tile i - 1, then the scores of tile i, which take the weights' place
          for (int i = 0; i <= n && ok; ++i) {
            if (i < n) ok = keys(g + i);
            // the tiles take turns: MMAs of both in one another's midst would end together, both softmax groups would
            // then run side by side and the tensor core wait for both
            auto turn = [&]() { return mma == 0 ? steps == 0 || wait(&sh.turn[1], (steps - 1) & 1) : wait(&sh.turn[0], steps & 1); };
            if (ok && i == 0) ok = turn();
            if (ok && i > 0) {
              ok = values(g + i - 1) && turn() && outputs(mma, mma, (g + i - 1) & 1, i - 1, i == 1);
              if (ok) commit(&sh.vempty[(g + i - 1) & 1]);
            }
            if (ok && i < n) {
              scores(mma, mma, (g + i) % C::K_STAGES);
              commit(&sh.kempty[(g + i) % C::K_STAGES]);
            }
            if (lead) mbar_arrive(&sh.turn[mma]);
            ++steps;
          }
        } else if (mma == 0) {  // one row tile: the scores of tile i, in the other buffer, then the outputs of tile i - 1
          for (int i = 0; i <= n && ok; ++i) {
            if (i < n) {
              ok = keys(g + i);
              if (!ok) break;
              scores(0, i & 1, (g + i) % C::K_STAGES);
              commit(&sh.kempty[(g + i) % C::K_STAGES]);
              commit(&sh.kempty[(g + i) % C::K_STAGES]);  // (for the other thread)
            }
            if (i > 0) {
              ok = values(g + i - 1) && outputs(0, (i - 1) & 1, (g + i - 1) & 1, (i - 1) >> 1, i == 1);
              if (!ok) break;
              commit(&sh.vempty[(g + i - 1) & 1]);
              commit(&sh.vempty[(g + i - 1) & 1]);
            }
          }
        }
        g += n;
        before ^= two ? 3u * (n & 1) : ((n + 1) >> 1 & 1) | (n >> 1 & 1) << 1;
      }
      commit(&sh.drain[mma]);
      wait_drain(&sh.drain[mma], 0, a.status);
    } else if (warp == 14) {
      // ---------------------------------------------------------- the segments, for all the others
      Walk<C> k(a, sh);
      bool more = true;
      for (int seg = 0; ok && more; ++seg) {
        more = k.next();
        const int slot = seg % kSegments;
        if (seg >= kSegments) ok = wait_phase(&sh.sgempty[slot], (seg / kSegments + 1) & 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok && lane == 0) {
          Segment g = {};
          if (more) {
            const bool whole = k.t0 == 0 && k.t1 == k.w.tiles;
            g = {k.t1 - k.t0, k.b, k.head, k.s.row0, k.s.len - k.s.fresh, k.w.row, k.w.rows, (k.w.tile0 + k.t0) * C::BN, k.w.low,
                 k.s.len - k.s.fresh + (k.w.row + k.w.rows - 1) / group + 1,
                 whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (k.t0 == 0 ? 1 : 0), 0, 0};
            if (!whole) {
              g.r0 = k.first_range();
              g.r1 = k.last_range();
            }
          }
          sh.segment[slot] = g;
          mbar_arrive(&sh.sgfull[slot]);
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax: a row a thread
    more_regs<kRegsSoftmax>();
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // tokens before the first position see nothing
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const Seq s = seq_of(a, b);
      const int none = min(s.fresh, s.fresh - s.len);
      for (int i = 0; i < none; ++i) {
        const long long row = s.row0 + i;
        for (unsigned c = tid; c < static_cast<unsigned>(a.q_heads * hd); c += kSoftmax)  // (a row may have nearly 2^31 columns)
          a.out[row * a.ldo + c] = __float2bfloat16_rn(0.0f);
        if (a.lse)
          for (int c = tid; c < a.q_heads; c += kSoftmax) a.lse[row * a.q_heads + c] = -INFINITY;
      }
    }
    int g = 0, meets = 0;
    uint32_t before = 0, done = 0;  // bit b: parity of the tiles that went through score buffer b before this segment; outputs of this row tile
    // the softmax threads wait for one another
    auto meet = [&]() {
      mbar_arrive(&sh.meet);
      ok = wait_phase(&sh.meet, meets++ & 1, a.status);
      ok = __all_sync(0xFFFFFFFFu, ok);
      return ok;
    };
    // Queries: copied as they are while the last tile of the segment before is under way, then turned in place into two
    // pieces, e4m3 and the rest as e5m2 (16 values as bf16 lie where their 16 bytes of each piece come to lie).
    const int q_steps = (hd + 31) >> 5 << 1;
    const uint32_t q_tile = smem_addr(smem) + 2 * tile * C::Q_PIECE;
    auto spot = [&](int row, int step) { return q_tile + (step >> 3) * (128 * 128) + row * 128 + (((step & 7) ^ (row & 7)) << 4); };
    auto copy_queries = [&](const Segment& s) {  // the warp's rows; zeros past the head and past the unit
      if (tile * 128 >= s.rows && tile != 0) return;
      const int vec = lane % C::Q_LANES;
      constexpr int kStep = 32 / C::Q_LANES;  // rows that the warp copies at a time
      int row = (warp & 3) * 32 + lane / C::Q_LANES;
      int token = (s.row + tile * 128 + row) / group, qh = s.row + tile * 128 + row - token * group;  // (head of the group)
#pragma unroll 4
      for (int x = 0; x < C::Q_LANES; ++x) {
        const bool there = tile * 128 + row < s.rows && vec * 8 < hd;
        const __nv_bfloat16* src = a.q;
        if (there) src += static_cast<long long>(s.qrow + token) * a.ldq + static_cast<long long>(s.head * group + qh) * hd + vec * 8;
        if (vec < 2 * q_steps) cp_async16(spot(row, vec >> 1) + (vec & 1) * C::Q_PIECE, src, there ? 16 : 0);
        row += kStep;
        for (qh += kStep; qh >= group; qh -= group) ++token;
      }
    };
    auto turn_queries = [&]() {  // this thread's row; returns what makes log2 units of a raw score times the key's scale
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      __nv_bfloat162 m = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll 2
      for (int i = 0; i < q_steps; ++i) {
        const uint4 u0 = ld_shared(spot(r, i)), u1 = ld_shared(spot(r, i) + C::Q_PIECE);
        const uint32_t uw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = uw[e] & 0x7FFF7FFFu;
          m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&x));
        }
      }
      const float top = fmaxf(__low2float(m), __high2float(m));
      // (a row below 2^-113: fewer bits, nothing to score)
      const int up = min(7 - exponent(top), 120);
      const float f1 = a.scale < 0.0f ? -pow2(up / 2) : pow2(up / 2), f2 = pow2(up - up / 2);
#pragma unroll 1
      for (int i = 0; i < q_steps; ++i) {
        const uint4 u0 = ld_shared(spot(r, i)), u1 = ld_shared(spot(r, i) + C::Q_PIECE);
        const uint32_t uw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = __uint_as_float(uw[e] << 16) * f1 * f2, x1 = __uint_as_float(uw[e] & 0xFFFF0000u) * f1 * f2;
          const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
          const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
          const uint32_t d = __nv_cvt_float2_to_fp8x2(make_float2(x0 - v.x, x1 - v.y), __NV_SATFINITE, __NV_E5M2);
          hi[e >> 1] = (e & 1) != 0 ? hi[e >> 1] | c << 16 : c;
          lo[e >> 1] = (e & 1) != 0 ? lo[e >> 1] | d << 16 : d;
        }
        st_shared(spot(r, i), make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared(spot(r, i) + C::Q_PIECE, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      fence_proxy_async_smem();
      // (e4m3 and e5m2 here end at their largest numbers: an infinite value is not in the pieces, so it is in the factor)
      return top < INFINITY ? fabsf(a.scale) * 1.44269504088896340736f / fabsf(f1) / f2 : __uint_as_float(0x7FC00000u);
    };
    Segment k;
    float f = 0.0f;
    bool more = next_segment(sh, 0, k, ok, a.status);
    if (more) {
      copy_queries(k);
      if (tile == 0 || k.rows > 128) f = turn_queries();
      mbar_arrive(&sh.qfull);
    }
    for (int seg = 0; ok && more; ++seg) {
      const int n = k.n;
      const bool two = k.rows > 128, active = tile == 0 || two;
      const bool mine = tile * 128 + r < k.rows;
      const int pair = k.row + tile * 128 + r;  // this thread's (token, head)
      const int token = pair / group, qh = k.head * group + (pair - token * group);
      const int pos = k.pos + token;
      const uint32_t o_addr = lane_base + C::TM_O + tile * 64 * PANELS;
      float R = -INFINITY, l = 0.0f;
      bool wide = false, fresh = true;  // (fresh: no reference yet)
      bool nan = false;                 // one of the values that the row sees is no number
      if (active) {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int buf = two ? tile : i & 1, ring = (g + i) % kRing;
          ok = wait_phase(&sh.scfull[ring], ((g + i) / kRing) & 1, a.status) &&
               wait_phase(&sh.sfull[buf], ((before >> buf) + (two ? i : i >> 1)) & 1, a.status);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          if (i == n - 1) {  // the queries have been read: the next segment's
            ok = wait_phase(&sh.sgfull[(seg + 1) % kSegments], ((seg + 1) / kSegments) & 1, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (sh.segment[(seg + 1) % kSegments].n > 0) copy_queries(sh.segment[(seg + 1) % kSegments]);
          }
          const uint32_t s_addr = lane_base + buf * C::TM_S;
          // columns of this tile that the row sees (a row past the unit's: all, of a query of zeros; none in a warp of such rows)
          const int j0 = k.first + (n - 1 - i) * C::BN;
          const int hi = mine ? pos + 1 - j0 : tile * 128 + (warp & 3) * 32 < k.rows ? C::BN : 0, reach = mine && a.window > 0 ? a.window : INT_MAX;
          bool waited = i == 0;  // for the outputs of the tile before
          uint32_t every = 0xFFFFFFFFu;
#pragma unroll
          for (int c = 0; c < C::BN / 32; ++c) every &= sh.valid[ring][c];
          const bool mask = __any_sync(0xFFFFFFFFu, hi > reach || hi < C::BN || every != 0xFFFFFFFFu);
#pragma unroll 1
          for (int c = 0; c < C::BN / 64; ++c) {
            const uint32_t ks = smem_addr(sh.ks[ring]) + 256 * c, vs = smem_addr(sh.vs[ring]) + 256 * c;
            if (!mask && !wide && !fresh) {
              float s[64];
              uint32_t w[32];
              float2 sum;
              tmem_row64(s_addr + 64 * c, s);
              const float top = weights64(s, ks, vs, f, R, sum, w);
              // (the sum too: of tokens without a value, and of all where there is no reference yet)
              const bool over = !(top <= kHeavy) || !(sum.x + sum.y <= kMuch);
              if (__builtin_expect(!__any_sync(0xFFFFFFFFu, over), 1)) {
                l += sum.x + sum.y;
                tmem_st32(s_addr + 32 * c, w);
                continue;
              }
            }
            const int lo = max(hi, 0) - reach;
            if ((sh.valid[ring][2 * c] | sh.valid[ring][2 * c + 1]) == 0 ||
                !__any_sync(0xFFFFFFFFu, hi > 64 * c && lo < 64 * c + 64)) {  // no row of the warp sees any of these tokens
              const uint32_t none[16] = {};
              tmem_st16(s_addr + 32 * c, none);
              tmem_st16(s_addr + 32 * c + 16, none);
              continue;
            }
            const float to = reference64(s_addr + 64 * c, ks, vs, f, 64 * c, lo, hi, &sh.valid[ring][2 * c]);
            float2 by = make_float2(1.0f, 1.0f);  // what the old reference's terms are multiplied by
            // (not for 2^8 or less: the weights may be as much above where a reference puts them)
            const bool moves = to > R + 8.0f || (fabsf(to) >= kWide && to > R);
            if (moves) {
              by = factors(R - to);
              R = to;
            }
            wide = __any_sync(0xFFFFFFFFu, wide || (fabsf(R) >= kWide && R > -INFINITY));
            if (!fresh && __any_sync(0xFFFFFFFFu, moves)) {
              // what was summed by the old reference is scaled
              l = l * by.x * by.y;
              const float back = by.x * by.y;
              if (!waited) {
                ok = wait_phase(&sh.ofull[tile], (done - 1) & 1, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                waited = true;
                tc_fence_after();
              }
              const int outs = i > 0 ? hd : 0;
              tmem_wait_st();
#pragma unroll 1
              for (int x = 0; x < outs; x += 16) {
                uint32_t o[16];
                tmem_ld16(o_addr + x, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * back);
                tmem_st16(o_addr + x, o);
              }
#pragma unroll 1
              for (int x = 0; x < 32 * c; x += 16) {
                uint32_t o[16];
                tmem_ld16(s_addr + x, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
                  o[e] = half2_bits(v.x * back, v.y * back);
                }
                tmem_st16(s_addr + x, o);
              }
            }
            fresh = false;
            l += weights64_slow(s_addr + 64 * c, s_addr + 32 * c, ks, vs, f, R, 64 * c, lo, hi, &sh.valid[ring][2 * c]);
          }
          if (!ok) break;
          // the weights are only handed over once the outputs of the tile before are there: a wait by parity must not
          // be two phases behind
          if (!waited) {
            ok = wait_phase(&sh.ofull[tile], (done - 1) & 1, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sh.pfull[buf]);
          ++done;
        }
        if (ok) ok = wait_phase(&sh.ofull[tile], (done - 1) & 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;  // nothing is stored, counted or joined
        tc_fence_after();
        // (set before the last outputs' values were handed over)
        if (__builtin_expect(*reinterpret_cast<volatile int*>(&sh.nan) != 0, 0))
          nan = sees_nan<C>(a, k, mine, pos, mine && a.window > 0 ? a.window : INT_MAX);
      }
      // (the group without rows waits for the other: the score buffers' and the scales' phases that it did not watch
      // have passed when it watches them again)
      if (!two && !meet()) break;
      g += n;
      before ^= two ? 3u * (n & 1) : ((n + 1) >> 1 & 1) | (n >> 1 & 1) << 1;
      // the next segment's scores are computed while this one's outputs are stored
      const Segment was = k;
      more = next_segment(sh, seg + 1, k, ok, a.status);
      if (!ok) break;
      if (more) {
        if (!active) copy_queries(k);  // (the other threads have)
        if (tile == 0 || k.rows > 128) f = turn_queries();
        tc_fence_before();
        mbar_arrive(&sh.qfull);
      }
      const bool whole = was.part < 0;
      if (active) {
        // the whole unit: the outputs; a part of it: (reference, sum, unnormalised outputs) into the workspace
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const long long orow = was.qrow + token;
        __nv_bfloat16* out = a.out + orow * a.ldo + static_cast<long long>(qh) * hd;
        float* dst = p.partial + static_cast<long long>(whole ? 0 : was.part) * C::ROWS * hd + (tile * 128 + r) * 4;
#pragma unroll 1
        for (int c = 0; c < hd; c += 16) {
          uint32_t u[16];
          tmem_ld16(o_addr + c, u);
          if (__builtin_expect(nan, 0)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = 0x7FC00000u;
          }
          if (mine && whole) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(u[2 * e]) * inv, __uint_as_float(u[2 * e + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(reinterpret_cast<uint4*>(dst + static_cast<long long>(c / 4 + e) * C::ROWS * 4),
                     make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]));
          }
          __syncwarp();
        }
        if (mine && whole && a.lse) a.lse[orow * a.q_heads + qh] = log_sum(R, l);
        if (mine && !whole)
          __stcg(reinterpret_cast<float2*>(p.partial_ml + (static_cast<long long>(was.part) * C::ROWS + tile * 128 + r) * 2), make_float2(R, l));
      }
      tc_fence_before();
      if (whole) continue;
      __threadfence();
      if (!meet()) break;
      if (tid == 0) {
        sh.last = atomicAdd(p.counter + was.r0, 1u) == static_cast<unsigned>(was.r1 - was.r0);
        if (sh.last) p.counter[was.r0] = 0;  // ready for the next call
        __threadfence();
      }
      if (!meet()) break;
      if (sh.last == 0) continue;
      // the parts in order of their ranges; a thread takes 4 columns of a row, of 4 rows at a time
      const int all = was.rows * (hd >> 2);
#pragma unroll 1
      for (int it0 = tid; it0 < all; it0 += 4 * kSoftmax) {
        float m[4], sum[4];
        float4 o[4];
        int c4[4], rr[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int it = min(it0 + y * kSoftmax, all - 1);
          c4[y] = it / was.rows;
          rr[y] = it - c4[y] * was.rows;
          m[y] = -INFINITY;
          sum[y] = 0.0f;
          o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll 2
        for (int x = was.r0; x <= was.r1; ++x) {
          const long long q = (2LL * x + (x == was.r0 ? 1 : 0)) * C::ROWS;
          float2 ml[4];
          float4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            ml[y] = __ldcg(reinterpret_cast<const float2*>(p.partial_ml + (q + rr[y]) * 2));
            v[y] = __ldcg(reinterpret_cast<const float4*>(p.partial + q * hd + (static_cast<long long>(c4[y]) * C::ROWS + rr[y]) * 4));
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float to = fmaxf(m[y], ml[y].x);
            // (the square roots of the factors: a sum is scaled in two steps, as where a reference moves; nothing has been rounded
            // to 16 bits here, so that they need not be exact)
            const float h0 = m[y] > -INFINITY ? ex2(0.5f * (m[y] - to)) : 0.0f;
            const float h1 = ml[y].x > -INFINITY ? ex2(0.5f * (ml[y].x - to)) : 0.0f;
            const float f0 = h0 * h0, f1 = h1 * h1;
            m[y] = to;
            sum[y] = sum[y] * h0 * h0 + ml[y].y * h1 * h1;
            o[y].x = o[y].x * f0 + v[y].x * f1;
            o[y].y = o[y].y * f0 + v[y].y * f1;
            o[y].z = o[y].z * f0 + v[y].z * f1;
            o[y].w = o[y].w * f0 + v[y].w * f1;
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (it0 + y * kSoftmax >= all) break;
          const int pr = was.row + rr[y], tok = pr / group, h = was.head * group + (pr - tok * group);
          const float inv = sum[y] > 0.0f ? 1.0f / sum[y] : 0.0f;
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(o[y].x * inv, o[y].y * inv), h1 = __floats2bfloat162_rn(o[y].z * inv, o[y].w * inv);
          *reinterpret_cast<uint2*>(a.out + static_cast<long long>(was.qrow + tok) * a.ldo + static_cast<long long>(h) * hd + 4 * c4[y]) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
          if (a.lse && c4[y] == 0) a.lse[static_cast<long long>(was.qrow + tok) * a.q_heads + h] = log_sum(m[y], sum[y]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (behind a wait that ran out)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t counter_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * sizeof(unsigned) + 255) & ~static_cast<size_t>(255); }
int rows_of(int head_dim) { return head_dim <= 128 ? 256 : 128; }

template <int PANELS>
cudaError_t launch_inst(const AttnChunkArgs& a, const ChunkPlan& p, int grid, cudaStream_t st) {
  auto kern = kv_attn_chunk_kernel<PANELS>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<PANELS>::SMEM);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl(kern, dim3(grid), dim3(kThreads), ChunkCfg<PANELS>::SMEM, st, a, p);
}

}  // namespace

size_t attn_chunk_workspace_bytes(int, int, int head_dim, int num_sms) {
  return counter_bytes(num_sms) + static_cast<size_t>(2) * num_sms * rows_of(head_dim) * (head_dim + 2) * 4;
}

cudaError_t launch_kv_attn_chunk(const AttnChunkArgs& a, int num_sms, cudaStream_t st) {
  ChunkPlan p{};
  p.counter = reinterpret_cast<unsigned*>(a.ws);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + counter_bytes(num_sms));
  p.partial_ml = p.partial + static_cast<size_t>(2) * num_sms * rows_of(a.head_dim) * a.head_dim;
  if (a.head_dim <= 64) return launch_inst<1>(a, p, num_sms, st);
  if (a.head_dim <= 128) return launch_inst<2>(a, p, num_sms, st);
  if (a.head_dim <= 192) return launch_inst<3>(a, p, num_sms, st);
  return launch_inst<4>(a, p, num_sms, st);
}

}  // namespace qurl
