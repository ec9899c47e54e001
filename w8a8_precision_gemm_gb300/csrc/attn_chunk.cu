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
// Both products run as kind::f16: every e4m3 code is an fp16 number, so keys and
// values are converted without a rounding and their scales are applied in fp32, the keys' to
// the scores, the values' to the weights.
//   * A query row, scaled by a power of two so that its largest value is in [2^14, 2^15),
//     is an fp16 row: a bf16 value has 8 significant bits, so values within 2^-31 of the largest are
//     exact and smaller ones off by at most 2^-40 of it.  Products are exact, sums fp32.
//   * The weights w_ij = exp2(x_ij - R_i) vs_j (x: scores in log2 units) are rounded to
//     fp16, 2^-12 of a value of 2^-14 or more and 2^-25 below.  The reference R_i
//     is a bound on log2 of row i's largest p vs so far, less 8 to 15: the largest weight
//     lies in [2^8, 2^15) if the bound is met.  It is the largest score and the tile's
//     largest value scale together while a tile's scales lie within 2^6 of each other;
//     a tile with others takes the largest of x_ij + log2 vs_j itself.  So what is lost
//     of a row is below 2^-27 of its largest weight for every token.
//
// Rows of the MMAs are (token, query head of the group) pairs in a row, so a group of any
// size fills them: 256 rows in two tiles of 128 (one for head_dim above 128) against tiles of 128
// (64) tokens.  Four warps gather a tile's codes through the block table, convert them
// and write them swizzled into shared memory; one thread issues the MMAs (scores: both
// operands in shared memory; output: weights in TMEM in the place of the scores, the value tile
// read transposed); four warps per row tile do the softmax, a row a thread, one row
// tile's softmax beside the other's MMAs.  A unit of one row tile takes the two score
// buffers in turn instead.  The outputs stay in TMEM and are rescaled when a reference moves.
//
// A unit of work is (row tiles of a sequence, KV head).  The token tiles of all units in a
// row, each unit with a fixed amount for its start and end, are cut into equal
// ranges, one per CTA, whatever the lengths; a unit that lies in several ranges leaves
// partial sums in the workspace, and the CTA that is done with it last joins
// them in order: one launch, the same result every run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"

namespace qurl {
namespace {

constexpr int kSoftmax = 256;     // threads 0..255: two groups of 128, a row a thread
constexpr int kConverters = 128;  // threads 256..383
constexpr int kThreads = kSoftmax + kConverters + 32;  // and the MMA warp
constexpr int kRing = 8;          // tiles whose scales are kept
// What a unit costs beside its tiles, in tiles of one row tile, and the least that a range gets.
constexpr int kUnitCost = 2;
constexpr int kMinRange = 8;
constexpr float kWide = 0x1p24f;  // scores from here on are not told apart from their neighbours

// PANELS: 64-column panels of a head.
template <int PANELS_>
struct ChunkCfg {
  static constexpr int PANELS = PANELS_;
  static constexpr int TILES = PANELS <= 2 ? 2 : 1;    // row tiles
  static constexpr int ROWS = 128 * TILES;
  static constexpr int BN = PANELS <= 2 ? 128 : 64;    // tokens per tile
  static constexpr int STAGES = 2;
  static constexpr int Q_BYTES = PANELS * 128 * 128;   // a row tile of queries
  static constexpr int KV_BYTES = PANELS * BN * 128;   // a tile of keys, or of values
  static constexpr int OFF_K = TILES * Q_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * KV_BYTES;
  static constexpr int SMEM = OFF_V + STAGES * KV_BYTES + 1024;
  static constexpr int LANES = PANELS == 1 ? 4 : PANELS == 2 ? 8 : 16;  // lanes per token row in the gather
  static constexpr int WARP_ROWS = BN / 4;             // token rows of a tile per converter warp
  static constexpr int LOADS = WARP_ROWS * LANES / 32; // 16-byte pieces per lane, keys and values each
  static constexpr int TM_S = BN;                      // columns between the two score buffers
  static constexpr int TM_O = 256;                     // first column of the outputs (64 PANELS per row tile)
  static_assert(2 * TM_S <= TM_O && TM_O + TILES * 64 * PANELS <= 512, "TMEM columns");
  static_assert(SMEM <= 216 * 1024, "shared memory");
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
__device__ __forceinline__ float warp_fmax(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// 2^n, n in [-126, 127], and floor(log2 x) of a normal x > 0 (-127 for zero and subnormals).
__device__ __forceinline__ float pow2(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }

// mbar_wait (ptx.cuh) that gives up for a timeout only: a page out of range latched by
// this kernel leaves the other sequences' results alone.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(status) == kDevTimeout) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
  return true;
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

__device__ __forceinline__ void umma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

// One arrival per thread of the softmax warps, and whether `v` holds in any of them.
__device__ __forceinline__ bool any_of(bool v) {
  int r = v ? 1 : 0;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %0, 0;\n\tbarrier.cta.red.or.pred b, 1, 256, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
      : "+r"(r)::"memory");
  return r != 0;
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
  int weight;  // row tiles
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
  const int lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  w.tile0 = lo / C::BN;
  w.tiles = last < 0 ? 0 : last / C::BN + 1 - w.tile0;
  w.weight = w.rows > 128 ? 2 : 1;
  return w;
}

struct Shared {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];  // a stage of keys, of values
  uint64_t scfull[kRing];                             // the scales of a tile
  uint64_t qfull;                                     // a segment's queries, and its outputs may be overwritten
  uint64_t sfull[2], pfull[2], ofull[2];              // scores, weights (per score buffer), outputs (per row tile)
  uint64_t drain;
  uint32_t tmem;
  int ranges;                 // ranges in use
  long long total;            // the cost of all units
  long long before[kThreads + 1];  // cost before each thread's sequences
  // where this CTA's range begins
  int b, u, head;
  long long at;               // cost before that unit
  alignas(16) float ks[kRing][128];
  alignas(16) float vs[kRing][128];
  float vmax[kRing][4], vmin[kRing][4];  // of the scales each converter warp has loaded (0, infinity: none)
  uint32_t valid[kRing][4];   // tokens whose page exists
  int last;
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

// Walks the segments (one unit's tiles inside this CTA's range) in order; every role
// walks the same ones.
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
    w = {0, 0, 0, 0, 0};
    s = {0, 0, 0};
    end = static_cast<int>(blockIdx.x) < sh.ranges ? range_start(sh, blockIdx.x + 1) : -1;
    if (end < 0) at = 0;
    else {
      s = seq_of(a, b);
      w = unit_of<C>(a, s, group, u);
      at -= w.cost();
    }
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
      const long long base = at + kUnitCost;  // tile t costs [base + t weight, + weight)
      t0 = start > base ? static_cast<int>(min((start - base + w.weight - 1) / w.weight, static_cast<long long>(w.tiles))) : 0;
      t1 = end > base ? static_cast<int>(min((end - base + w.weight - 1) / w.weight, static_cast<long long>(w.tiles))) : 0;
      if (t1 > t0) return true;
    }
  }
  // the range that holds a tile of this unit
  __device__ int range_of(int t) const {
    const long long p = at + kUnitCost + static_cast<long long>(t) * w.weight;
    return static_cast<int>(((p + 1) * sh.ranges - 1) / sh.total);
  }
};

// 16 codes -> 32 bytes of fp16.
__device__ __forceinline__ void widen16(const uint4 c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xFFFF), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
    o[2 * i] = static_cast<uint32_t>(a.x) | static_cast<uint32_t>(a.y) << 16;
    o[2 * i + 1] = static_cast<uint32_t>(b.x) | static_cast<uint32_t>(b.y) << 16;
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A tile's scores seen by one row: columns [lo, hi) of the tile, and only those that are valid.
struct Seen {
  int lo, hi;
  __device__ uint32_t bits(int chunk, uint32_t valid) const {
    const int l = min(max(lo - 32 * chunk, 0), 32), h = min(max(hi - 32 * chunk, 0), 32);
    const uint32_t below_h = h == 32 ? 0xFFFFFFFFu : (1u << h) - 1, below_l = l == 32 ? 0xFFFFFFFFu : (1u << l) - 1;
    return below_h & ~below_l & valid;
  }
};

// The largest of the scores s_j ks_j over the columns a row sees (not yet times the row's factor).
template <int BN, bool MASK>
__device__ __forceinline__ float tile_max(uint32_t s_addr, const float* ks, const Seen& seen, const uint32_t* valid) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t s[32];
    tmem_ld32(s_addr + 32 * c, s);
    const uint32_t bits = MASK ? seen.bits(c, valid[c]) : 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + 4 * i);
      const float2 y0 = __fmul2_rn(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), make_float2(k.x, k.y));
      const float2 y1 = __fmul2_rn(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), make_float2(k.z, k.w));
      if (MASK) {
        if (bits >> (4 * i) & 1) m0 = fmaxf(m0, y0.x);
        if (bits >> (4 * i + 1) & 1) m1 = fmaxf(m1, y0.y);
        if (bits >> (4 * i + 2) & 1) m0 = fmaxf(m0, y1.x);
        if (bits >> (4 * i + 3) & 1) m1 = fmaxf(m1, y1.y);
      } else {
        m0 = fmaxf(m0, fmaxf(y0.x, y1.x));
        m1 = fmaxf(m1, fmaxf(y0.y, y1.y));
      }
    }
  }
  return fmaxf(m0, m1);
}

// The largest of x_j + log2 |vs_j| over the columns a row sees.
template <int BN>
__device__ __noinline__ float tile_max_weight(uint32_t s_addr, const float* ks, const float* vs, float f, Seen seen,
                                              const uint32_t* valid) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t s[32];
    tmem_ld32(s_addr + 32 * c, s);
    const uint32_t bits = seen.bits(c, valid[c]);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float y = __fmul_rn(__fmul_rn(__uint_as_float(s[i]), ks[32 * c + i]), f) + lg2(fabsf(vs[32 * c + i]));
      if (bits >> i & 1) m = fmaxf(m, y);
    }
  }
  return m;
}

// The weights of a tile, written over its scores as fp16 pairs; returns the sum of exp2(x_j - R).
// WIDE: scores so large that a product rounded apart from the difference decides (kWide).
template <int BN, bool MASK, bool WIDE>
__device__ __forceinline__ float tile_weights(uint32_t s_addr, const float* ks, const float* vs, float f, float R,
                                              const Seen& seen, const uint32_t* valid) {
  float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
  const float2 f2 = make_float2(f, f), r2 = make_float2(-R, -R);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t s[32];
    tmem_ld32(s_addr + 32 * c, s);
    const uint32_t bits = MASK ? seen.bits(c, valid[c]) : 0xFFFFFFFFu;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + 4 * i);
      const float4 v = *reinterpret_cast<const float4*>(vs + 32 * c + 4 * i);
      const float2 y0 = __fmul2_rn(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), make_float2(k.x, k.y));
      const float2 y1 = __fmul2_rn(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), make_float2(k.z, k.w));
      const float2 z0 = WIDE ? __fadd2_rn(__fmul2_rn(y0, f2), r2) : __ffma2_rn(y0, f2, r2);
      const float2 z1 = WIDE ? __fadd2_rn(__fmul2_rn(y1, f2), r2) : __ffma2_rn(y1, f2, r2);
      float2 p0 = make_float2(ex2(z0.x), ex2(z0.y)), p1 = make_float2(ex2(z1.x), ex2(z1.y));
      float2 w0, w1;
      if (MASK) {
        const bool b0 = bits >> (4 * i) & 1, b1 = bits >> (4 * i + 1) & 1, b2 = bits >> (4 * i + 2) & 1, b3 = bits >> (4 * i + 3) & 1;
        p0 = make_float2(b0 ? p0.x : 0.0f, b1 ? p0.y : 0.0f);
        p1 = make_float2(b2 ? p1.x : 0.0f, b3 ? p1.y : 0.0f);
        w0 = make_float2(b0 ? p0.x * v.x : 0.0f, b1 ? p0.y * v.y : 0.0f);
        w1 = make_float2(b2 ? p1.x * v.z : 0.0f, b3 ? p1.y * v.w : 0.0f);
      } else {
        w0 = __fmul2_rn(p0, make_float2(v.x, v.y));
        w1 = __fmul2_rn(p1, make_float2(v.z, v.w));
      }
      sum0 = __fadd2_rn(sum0, p0);
      sum1 = __fadd2_rn(sum1, p1);
      w[2 * i] = half2_bits(w0.x, w0.y);
      w[2 * i + 1] = half2_bits(w1.x, w1.y);
    }
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(s_addr + 16 * c),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
        "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
        : "memory");
  }
  return (sum0.x + sum0.y) + (sum1.x + sum1.y);
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kfull[i], kConverters);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.vfull[i], kConverters);
      mbar_init(&sh.vempty[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i], 128);
      mbar_init(&sh.ofull[i], 1);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(&sh.scfull[i], kConverters);
    mbar_init(&sh.qfull, kSoftmax);
    mbar_init(&sh.drain, 1);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
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
    const int w = warp - 8, chunks = hd >> 4;  // 16-byte pieces of a head
    const int sub = lane / C::LANES, piece = lane % C::LANES;
    const bool swap = (piece & 4) != 0;        // (lanes of a row write both halves of their pieces in turn: no bank twice)
    const bool loads = piece < chunks;
    auto put = [&](uint8_t* base, const uint4 (&raw)[C::LOADS]) {
#pragma unroll
      for (int i = 0; i < C::LOADS; ++i) {
        const int row = w * C::WARP_ROWS + i * (32 / C::LANES) + sub;
        uint4 lo, hi;
        widen16(raw[i], lo, hi);
        uint8_t* at = base + (piece >> 2) * (C::BN * 128) + row * 128;
        const int c0 = ((2 * piece) & 7) ^ (row & 7), c1 = ((2 * piece + 1) & 7) ^ (row & 7);
        if (loads) {
          *reinterpret_cast<uint4*>(at + (swap ? c1 : c0) * 16) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(at + (swap ? c0 : c1) * 16) = swap ? lo : hi;
        }
      }
    };
    int g = 0;
    for (Walk<C> k(a, sh); ok && k.next();) {
      const int* table = a.block_table + static_cast<long long>(k.b) * a.ld_table;
      const int stop = k.s.len - k.s.fresh + (k.w.row + k.w.rows - 1) / group + 1;  // tokens the unit's last row sees
      for (int t = k.t0; t < k.t1; ++t, ++g) {
        const int st = g & 1, ring = g % kRing;
        const int row = w * C::WARP_ROWS + lane;
        const int j = (k.w.tile0 + t) * C::BN + row;
        long long at = -1;
        if (lane < C::WARP_ROWS && j < stop) {
          const int blk = j / a.block_size;
          const int page = __ldg(table + blk);
          const long long slot = static_cast<long long>(page) * a.block_size + (j - blk * a.block_size);
          if (page < 0 || slot >= a.num_slots) latch_bad_index(a.status);
          else at = slot * a.kv_heads + k.head;
        }
        uint4 kr[C::LOADS], vr[C::LOADS];
#pragma unroll
        for (int i = 0; i < C::LOADS; ++i) {
          const long long r = __shfl_sync(0xFFFFFFFFu, at, i * (32 / C::LANES) + sub);
          kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
          if (r >= 0 && loads) {
            kr[i] = __ldg(reinterpret_cast<const uint4*>(a.k_cache + r * hd) + piece);
            vr[i] = __ldg(reinterpret_cast<const uint4*>(a.v_cache + r * hd) + piece);
          }
        }
        const float ks = at >= 0 ? __ldg(a.k_scale + at) : 0.0f, vs = at >= 0 ? __ldg(a.v_scale + at) : 0.0f;
        // (a scale that is no number: a range that no tile's scales keep to)
        const float va = fabsf(vs), vfin = va < INFINITY ? va : 0.0f;
        const float top = warp_fmax(at >= 0 ? va < INFINITY ? va : FLT_MAX : 0.0f);
        const float low = -warp_fmax(at >= 0 ? -vfin : -INFINITY);
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, at >= 0);
        if (g >= 2) ok = wait_phase(&sh.kempty[st], ((g >> 1) & 1) ^ 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane < C::WARP_ROWS) {
          sh.ks[ring][row] = ks;
          sh.vs[ring][row] = vs;
        }
        if (lane == 0) {
          sh.vmax[ring][w] = top;
          sh.vmin[ring][w] = low;
          if (C::WARP_ROWS == 32) sh.valid[ring][w] = there;
          else reinterpret_cast<uint16_t*>(&sh.valid[ring][0])[w] = static_cast<uint16_t>(there);
        }
        put(smem + C::OFF_K + st * C::KV_BYTES, kr);
        fence_proxy_async_smem();
        mbar_arrive(&sh.scfull[ring]);
        mbar_arrive(&sh.kfull[st]);
        if (g >= 2) ok = wait_phase(&sh.vempty[st], ((g >> 1) & 1) ^ 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        put(smem + C::OFF_V + st * C::KV_BYTES, vr);
        fence_proxy_async_smem();
        mbar_arrive(&sh.vfull[st]);
      }
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = umma_idesc_f32acc(0, 0, 128, C::BN);
      const uint32_t id_o = umma_idesc_f32acc(0, 0, 128, hd) | (1u << 16);  // B (values) transposed
      const uint32_t s_q = smem_addr(smem), s_k = s_q + C::OFF_K, s_v = s_q + C::OFF_V;
      const int ksteps = hd >> 4;
      int g = 0, seg = 0;
      uint32_t weights[2] = {0, 0};  // tiles of weights taken from each score buffer
      auto scores = [&](int tile, int buf, int st) {
        for (int kk = 0; kk < ksteps; ++kk)
          umma_f16(tmem + buf * C::TM_S, umma_desc_sw128(s_q + tile * C::Q_BYTES + (kk >> 2) * (128 * 128) + (kk & 3) * 32),
                   umma_desc_sw128(s_k + st * C::KV_BYTES + (kk >> 2) * (C::BN * 128) + (kk & 3) * 32), id_s, kk != 0);
        umma_commit(&sh.sfull[buf]);
      };
      auto outputs = [&](int tile, int buf, int st, bool first) {
        if (!wait_phase(&sh.pfull[buf], weights[buf] & 1, a.status)) return false;
        ++weights[buf];
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < C::BN / 16; ++kk)
          umma_f16_tmem_a(tmem + C::TM_O + tile * 64 * PANELS, tmem + buf * C::TM_S + kk * 8,
                          desc_transposed(s_v + st * C::KV_BYTES + kk * 16 * 128, C::BN * 128), id_o, !first || kk != 0);
        umma_commit(&sh.ofull[tile]);
        return true;
      };
      auto keys = [&](int i) {
        if (!wait_phase(&sh.kfull[i & 1], (i >> 1) & 1, a.status)) return false;
        tc_fence_after();
        return true;
      };
      auto values = [&](int i) { return wait_phase(&sh.vfull[i & 1], (i >> 1) & 1, a.status); };
      for (Walk<C> k(a, sh); ok && k.next(); ++seg) {
        ok = wait_phase(&sh.qfull, seg & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        const int n = k.t1 - k.t0;
        const bool two = k.w.rows > 128;
        for (int i = 0; i <= n && ok; ++i) {
          if (i < n && !keys(g + i)) ok = false;
          if (ok && i > 0 && !values(g + i - 1)) ok = false;
          if (!ok) break;
          if (two) {  // scores of tile i take the place of the weights of tile i - 1
#pragma unroll
            for (int q = 0; q < C::TILES; ++q) {
              if (ok && i > 0) ok = outputs(q, q, (g + i - 1) & 1, i == 1);
              if (ok && i < n) scores(q, q, (g + i) & 1);
            }
            if (ok && i < n) umma_commit(&sh.kempty[(g + i) & 1]);
          } else {
            if (i < n) {
              scores(0, i & 1, (g + i) & 1);
              umma_commit(&sh.kempty[(g + i) & 1]);
            }
            if (i > 0) ok = outputs(0, (i - 1) & 1, (g + i - 1) & 1, i == 1);
          }
          if (!ok) break;
          if (i > 0) umma_commit(&sh.vempty[(g + i - 1) & 1]);
        }
        g += n;
      }
      umma_commit(&sh.drain);
      wait_drain(&sh.drain, 0, a.status);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax: a row a thread
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // tokens before the first position see nothing
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const Seq s = seq_of(a, b);
      const int none = min(s.fresh, s.fresh - s.len);
      for (int i = 0; i < none; ++i) {
        const long long row = s.row0 + i;
        for (int c = tid; c < a.q_heads * hd; c += kSoftmax) a.out[row * a.ldo + c] = __float2bfloat16_rn(0.0f);
        if (a.lse)
          for (int c = tid; c < a.q_heads; c += kSoftmax) a.lse[row * a.q_heads + c] = -INFINITY;
      }
    }
    int g = 0, seg = 0;
    uint32_t before[2] = {0, 0}, done = 0;  // tiles that went through each score buffer before this segment, outputs of this row tile
    for (Walk<C> k(a, sh); k.next(); ++seg) {
      const int n = k.t1 - k.t0;
      const bool two = k.w.rows > 128, active = tile == 0 || two;
      const int pair = k.w.row + tile * 128 + r;  // this thread's (token, head)
      const bool mine = tile * 128 + r < k.w.rows;
      const int token = pair / group, qh = k.head * group + (pair - token * group);
      const int pos = k.s.len - k.s.fresh + token;
      float f = 0.0f;
      if (ok && active) {
        // this row's queries as fp16
        const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(k.s.row0 + token) * a.ldq +
                                                          static_cast<long long>(qh) * hd);
        float top = 0.0f;
        const int vecs = hd >> 3;
        if (mine)
          for (int i = 0; i < vecs; ++i) {
            const uint4 u = __ldg(src + i);
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(uw[e] << 16)), fabsf(__uint_as_float(uw[e] & 0xFFFF0000u))));
          }
        // (a row below 2^-106: fewer bits, nothing to score)
        const int up = min(14 - exponent(top), 120);
        const float f1 = a.scale < 0.0f ? -pow2(up / 2) : pow2(up / 2), f2 = pow2(up - up / 2);
        uint8_t* dst = smem + tile * C::Q_BYTES + r * 128;
        for (int i = 0; i < vecs; ++i) {
          const uint4 u = mine ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = half2_bits(__uint_as_float(uw[e] << 16) * f1 * f2, __uint_as_float(uw[e] & 0xFFFF0000u) * f1 * f2);
          *reinterpret_cast<uint4*>(dst + (i >> 3) * (128 * 128) + (((i & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        // raw score x the key's scale x this = score in log2 units
        f = fabsf(a.scale) * 1.44269504088896340736f / fabsf(f1) / f2;
        fence_proxy_async_smem();
      }
      if (ok) {
        tc_fence_before();
        mbar_arrive(&sh.qfull);
      }
      float R = -INFINITY, l = 0.0f, most = -INFINITY, heavy = -INFINITY;  // largest x, bound on log2 of the largest p vs
      if (active) {
        for (int i = 0; i < n && ok; ++i) {
          const int buf = two ? tile : i & 1, ring = (g + i) % kRing;
          ok = wait_phase(&sh.scfull[ring], ((g + i) / kRing) & 1, a.status) &&
               wait_phase(&sh.sfull[buf], (before[buf] + (two ? i : i >> 1)) & 1, a.status);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t s_addr = lane_base + buf * C::TM_S;
          const float *ks = sh.ks[ring], *vs = sh.vs[ring];
          const uint32_t* valid = sh.valid[ring];
          // columns of this tile that the row sees (a row past the unit's: all, of a query of zeros)
          const int j0 = (k.w.tile0 + k.t0 + i) * C::BN;
          Seen seen = {0, C::BN};
          if (mine) seen = {a.window > 0 ? pos - a.window + 1 - j0 : 0, pos + 1 - j0};
          uint32_t all = valid[0] & (C::BN > 32 ? valid[1] : ~0u);
          if (C::BN == 128) all &= valid[2] & valid[3];
          const bool mask = __any_sync(0xFFFFFFFFu, (mine && (seen.lo > 0 || seen.hi < C::BN)) || all != 0xFFFFFFFFu);
          const float vtop = fmaxf(fmaxf(sh.vmax[ring][0], sh.vmax[ring][1]), fmaxf(sh.vmax[ring][2], sh.vmax[ring][3]));
          const float vlow = fminf(fminf(sh.vmin[ring][0], sh.vmin[ring][1]), fminf(sh.vmin[ring][2], sh.vmin[ring][3]));
          float tm = mask ? tile_max<C::BN, true>(s_addr, ks, seen, valid) : tile_max<C::BN, false>(s_addr, ks, seen, valid);
          if (tm > -INFINITY) tm = __fmul_rn(tm, f);
          most = fmaxf(most, tm);
          const bool apart = !(vtop <= vlow * 64.0f);
          if (apart) heavy = fmaxf(heavy, tile_max_weight<C::BN>(s_addr, ks, vs, f, seen, valid));
          else heavy = fmaxf(heavy, tm + lg2(vtop));
          const bool wide = __any_sync(0xFFFFFFFFu, fabsf(most) >= kWide && most > -INFINITY);
          // the reference, where it has to move
          const bool move = most > -INFINITY && (!(R > -INFINITY) || !(heavy - R < 15.0f) || !(most - R < 112.0f));
          float back = 1.0f;
          if (move) {
            const float to = fabsf(most) < kWide ? fmaxf(heavy - 11.5f, most - 100.0f) : most;
            back = to > R ? ex2(R - to) : 1.0f;
            R = fmaxf(R, to);
            l *= back;
          }
          // the tile's weights are only handed over once the outputs of the one before are there: a wait by parity
          // must not be two phases behind
          if (i > 0) {
            ok = wait_phase(&sh.ofull[tile], (done - 1) & 1, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
          }
          if (i > 0 && __any_sync(0xFFFFFFFFu, back != 1.0f)) {
            tc_fence_after();
            const uint32_t o_addr = lane_base + C::TM_O + tile * 64 * PANELS;
            for (int c = 0; c < hd; c += 16) {
              float o[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                  "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                  "tcgen05.wait::ld.sync.aligned;"
                  : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]), "=f"(o[8]),
                    "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
                  : "r"(o_addr + c)
                  : "memory");
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= back;
              asm volatile(
                  "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                  "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(o_addr + c),
                  "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7]), "f"(o[8]), "f"(o[9]),
                  "f"(o[10]), "f"(o[11]), "f"(o[12]), "f"(o[13]), "f"(o[14]), "f"(o[15])
                  : "memory");
            }
          }
          if (wide) l += tile_weights<C::BN, true, true>(s_addr, ks, vs, f, R, seen, valid);
          else if (mask) l += tile_weights<C::BN, true, false>(s_addr, ks, vs, f, R, seen, valid);
          else l += tile_weights<C::BN, false, false>(s_addr, ks, vs, f, R, seen, valid);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sh.pfull[buf]);
          ++done;
        }
        if (ok) ok = wait_phase(&sh.ofull[tile], (done - 1) & 1, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
      }
      // (the group without rows waits for the other: the score buffers' and the scales' phases that it did not watch
      // have passed when it watches them again)
      if (!two) named_barrier(1, kSoftmax);
      g += n;
      before[0] += two ? n : (n + 1) >> 1;
      before[1] += two ? n : n >> 1;
      const bool whole = n == k.w.tiles;
      const long long orow = k.s.row0 + token;
      if (whole) {
        if (ok && active) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          __nv_bfloat16* out = a.out + orow * a.ldo + static_cast<long long>(qh) * hd;
          for (int c = 0; c < hd; c += 16) {
            float o[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                "tcgen05.wait::ld.sync.aligned;"
                : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]), "=f"(o[8]),
                  "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
                : "r"(lane_base + C::TM_O + tile * 64 * PANELS + c)
                : "memory");
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if (mine) {
              reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          if (a.lse && mine) {
            const int e = exponent(l);  // (the reference may lie far from the largest score)
            a.lse[orow * a.q_heads + qh] = l > 0.0f ? ((R + static_cast<float>(e)) + log2f(l * pow2(-e))) * 0.693147180559945309f : -INFINITY;
          }
        }
        tc_fence_before();
        continue;
      }
      // part of a unit: (reference, sum, outputs) into the workspace
      const int part = 2 * static_cast<int>(blockIdx.x) + (k.t0 == 0 ? 1 : 0);
      if (ok && active) {
        float* dst = p.partial + static_cast<long long>(part) * C::ROWS * hd + (tile * 128 + r) * 4;
        for (int c = 0; c < hd; c += 16) {
          float o[16];
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
              "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
              "tcgen05.wait::ld.sync.aligned;"
              : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]), "=f"(o[8]),
                "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
              : "r"(lane_base + C::TM_O + tile * 64 * PANELS + c)
              : "memory");
          if (mine)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(reinterpret_cast<float4*>(dst + static_cast<long long>(c / 4 + e) * C::ROWS * 4),
                     make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
        }
        if (mine) __stcg(reinterpret_cast<float2*>(p.partial_ml + (static_cast<long long>(part) * C::ROWS + tile * 128 + r) * 2), make_float2(R, l));
      }
      tc_fence_before();
      __threadfence();
      if (any_of(!ok)) {  // nothing is counted or joined
        ok = false;
        continue;
      }
      const int r0 = k.range_of(0), r1 = k.range_of(k.w.tiles - 1);
      if (tid == 0) {
        sh.last = atomicAdd(p.counter + r0, 1u) == static_cast<unsigned>(r1 - r0);
        if (sh.last) p.counter[r0] = 0;  // ready for the next call
        __threadfence();
      }
      named_barrier(1, kSoftmax);
      const bool join = sh.last != 0;
      if (join) {
        // the parts in order of their ranges; a thread takes 4 columns of a row
        const int rows = k.w.rows;
        for (int it = tid; it < rows * (hd >> 2); it += kSoftmax) {
          const int c4 = it / rows, rr = it - c4 * rows;
          float m = -INFINITY, sum = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int x = r0; x <= r1; ++x) {
            const long long q = 2LL * x + (x == r0 ? 1 : 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.partial_ml + (q * C::ROWS + rr) * 2));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.partial + q * C::ROWS * hd + (static_cast<long long>(c4) * C::ROWS + rr) * 4));
            const float to = fmaxf(m, ml.x);
            const float f0 = m > -INFINITY ? ex2(m - to) : 0.0f, f1 = ml.x > -INFINITY ? ex2(ml.x - to) : 0.0f;
            m = to;
            sum = sum * f0 + ml.y * f1;
            o.x = o.x * f0 + v.x * f1;
            o.y = o.y * f0 + v.y * f1;
            o.z = o.z * f0 + v.z * f1;
            o.w = o.w * f0 + v.w * f1;
          }
          const int pr = k.w.row + rr, tok = pr / group, h = k.head * group + (pr - tok * group);
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(a.out + static_cast<long long>(k.s.row0 + tok) * a.ldo + static_cast<long long>(h) * hd + 4 * c4) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
          if (a.lse && c4 == 0) {
            const int e = exponent(sum);
            a.lse[static_cast<long long>(k.s.row0 + tok) * a.q_heads + h] =
                sum > 0.0f ? ((m + static_cast<float>(e)) + log2f(sum * pow2(-e))) * 0.693147180559945309f : -INFINITY;
          }
        }
        named_barrier(1, kSoftmax);  // (sh.last is read before it is written again)
      }
    }
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
