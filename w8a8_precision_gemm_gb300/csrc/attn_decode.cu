// attn_decode.cu -- attention of one new token per sequence over the paged FP8
// key/value cache that qurl_kv_cache_quant fills.
//
//   s_j = scale * ks_j * sum_d q_d k_jd,   p = softmax(s),   o_d = sum_j p_j vs_j v_jd
//
// over the cached tokens j the sequence sees (its last `window` ones, or all).
//
// Bound by HBM: a cached token is read once per KV head, 2 head_dim + 8 bytes
// for 4 head_dim operations per query head of the group, so every byte is used
// about 2 x group times -- too often for the fp32 pipes to keep up with HBM once
// the codes also have to be converted, and nothing for the tensor cores.  They
// read the e4m3 codes as they lie in the cache (kind::f8f6f4, no conversion);
// the other operand is split into e4m3 pieces that add up to it:
//   * q, scaled by a power of two so that its largest value is in [128, 256):
//     q = hi + lo / 16 with hi the e4m3 rounding, lo that of 16 (q - hi).  A bf16
//     has 8 significant bits and each piece 4, so values within 2^-13 of the
//     largest are exact and smaller ones off by at most 2^-21 of the largest (half
//     lo's smallest step, 2^-14, beside 128).
//   * x_j = p_j vs_j, scaled by a power of two so that it lies below 256, in three
//     pieces: 12 significant bits, 2^-12 relative, or an error of 2^-18 where the
//     last piece underflows (2^-11 in all the tile).  The token that a head attends may
//     have a far smaller value scale than its neighbours: while the scales lie within
//     2^6 of each other, one power keeps them in [2, 256); a tile with others in it
//     takes p_j against a reference below the largest score, so that each head's
//     largest p_j vs_j is in [128, 256), from one more maximum a head.
// Products are exact and sums fp32.  Keys and values are the A operand (M = 128
// tokens for the scores, M = 128 dimensions for the output, the value tile read
// transposed), the pieces of all the group's heads the N = 16 or 32 columns of
// B: one MMA chain per tile serves every query head of the group.
//
// A CTA works on 128-token tiles: four loader warps gather the tile's rows, each
// page's slot looked up on the way (cp.async, 16 bytes a lane, into the 128-byte
// swizzled layout; rows of tokens that do not count are zero-filled), one thread
// issues the MMAs, four warps hold one token a lane for the softmax and one
// output dimension a lane for the sums.  Each tile has its own maximum (scores
// never need a second look); its output columns are rescaled into fp32
// accumulators in registers when they are added.
//
// The tiles of all sequences in a row are cut into R equal ranges, whatever the
// lengths; (range, KV head) is a unit of work, heads innermost, so that the CTAs
// that run together share the cache lines that hold several heads' scales.  A
// sequence that ends up in several ranges leaves unnormalised partial sums in
// the workspace, and the unit that finishes it last (a counter per range and
// head) joins them in range order (a sequence over many ranges in groups): one
// launch, the same result every run.
//
// Measured on the device, 40 query heads over 8 KV heads of 128: 64 sequences of 256
// to 8192 tokens (about 590 MB) 107 to 120 us (other lengths, other times), 5.2 TB/s; 4
// of 98 k to 131 k tokens (1.0 GB) 172 to 176 us, 5.8 TB/s, 0.85 of the copy rate; value
// scales spread over 2^10 in every tile 2 to 4% more.  The first tiles are there after
// 5 us, then the cache streams at 6.3 TB/s; equal units end up to 16 us apart (whoever
// ends first leaves its share of HBM to the others), the joins take 4 to 5 us more.  64
// query heads over 4 (two parts, each of which reads the keys and values): 126 us of
// 43 at the copy rate.  One sequence of 300 tokens, 28 heads over 4: 10.8 us, of which
// 3.6 to the first tile (lengths, table, rows: one after the other), 1.3 a tile,
// nothing to join, 2.5 to the end.
// Taking units from a shared counter in shorter ranges was slower (more joins).
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

constexpr int kTile = 128;      // tokens per tile
constexpr int kSoftmax = 128;   // threads 0..127: softmax and sums (TMEM lanes)
constexpr int kLoaders = 128;   // threads 128..255
constexpr int kThreads = kSoftmax + kLoaders + 32;  // and the MMA warp
// Tiles per range at least: a tile more costs a unit about 0.75 us, joining partial sums about 3.
constexpr int kMinTiles = 4;
constexpr int kJoin = 12;        // partial sums that one unit joins; of more, groups of that many are joined first
constexpr float kNone = -FLT_MAX;  // a maximum over no tokens: no score lies below it

constexpr int round16(int n) { return (n + 15) / 16 * 16; }

// G: query heads per unit at most (a KV head's group is cut into equal parts
// of at most that many); PANELS: 128-column panels of a head.  Two CTAs share
// an SM with one panel.
template <int G_, int PANELS_>
struct AttnCfg {
  static constexpr int G = G_, PANELS = PANELS_;
  static constexpr int NS = round16(2 * G);  // B rows of the score MMA: hi and lo of each head
  static constexpr int NP = round16(3 * G);  // B rows of the output MMA: three pieces of each head
  static constexpr int STAGES = 3;
  static constexpr int CTAS = PANELS == 1 ? 2 : 1;
  static constexpr int PANEL = kTile * 128;
  static constexpr int OPERAND = PANELS * PANEL;  // a tile of keys, or of values
  static constexpr int QBUF = PANELS * NS * 128;
  static constexpr int OFF_V = STAGES * OPERAND;
  static constexpr int OFF_Q = 2 * STAGES * OPERAND;
  static constexpr int OFF_P = OFF_Q + STAGES * QBUF;
  static constexpr int OFF_SCALE = OFF_P + NP * 128;
  static constexpr int SMEM = OFF_SCALE + STAGES * 2 * kTile * 4 + 1024;
  static constexpr int TM_O = 2 * NS;  // TMEM: two score buffers, then the output columns of each panel
  static constexpr int TM_USED = TM_O + PANELS * NP;
  static constexpr int TM_COLS = TM_USED <= 32 ? 32 : TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128 : 256;
  static_assert(CTAS * (SMEM + 3 * 1024) <= 228 * 1024, "shared memory per SM");
  static_assert(QBUF % 1024 == 0 && (NP * 128) % 1024 == 0, "swizzle atoms");
};

// How the launch is cut: R ranges x heads units over the grid.
struct AttnPlan {
  int ranges;     // R
  int parts;      // equal parts of a KV head's group
  int per_part;   // query heads per part (the last may have fewer)
  int grid;
  float* partial;     // [2 R][heads][G][head_dim], then [2 R][heads][G][2] of (maximum, sum)
  unsigned* counter;  // [3][R][heads]: sequences that begin in a range; groups, see below
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_fmax(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// mbar_wait (ptx.cuh) that gives up for a timeout only: a page out of range
// latched by this kernel leaves the other sequences' results alone.
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

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    uint32_t u[32];
    tmem_ld32(taddr, u);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
  }
}

// e4m3 rounding of a pair (a in the low byte), and its values.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Barrier of the softmax threads; whether `v` holds in any of them.
__device__ __forceinline__ bool any_of(bool v) {
  int r = v ? 1 : 0;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %0, 0;\n\tbarrier.cta.red.or.pred b, 1, 128, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
      : "+r"(r)::"memory");
  return r != 0;
}

// 2^n, n in [-126, 128] (2^128: infinity).
__device__ __forceinline__ float pow2(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }
// floor(log2 x) of a normal x > 0 (-127 for zero and subnormals).
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));  // (subnormal scales too)
  return y;
}

// Matrix descriptor of a tile whose rows are the MMA's K (tokens) and whose 128
// contiguous bytes are its M (dimensions), 128-byte swizzle: groups of 8 rows
// lie 1024 bytes apart (the stride between groups along K; M fills one
// swizzle row, so no other stride is used).
__device__ __forceinline__ uint64_t desc_transposed(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1024u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Tokens a sequence sees: [first, len), and their tiles.
struct Span {
  int first, len, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  const long long room = static_cast<long long>(a.max_blocks) * a.block_size;
  int len = __ldg(a.seq_lens + b);
  len = len < 0 ? 0 : static_cast<int>(len < room ? len : room);
  const int first = a.window > 0 && len > a.window ? len - a.window : 0;
  return {first, len, (len - first + kTile - 1) / kTile};
}

// The power of two that takes scales below 2^(top + 1) below 256.
__device__ __forceinline__ int scale_power(int top) { return min(max(7 - top, -120), 120); }
__device__ __forceinline__ float most(const float (&v)[4]) {
  const float4 q = *reinterpret_cast<const float4*>(v);
  return fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w));
}

// A tile whose value scales lie far apart, by the softmax threads behind the vote that found it: takes each head's
// score maximum in `red` to a reference 2^e below it, such that its largest p vs lies in [128, 256) (to the rounding
// of its logarithm; scores so large that a sum with log2 vs loses it stay as they are).  Sums and outputs go by the
// reference, whatever it is.  Returns the power that bounds the tile's scales with one to spare, or kFailed.  (Called,
// not inlined: inlined it cost the other tiles 2%.)
constexpr int kFailed = 1 << 20;
template <int G>
struct PerHead {
  float v[G];
};
template <int G>
__device__ __noinline__ int lower_references(float (*red)[4], PerHead<G> x, float va, bool got) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const float lv = lg2(va), vw = warp_fmax(va);
  if ((tid & 31) == 0) red[2 * G][warp] = vw;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float yw = warp_fmax(x.v[h] + lv);
    if ((tid & 31) == 0) red[G + h][warp] = yw;
  }
  if (any_of(!got)) return kFailed;
  const int top = exponent(most(red[2 * G])) + 1;
  if (tid < G) {
    const float mx = most(red[tid]);
    if (fabsf(mx) < 0x1p22f) {
      const int e = 7 - scale_power(top) - __float2int_rd(fmaxf(most(red[G + tid]) - mx, -200.0f));
      *reinterpret_cast<float4*>(red[tid]) =
          make_float4(mx - static_cast<float>(min(max(e, 0), 100)), -INFINITY, -INFINITY, -INFINITY);
    }
  }
  named_barrier(1, kSoftmax);
  return top;
}

struct Shared {
  uint64_t full[3], empty[3];  // a stage's rows have landed / its MMAs have read them
  uint64_t sfull[2];           // scores of a tile are in TMEM
  uint64_t pfull, ofull;       // weights of a tile are in shared memory / its output columns in TMEM
  uint64_t drain;
  uint32_t tmem;
  int chunk;                             // sequences per thread of the scan
  int ranges;                            // ranges in use: the first `longer` have base + 1 tiles, the others base
  long long base, longer;
  long long tiles_before[kSoftmax + 1];  // tiles before each thread's chunk
  uint32_t valid[3][4];                  // tokens of a stage that count
  float qfac[3][16];                     // per head: what turns a raw score into log2 units
  // per-warp maxima of a tile (double-buffered): scores; where scales lie apart, log2 of the weights, and the scales
  alignas(16) float red[2][8 + 8 + 1][4];
  alignas(16) float sum[16][4];
  int last;
  int failed;  // a wait for an output has run out
};

// a / b of small results: 32-bit where both fit (64-bit divisions took a microsecond of the call's start).
__device__ __forceinline__ int quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
  return static_cast<int>(a / b);
}

// Walks the segments (one sequence's tiles inside one range) of the CTA's
// units in order; every role walks the same ones.
struct Walk {
  const AttnArgs& a;
  const AttnPlan& p;
  const Shared& sh;
  long long total;  // tiles of all sequences
  int unit, heads;
  // current segment
  int head, range, b;
  Span s;
  int t0, t1;              // tiles of the sequence in this segment
  long long seq_tile0;     // first tile of the sequence in the row of all tiles
  long long at, range_end;

  __device__ Walk(const AttnArgs& a_, const AttnPlan& p_, const Shared& sh_)
      : a(a_), p(p_), sh(sh_), total(sh_.tiles_before[kSoftmax]), unit(blockIdx.x), heads(a_.kv_heads * p_.parts) {
    at = range_end = 0;
    b = 0;
    s = {0, 0, 0};
    t0 = t1 = 0;
    seq_tile0 = 0;
    head = range = 0;
    unit -= gridDim.x;
  }

  __device__ long long start_of(int r) const { return r * sh.base + (r < sh.longer ? r : sh.longer); }

  __device__ bool next() {
    if (at < range_end) {  // the rest of the range: the next sequence that has tiles
      seq_tile0 += s.tiles;
      do {
        ++b;
        s = span_of(a, b);
      } while (s.tiles == 0);
    } else {
      unit += gridDim.x;
      if (unit >= sh.ranges * heads) return false;
      range = unit / heads;
      head = unit - range * heads;
      at = start_of(range);
      range_end = start_of(range + 1);
      int lo = 0, hi = kSoftmax;  // the chunk of sequences that holds tile `at`
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.tiles_before[mid] <= at) lo = mid;
        else hi = mid;
      }
      b = lo * sh.chunk;
      seq_tile0 = sh.tiles_before[lo];
      s = span_of(a, b);
      while (seq_tile0 + s.tiles <= at) {
        seq_tile0 += s.tiles;
        ++b;
        s = span_of(a, b);
      }
    }
    t0 = static_cast<int>(at - seq_tile0);
    const long long end = range_end - seq_tile0;
    t1 = end < s.tiles ? static_cast<int>(end) : s.tiles;
    at = seq_tile0 + t1;
    return true;
  }
  // the range that holds tile t of the row of all tiles
  __device__ int range_of(long long t) const {
    const long long over = t - sh.longer * (sh.base + 1);
    return over < 0 ? quotient(t, sh.base + 1) : static_cast<int>(sh.longer) + quotient(over, sh.base);
  }
};

template <int G, int PANELS>
__global__ void __launch_bounds__(kThreads, AttnCfg<G, PANELS>::CTAS)
    kv_attn_decode_kernel(const AttnArgs a, const AttnPlan p) {
  using C = AttnCfg<G, PANELS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_k = smem_addr(smem), s_v = s_k + C::OFF_V, s_q = s_k + C::OFF_Q, s_p = s_k + C::OFF_P;
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE);  // [STAGES][keys, values][kTile]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hd = a.head_dim;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&sh.full[i], 2 * kLoaders);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.sfull[0], 1);
    mbar_init(&sh.sfull[1], 1);
    mbar_init(&sh.pfull, kSoftmax);
    mbar_init(&sh.ofull, 1);
    mbar_init(&sh.drain, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&sh.tmem, C::TM_COLS);
    tmem_relinquish();
  }
  // head_dim an odd multiple of 16: the MMA's last 32 columns reach past the head, into bytes that no copy
  // writes; they are zero in keys and queries (never NaN)
  if (hd & 16) {
    const int col = hd & 127, panel = hd >> 7;
    for (int i = tid; i < C::STAGES * kTile; i += kThreads) {
      const int st = i / kTile, r = i % kTile;
      *reinterpret_cast<uint4*>(smem + st * C::OPERAND + panel * C::PANEL + r * 128 + (col ^ ((r & 7) << 4))) = make_uint4(0, 0, 0, 0);
    }
    for (int i = tid; i < C::STAGES * C::NS; i += kThreads) {
      const int st = i / C::NS, r = i % C::NS;
      *reinterpret_cast<uint4*>(smem + C::OFF_Q + st * C::QBUF + panel * C::NS * 128 + r * 128 + (col ^ ((r & 7) << 4))) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_wait();
  griddep_launch_dependents();

  // tiles before each chunk of sequences
  {
    const int chunk = (a.B + kSoftmax - 1) / kSoftmax;
    if (tid < kSoftmax) {
      const long long room = static_cast<long long>(a.max_blocks) * a.block_size;
      long long n = 0;
      for (int i = 0; i < chunk; ++i) {
        const int b = tid * chunk + i;
        if (b >= a.B) break;
        n += span_of(a, b).tiles;
        if (blockIdx.x == 0 && __ldg(a.seq_lens + b) > room) latch_bad_index(a.status);
      }
      long long c = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, c, o);
        if (lane >= o) c += v;
      }
      sh.tiles_before[tid + 1] = c;
    }
    if (tid == 0) {
      sh.failed = 0;
      sh.tiles_before[0] = 0;
      sh.chunk = chunk;
    }
    __syncthreads();
    if (tid < kSoftmax) {  // (the warp sums are read before any is changed)
      long long add = 0;
      for (int w = 0; w < warp; ++w) add += sh.tiles_before[32 * (w + 1)];
      named_barrier(1, kSoftmax);
      add += sh.tiles_before[tid + 1];
      sh.tiles_before[tid + 1] = add;
      if (tid == kSoftmax - 1) {  // all tiles
        const long long want = (add + kMinTiles - 1) / kMinTiles;
        sh.ranges = static_cast<int>(want < p.ranges ? want : p.ranges);
        if (sh.ranges > 0) {
          const long long base = (add >> 32) == 0 ? static_cast<uint32_t>(add) / static_cast<uint32_t>(sh.ranges) : add / sh.ranges;
          sh.base = base;
          sh.longer = add - base * sh.ranges;
        }
      }
    }
    __syncthreads();
  }

  const int group = a.q_heads / a.kv_heads;
  bool ok = true;
  if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ loaders: lane = token row for the lookups
    const int w = warp - 4;
    const int chunks = hd >> 4;                // 16-byte pieces of a head
    const int sub = lane >> 3, piece = lane & 7;
    int g = 0, seg = 0;
    for (Walk k(a, p, sh); ok && k.next(); ++seg) {
      const int kvh = k.head / p.parts, part = k.head - kvh * p.parts;
      const int h0 = part * p.per_part, nh = min(p.per_part, group - h0);
      const int* table = a.block_table + static_cast<long long>(k.b) * a.ld_table;
      for (int t = k.t0; t < k.t1; ++t, ++g) {
        const int st = g % C::STAGES;
        // this lane's token
        const int j = k.s.first + t * kTile + w * 32 + lane;
        long long at = -1;
        if (j < k.s.len) {
          const int blk = j / a.block_size;
          const int page = __ldg(table + blk);
          const long long slot = static_cast<long long>(page) * a.block_size + (j - blk * a.block_size);
          if (page < 0 || slot >= a.num_slots) latch_bad_index(a.status);
          else at = slot * a.kv_heads + kvh;
        }
        if (g >= C::STAGES && !wait_phase(&sh.empty[st], ((g / C::STAGES) & 1) ^ 1, a.status)) ok = false;
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, at >= 0);
        if (lane == 0) sh.valid[st][w] = mask;
        // a new segment's queries (warp w takes heads w and w + 4, a lane 8 of a head's dimensions) are read while
        // the rows are gathered
        uint4 qu[2] = {};
        const __nv_bfloat16* qsrc = a.q + static_cast<long long>(k.b) * a.ldq + static_cast<long long>(kvh * group + h0) * hd;
        if (t == k.t0 && lane * 8 < hd) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (w + 4 * i < nh) qu[i] = __ldg(reinterpret_cast<const uint4*>(qsrc + static_cast<long long>(w + 4 * i) * hd) + lane);
        }
        {
          const uint32_t n = at >= 0 ? 4 : 0;
          const long long i = at >= 0 ? at : 0;
          const uint32_t d = smem_addr(scales + st * 2 * kTile + w * 32 + lane);
          cp_async4(d, a.k_scale + i, n);
          cp_async4(d + kTile * 4, a.v_scale + i, n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + sub;
          const long long rat = __shfl_sync(0xFFFFFFFFu, at, r);
          const uint32_t n = rat >= 0 ? 16 : 0;
          const long long off = rat >= 0 ? rat * hd : 0;
          const int row = w * 32 + r;
#pragma unroll
          for (int q = 0; q < PANELS; ++q) {
            const int c = q * 8 + piece;
            if (c < chunks) {
              const uint32_t d = st * C::OPERAND + q * C::PANEL + row * 128 + ((piece ^ (row & 7)) << 4);
              cp_async16(s_k + d, a.k_cache + off + c * 16, n);
              cp_async16(s_v + d, a.v_cache + off + c * 16, n);
            }
          }
        }
        cp_async_arrive(&sh.full[st]);
        if (t == k.t0) {
          const int qb = seg % C::STAGES;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = w + 4 * i;
            if (h >= nh) break;
            float x[8];
            const uint32_t uw[4] = {qu[i].x, qu[i].y, qu[i].z, qu[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = __uint_as_float(uw[e] << 16);
              x[2 * e + 1] = __uint_as_float(uw[e] & 0xFFFF0000u);
            }
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
            m = warp_fmax(m);
            const int up = min(7 - exponent(m), 120);  // (a query of less than 2^-113: fewer bits, nothing to score)
            const float f1 = pow2(up / 2), f2 = pow2(up - up / 2);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = x[2 * e] * f1 * f2, y1 = x[2 * e + 1] * f1 * f2;
              hi[e] = e4m3x2(y0, y1);
              const float2 v = e4m3x2_value(hi[e]);
              lo[e] = e4m3x2((y0 - v.x) * 16.0f, (y1 - v.y) * 16.0f);
            }
            if (lane * 8 < hd) {
              const int q = lane >> 4, byte = (lane & 15) * 8;
              uint8_t* base = smem + C::OFF_Q + qb * C::QBUF + q * C::NS * 128;
              const int r1 = h, r2 = G + h;
              *reinterpret_cast<uint2*>(base + r1 * 128 + (byte ^ ((r1 & 7) << 4))) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
              *reinterpret_cast<uint2*>(base + r2 * 128 + (byte ^ ((r2 & 7) << 4))) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            }
            // raw score x this x the key's scale = score in log2 units
            if (lane == 0) sh.qfac[qb][h] = a.scale * 1.44269504088896340736f / f1 / f2;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(&sh.full[st]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = umma_idesc_f32acc(0, 0, 128, C::NS);
      constexpr uint32_t id_o = umma_idesc_f32acc(0, 0, 128, C::NP) | (1u << 15);  // A (values) transposed
      int g = 0, seg = 0;
      const int ksteps = (hd + 31) / 32;
      int prev = -1;  // stage of the tile whose output is still to be issued
      auto outputs = [&](int tile, int st) {
        if (!wait_phase(&sh.pfull, tile & 1, a.status)) return false;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < PANELS; ++q)
#pragma unroll
          for (int kk = 0; kk < kTile / 32; ++kk)
            umma_f8f6f4(tmem + C::TM_O + q * C::NP, desc_transposed(s_v + st * C::OPERAND + q * C::PANEL + kk * 32 * 128),
                        umma_desc_sw128(s_p + kk * 32), id_o, kk != 0);
        umma_commit(&sh.ofull);
        umma_commit(&sh.empty[st]);
        return true;
      };
      for (Walk k(a, p, sh); ok && k.next(); ++seg) {
        const uint32_t qbase = s_q + (seg % C::STAGES) * C::QBUF;
        for (int t = k.t0; t < k.t1; ++t, ++g) {
          const int st = g % C::STAGES;
          if (!wait_phase(&sh.full[st], (g / C::STAGES) & 1, a.status)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();  // the rows came by cp.async, the MMA reads them through the async proxy
          tc_fence_after();
          for (int kk = 0; kk < ksteps; ++kk) {
            const uint32_t ko = (kk >> 2) * C::PANEL + (kk & 3) * 32, qo = (kk >> 2) * C::NS * 128 + (kk & 3) * 32;
            umma_f8f6f4(tmem + (g & 1) * C::NS, umma_desc_sw128(s_k + st * C::OPERAND + ko), umma_desc_sw128(qbase + qo),
                        id_s, kk != 0);
          }
          umma_commit(&sh.sfull[g & 1]);
          if (prev >= 0 && !outputs(g - 1, prev)) {
            ok = false;
            break;
          }
          prev = st;
        }
      }
      if (ok && prev >= 0) ok = outputs(g - 1, prev);
      umma_commit(&sh.drain);
      wait_drain(&sh.drain, 0, a.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and sums
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // sequences that see nothing
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      if (span_of(a, b).tiles != 0) continue;
      __nv_bfloat16* o = a.out + static_cast<long long>(b) * a.ldo;
      for (int i = tid; i < a.q_heads * hd; i += kSoftmax) o[i] = __float2bfloat16_rn(0.0f);
      if (a.lse)
        for (int i = tid; i < a.q_heads; i += kSoftmax) a.lse[static_cast<long long>(b) * a.q_heads + i] = -INFINITY;
    }
    int g = 0, seg = 0;
    const long long part_rows = 2LL * p.ranges * a.kv_heads * p.parts;
    float* part_ml = p.partial + part_rows * G * hd;
    for (Walk k(a, p, sh); ok && k.next(); ++seg) {
      const int kvh = k.head / p.parts, part = k.head - kvh * p.parts;
      const int h0 = part * p.per_part, nh = min(p.per_part, group - h0);
      float qf[G], m[G], l[G], acc[PANELS][G];
      // value scales in [v_lo, v_hi) times 2^up lie in [2, 256)
      int up = 0;
      float v_lo = INFINITY, v_hi = INFINITY;  // (none yet)
      auto window = [&](int top) {             // scales below 2^(top + 1)
        up = scale_power(top);
        v_lo = top < -113 ? INFINITY : pow2(top - 6);  // (scales so small that 2^up would pass fp32: none)
        v_hi = pow2(min(top + 1, 128));
      };
      float mt[G], ps[G], back = 0.0f;  // the last tile's reference, this lane's weight, and scale of its output
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = mt[h] = kNone;
        l[h] = ps[h] = 0.0f;
#pragma unroll
        for (int q = 0; q < PANELS; ++q) acc[q][h] = 0.0f;
      }
      // adds tile i's output columns
      auto add_tile = [&](int i) {
        if (!wait_phase(&sh.ofull, i & 1, a.status)) sh.failed = 1;
        __syncwarp();  // (lanes leave the wait each by itself; the loads below are the warp's)
        tc_fence_after();
        float f[G], r[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float mn = fmaxf(m[h], mt[h]);
          r[h] = ex2(m[h] - mn);
          f[h] = ex2(mt[h] - mn);
          m[h] = mn;
          l[h] = l[h] * r[h] + ps[h] * f[h];
          f[h] *= back;
        }
#pragma unroll
        for (int q = 0; q < PANELS; ++q) {
          float o[C::NP];
          tmem_ld<C::NP>(lane_base + C::TM_O + q * C::NP, o);
#pragma unroll
          for (int h = 0; h < G; ++h)
            acc[q][h] = acc[q][h] * r[h] + f[h] * fmaf(o[2 * G + h], 0x1p-8f, fmaf(o[G + h], 0x1p-4f, o[h]));
        }
        tc_fence_before();
      };
      for (int t = k.t0; t < k.t1; ++t, ++g) {
        const int st = g % C::STAGES;
        const bool got = wait_phase(&sh.full[st], (g / C::STAGES) & 1, a.status) &&
                         wait_phase(&sh.sfull[g & 1], (g >> 1) & 1, a.status);
        tc_fence_after();
        if (t == k.t0) {
#pragma unroll
          for (int h = 0; h < G; ++h) qf[h] = h < nh ? sh.qfac[seg % C::STAGES][h] : 0.0f;
          // the segment's first token says where its scales may lie: 2^5 below its own to twice that
          const float v0 = fabsf(scales[st * 2 * kTile + kTile]);
          if (v0 > 0.0f) window(exponent(v0) + 1);
        }
        float s[C::NS];
        __syncwarp();
        tmem_ld<C::NS>(lane_base + (g & 1) * C::NS, s);
        const bool valid = (sh.valid[st][warp] >> lane) & 1;
        const float ks = scales[st * 2 * kTile + tid];
        const float vs = scales[st * 2 * kTile + kTile + tid];
        float (*red)[4] = sh.red[g & 1];
        float x[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          x[h] = valid && h < nh ? fmaf(s[G + h], 0x1p-4f, s[h]) * (qf[h] * ks) : -INFINITY;
          const float mw = warp_fmax(x[h]);
          if (lane == 0) red[h][warp] = mw;
        }
        const float va = fabsf(vs);
        const bool apart = any_of(!got || (valid && (va < v_lo || va >= v_hi)));  // (or a wait that ran out)
        if (__builtin_expect(apart, 0)) {
          PerHead<G> xs;
#pragma unroll
          for (int h = 0; h < G; ++h) xs.v[h] = x[h];
          const int top = lower_references<G>(red, xs, va, got);
          if (top == kFailed) {
            ok = false;
            break;
          }
          window(top);  // for the next tiles too
        }
        // the previous tile's outputs have long been summed: its weights make room
        if (t > k.t0) add_tile(g - 1);
        const float vn = vs * pow2(up);
        back = pow2(-up);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          mt[h] = fmaxf(most(red[h]), kNone);
          ps[h] = ex2(x[h] - mt[h]);
          x[h] = ps[h] * vn;
        }
        uint8_t* pt = smem + C::OFF_P + (tid & 15);
        const int ch = tid >> 4;
        auto put = [&](int row, uint32_t byte) { pt[row * 128 + ((ch ^ (row & 7)) << 4)] = static_cast<uint8_t>(byte); };
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          float y0 = x[h], y1 = h + 1 < G ? x[h + 1 < G ? h + 1 : h] : 0.0f;
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const uint32_t c = e4m3x2(y0, y1);
            put(e * G + h, c & 0xFF);
            if (h + 1 < G) put(e * G + h + 1, c >> 8);
            if (e < 2) {
              const float2 v = e4m3x2_value(c);
              y0 = (y0 - v.x) * 16.0f;
              y1 = (y1 - v.y) * 16.0f;
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.pfull);
      }
      if (!ok) break;
      add_tile(g - 1);
      // sums over the lanes (tokens)
#pragma unroll
      for (int h = 0; h < G; ++h) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], o);
        if (lane == 0) sh.sum[h][warp] = l[h];
      }
      named_barrier(1, kSoftmax);
      if (sh.failed != 0) {  // nothing is stored, joined or counted
        ok = false;
        break;
      }
#pragma unroll
      for (int h = 0; h < G; ++h) l[h] = (sh.sum[h][0] + sh.sum[h][1]) + (sh.sum[h][2] + sh.sum[h][3]);
      const int qh = kvh * group + h0;
      __nv_bfloat16* out = a.out + static_cast<long long>(k.b) * a.ldo + static_cast<long long>(qh) * hd;
      float* lse = a.lse ? a.lse + static_cast<long long>(k.b) * a.q_heads + qh : nullptr;
      const int r0 = k.range_of(k.seq_tile0), r1 = k.range_of(k.seq_tile0 + k.s.tiles - 1);
      const int n = r1 - r0 + 1;  // ranges that hold tiles of the sequence
      bool done = n == 1;
      if (!done) {
        const int heads = k.heads;
        auto row_of = [&](int range) { return (2LL * range + (range == r0 ? 1 : 0)) * heads + k.head; };
        // this thread's part of (m, l, acc) into a row of the workspace, then one more arrival on a counter;
        // whether it was the last of `of`, whose rows are then visible
        auto leave = [&](long long row, unsigned* counter, int of) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            if (h >= nh) break;
#pragma unroll
            for (int q = 0; q < PANELS; ++q)
              if (q * 128 + tid < hd) __stcg(p.partial + (row * G + h) * hd + q * 128 + tid, acc[q][h]);
            if (tid == 0) __stcg(reinterpret_cast<float2*>(part_ml + (row * G + h) * 2), make_float2(m[h], l[h]));
          }
          __threadfence();
          named_barrier(1, kSoftmax);
          if (tid == 0) {
            sh.last = atomicAdd(counter, 1u) == static_cast<unsigned>(of - 1);
            if (sh.last) *counter = 0;  // ready for the next call
            __threadfence();
          }
          named_barrier(1, kSoftmax);
          return sh.last != 0;
        };
        // (m, l, acc) = the rows of ranges from, from + step, ... (`of` of them), added in order
        auto join = [&](int from, int step, int of) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            m[h] = kNone;
            l[h] = 0.0f;
#pragma unroll
            for (int q = 0; q < PANELS; ++q) acc[q][h] = 0.0f;
          }
#pragma unroll 2
          for (int i = 0; i < of; ++i) {
            const long long row = row_of(from + i * step) * G;
            const float2 ml = lane < nh ? __ldcg(reinterpret_cast<const float2*>(part_ml + (row + lane) * 2)) : make_float2(kNone, 0.0f);
            float o[PANELS][G];
#pragma unroll
            for (int h = 0; h < G; ++h)
#pragma unroll
              for (int q = 0; q < PANELS; ++q)
                o[q][h] = h < nh && q * 128 + tid < hd ? __ldcg(p.partial + (row + h) * hd + q * 128 + tid) : 0.0f;
#pragma unroll
            for (int h = 0; h < G; ++h) {
              const float mr = __shfl_sync(0xFFFFFFFFu, ml.x, h), lr = __shfl_sync(0xFFFFFFFFu, ml.y, h);
              const float mn = fmaxf(m[h], mr), f0 = ex2(m[h] - mn), f1 = ex2(mr - mn);
              m[h] = mn;
              l[h] = l[h] * f0 + lr * f1;
#pragma unroll
              for (int q = 0; q < PANELS; ++q) acc[q][h] = acc[q][h] * f0 + o[q][h] * f1;
            }
          }
        };
        unsigned* counter = p.counter + static_cast<long long>(r0) * heads + k.head;
        const int groups = (n + kJoin - 1) / kJoin;
        if (groups == 1) {
          done = leave(row_of(k.range), counter, n);
          if (done) join(r0, 1, n);
        } else {
          const int g0 = r0 + (k.range - r0) / kJoin * kJoin, of = min(kJoin, r1 + 1 - g0);
          // (two sequences may have a group that begins in a range: the one that the range ends, the one it begins)
          const long long at = static_cast<long long>(g0 == r0 ? 2 : 1) * p.ranges + g0;
          if (leave(row_of(k.range), p.counter + at * heads + k.head, of)) {
            join(g0, 1, of);
            named_barrier(1, kSoftmax);  // every thread has read the group's rows; its first one takes their sum
            done = leave(row_of(g0), counter, groups);
            if (done) join(r0, kJoin, groups);
          }
        }
      }
      if (done) {
#pragma unroll
        for (int h = 0; h < G; ++h) {
          if (h >= nh) break;
          const float inv = l[h] > 0.0f ? 1.0f / l[h] : 0.0f;
#pragma unroll
          for (int q = 0; q < PANELS; ++q)
            if (q * 128 + tid < hd) out[static_cast<long long>(h) * hd + q * 128 + tid] = __float2bfloat16_rn(acc[q][h] * inv);
          if (lse && tid == 0) {
            const int k = exponent(l[h]);  // (the reference m may lie far below the largest score)
            lse[h] = l[h] > 0.0f ? ((m[h] + static_cast<float>(k)) + log2f(l[h] * pow2(-k))) * 0.693147180559945309f : -INFINITY;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// The workspace's counters: room for those of any layout, so that no layout's partial sums lie where another's
// counters do.  Several ranges (one needs no counter) have at most four rounds of two CTAs an SM as units, and
// each unit has three.
size_t counter_bytes(int num_sms) {
  return (static_cast<size_t>(num_sms) * 2 * 4 * 3 * sizeof(unsigned) + 255) & ~static_cast<size_t>(255);
}

// Equal parts of a group of at most 8 query heads.
constexpr int kMaxG = 8;

AttnPlan plan_attn(int q_heads, int kv_heads, int head_dim, int num_sms, size_t* bytes) {
  AttnPlan p{};
  const int group = q_heads / kv_heads;
  p.parts = (group + kMaxG - 1) / kMaxG;
  p.per_part = (group + p.parts - 1) / p.parts;
  const long long heads = static_cast<long long>(kv_heads) * p.parts;
  const long long slots = static_cast<long long>(num_sms) * (head_dim <= 128 ? 2 : 1);
  // as many ranges as fill the CTAs' first round to 97%, or the best of up to four rounds
  double best = 0.0;
  for (long long rounds = 1; rounds <= 4 && best < 0.97; ++rounds) {
    const long long r = rounds * slots / heads;
    const double fill = static_cast<double>(r * heads) / static_cast<double>(rounds * slots);
    if (fill > best) {
      best = fill;
      p.ranges = static_cast<int>(r);
    }
  }
  if (p.ranges < 1) p.ranges = 1;
  const long long units = p.ranges * heads;
  p.grid = static_cast<int>(units < slots ? units : slots);
  const int G = p.per_part <= 5 ? 5 : kMaxG;
  *bytes = counter_bytes(num_sms) + static_cast<size_t>(2 * units) * G * (head_dim + 2) * 4;
  return p;
}

template <int G, int PANELS>
cudaError_t launch_inst(const AttnArgs& a, const AttnPlan& p, cudaStream_t st) {
  using C = AttnCfg<G, PANELS>;
  auto kern = kv_attn_decode_kernel<G, PANELS>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl(kern, dim3(p.grid), dim3(kThreads), C::SMEM, st, a, p);
}

}  // namespace

size_t attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int num_sms) {
  size_t bytes = 0;
  plan_attn(q_heads, kv_heads, head_dim, num_sms, &bytes);
  return bytes;
}

cudaError_t launch_kv_attn_decode(const AttnArgs& a, int num_sms, cudaStream_t st) {
  size_t bytes = 0;
  AttnPlan p = plan_attn(a.q_heads, a.kv_heads, a.head_dim, num_sms, &bytes);
  p.counter = reinterpret_cast<unsigned*>(a.ws);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + counter_bytes(num_sms));
  if (a.head_dim <= 128) return p.per_part <= 5 ? launch_inst<5, 1>(a, p, st) : launch_inst<kMaxG, 1>(a, p, st);
  return p.per_part <= 5 ? launch_inst<5, 2>(a, p, st) : launch_inst<kMaxG, 2>(a, p, st);
}

}  // namespace qurl
