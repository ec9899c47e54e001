// sample.cu -- the next token of each row of logits, from a given uniform
// number: temperature, top-k, top-p and min-p.
//
//   w_v = exp((x_v - max x) / temperature),  order: x descending, index ascending
//   kept: the first top_k of the order, with w_v >= min_p; of those, while the
//         weight before v is below top_p times their whole weight
//   token = the first kept v, in vocabulary order, at which the running kept
//         weight exceeds u times the whole kept weight
//   logp = log w_token - log sum_v w_v,   logp_kept = log w_token - log sum_kept w_v
//
// A choice made by comparing sums of exponentials turns on their last bits, so
// the weights that decide are integers: fixed point, between 2^S and 2^(S+1) for
// the largest (S = 61 - ceil(log2 V), so the sum of V of them fits 63 bits), to a
// relative 2^-29 from a product carried as a pair and a 512-entry table of
// 2^(j/512).  Sums of integers do not depend on their order: the token is the
// same however the work is split, and is the exact one unless u or top_p lies
// within 2^-28 of a border.
//
// Bound by HBM for the first reading of a row; the weights (about 28
// instructions a logit) are what it costs beyond that, so they are computed for
// a whole row only where the choice needs the whole sum (no top-k, no min-p);
// elsewhere the row's sum, which only logp needs, is a plain fp32 one.
//
// 256 rows of 131072 bf16 logits (67 MB, 9.9 us at the copy rate): no limits 57 to 59 us,
// top-k 50 48, greedy 43, rows of mixed limits 88 to 92, top-p 0.95 at temperature 0.6 |
// 1.0: 109 | 181 (in a wave of 152 rows 13 us for the exact sum, 21 for what lies above
// the window, 25 for what one CTA does between the passes).  Without limits, stamped:
// the CTAs end the first reading after 10 to 27 us (512 of them on 152 SMs, so some SMs
// read for three and some for four), know the maximum 2 to 5 later, take 15 to 22 for
// the exact weights and 4 for the search; greedy 10 to 21, 3 to 6, 8, and 5 to 8 for
// the ranking.  One row of 32000: 14 us, 29 where the nucleus is large, the chain of
// passes.
//
// A row is worked on by a cluster of 1 to 8 CTAs, as many as fill the GPU with
// the batch.  Pass 1 takes the maximum; the threads' own maxima give a cut above
// which about 128 logits lie.  Pass 2 (the row now comes from L2) takes the sum
// and sends the logits above the cut to the cluster's first CTA, which ranks
// them against each other and draws -- all there is to do unless the kept set is
// larger.  Then an eighth of the row says between which logits a limit falls; one
// pass adds up what lies above that window and lists what lies in it, a few
// percent of the row at most.  A thread then takes one of these each: 512 steps of
// count and weight say in which step the limit falls, the logits of that step are
// ranked against each other (a radix select where there are many), and every
// segment's kept weight is known without another pass.  A limit outside its window
// is looked for in the whole row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"

namespace qurl {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTable = 512;
constexpr int kSeg = 512;        // logits per segment (or a multiple), the unit of the final search
constexpr int kMaxSegs = 512;    // segments a row is cut into at most
constexpr int kShort = 512;      // candidates ranked against each other
constexpr int kAim = 128;        // candidates the cut aims at, more for a large top-k
constexpr int kList = 1536;      // logits of one step collected for the radix select
constexpr int kWindow = 4096;    // logits of a CTA in the window: their indices take the room of `list` and `w`
constexpr int kBins = 512;
constexpr u64 kAll = ~0ull;

// 2^(j / 512) in units of 2^-30, by the Taylor series of exp in fp64 at
// compile time (arguments below ln 2: 24 terms leave less than 2^-60).
struct Exp2Table {
  uint32_t v[kTable];
  constexpr Exp2Table() : v() {
    for (int j = 0; j < kTable; ++j) {
      const double x = 0.693147180559945309417 * j / kTable;
      double term = 1.0, sum = 1.0;
      for (int n = 1; n < 24; ++n) {
        term = term * x / n;
        sum += term;
      }
      v[j] = static_cast<uint32_t>(sum * 1073741824.0 + 0.5);
    }
  }
};
__device__ const Exp2Table g_exp2 = Exp2Table();

// A logit as the sampler takes it: +inf as the largest float, NaN as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) {
  x = x + 0.0f;
  return x <= FLT_MAX ? x : (x > FLT_MAX ? FLT_MAX : -INFINITY);
}

// Monotone map of a cleaned logit to unsigned, and back.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Position of a logit in the order: smaller comes first.
__device__ __forceinline__ u64 place(float x, int i) {
  return (static_cast<u64>(~order_key(clean(x))) << 32) | static_cast<uint32_t>(i);
}
__device__ __forceinline__ float place_logit(u64 p) { return key_value(~static_cast<uint32_t>(p >> 32)); }

// What turns a row's logits into weights.
struct Scale {
  float top;       // the largest logit
  float chi, clo;  // log2(e) / temperature as a pair; for bf16 logits chi has 16 bits, so x chi is exact
  float c512;      // 512 log2(e) / temperature
  int bias;        // position of the weights' leading bit
  bool rel;        // logits of large magnitude: their difference to the top is taken first
};

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

// w as an integer: 2^(x log2(e) / temperature - E + S) with E the integer part of
// that exponent for the largest logit (in relative rows of x - top).
//   x log2(e) / temperature = k / 512 + r, |r| <= 2^-10 and a little;  w = 2^(k / 512) (1 + (2^r - 1))
// finish(): from t = k + magic and r.  2^32 (2^r - 1) = 2^32 (y + y^2 / 2 + y^3 / 6),
// y = r ln 2, as an integer (the next term is below 2^-43); (w : 0) is shifted
// down by n, and shifts of 64 and more -- logits so small, -inf and, as n is
// then negative, what is not a number -- give 0.
constexpr double kLn2 = 0.69314718055994530942, kUnit = 4294967296.0;
constexpr float kC1 = static_cast<float>(kUnit * kLn2), kC2 = static_cast<float>(kUnit * kLn2 * kLn2 / 2),
                kC3 = static_cast<float>(kUnit * kLn2 * kLn2 * kLn2 / 6);

__device__ __forceinline__ u64 finish_weight(float t, float q, const Scale& s, const uint32_t* table) {
  const int k = static_cast<int>(__float_as_uint(t));  // 0x4B400000 + k
  const int qi = static_cast<int>(__float_as_uint(q)) - 0x4B400000;
  const uint32_t tj = table[k & (kTable - 1)];
  uint32_t w;
  asm("mad.hi.s32 %0, %1, %2, %1;" : "=r"(w) : "r"(tj), "r"(qi));
  const int n = s.bias - (k >> 9);
  u64 v;
  asm("shr.b64 %0, %1, %2;" : "=l"(v) : "l"(static_cast<u64>(w) << 32), "r"(n));
  return v;
}

// One logit (kBf16: of bf16 precision).
template <bool kBf16>
__device__ __forceinline__ u64 weight(float x, const Scale& s, const uint32_t* table) {
  float t, r;
  if (s.rel) {  // x - top as an exact pair (two-sum); +inf counts as the largest float
    x = x > FLT_MAX ? FLT_MAX : x;
    const float d = __fsub_rn(x, s.top);
    const float bb = __fsub_rn(d, x);
    const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fadd_rn(s.top, bb));
    const float ph = __fmul_rn(d, s.chi);
    const float pl = __fmaf_rn(dl, s.chi, __fmaf_rn(d, s.clo, __fmaf_rn(d, s.chi, -ph)));
    t = __fmaf_rn(d, s.c512, kMagic);
    r = __fadd_rn(__fmaf_rn(__fsub_rn(t, kMagic), -1.0f / kTable, ph), pl);
  } else {
    const float ph = __fmul_rn(x, s.chi);
    t = __fmaf_rn(x, s.c512, kMagic);
    r = __fmaf_rn(__fsub_rn(t, kMagic), -1.0f / kTable, ph);
    r = kBf16 ? __fmaf_rn(x, s.clo, r) : __fadd_rn(r, __fmaf_rn(x, s.clo, __fmaf_rn(x, s.chi, -ph)));
  }
  const float c = __fmaf_rn(r, __fmaf_rn(r, kC3, kC2), kC1);
  return finish_weight(t, __fmaf_rn(r, c, kMagic), s, table);
}

// The same for a vector's logits, two at a time in the paired fp32 instructions.
template <bool kBf16, int N>
__device__ __forceinline__ void weights(const float (&x)[N], u64 (&w)[N], const Scale& s, const uint32_t* table) {
  if (s.rel) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = weight<kBf16>(x[e], s, table);
    return;
  }
  const float2 chi = make_float2(s.chi, s.chi), clo = make_float2(s.clo, s.clo), c512 = make_float2(s.c512, s.c512);
  const float2 mg = make_float2(kMagic, kMagic), nmg = make_float2(-kMagic, -kMagic);
  const float2 step = make_float2(-1.0f / kTable, -1.0f / kTable);
  const float2 c1 = make_float2(kC1, kC1), c2 = make_float2(kC2, kC2), c3 = make_float2(kC3, kC3);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2 v = make_float2(x[e], x[e + 1]);
    const float2 ph = __fmul2_rn(v, chi);
    const float2 t = __ffma2_rn(v, c512, mg);
    float2 r = __ffma2_rn(__fadd2_rn(t, nmg), step, ph);
    if (kBf16)
      r = __ffma2_rn(v, clo, r);
    else
      r = __fadd2_rn(r, __ffma2_rn(v, clo, __ffma2_rn(v, chi, make_float2(-ph.x, -ph.y))));
    const float2 q = __ffma2_rn(r, __ffma2_rn(r, __ffma2_rn(r, c3, c2), c1), mg);
    w[e] = finish_weight(t.x, q.x, s, table);
    w[e + 1] = finish_weight(t.y, q.y, s, table);
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- rows

template <typename T>
struct Load;
template <>
struct Load<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void vec(const uint4 u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ void vec(const uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
};

// A warp's part of a row: steps t0 .. t1 of 32 vectors, whole segments of `per`
// steps.
template <typename T>
struct Part {
  static constexpr int N = Load<T>::N;
  const T* x;
  int V, per, t0, t1;

  __device__ __forceinline__ uint4 load(int t) const {
    const int v = t * 32 + (threadIdx.x & 31);
    return t < t1 && v < V / N ? __ldg(reinterpret_cast<const uint4*>(x) + v) : make_uint4(0, 0, 0, 0);
  }
  // f(x, i, n): N logits from index i on, n of them in the row (the rest are -inf)
  template <typename F>
  __device__ __forceinline__ void step(int t, const uint4 u, F&& f) const {
    const int i = (t * 32 + (threadIdx.x & 31)) * N, n = min(V - i, N);
    float v[N];
    if (n == N) {
      Load<T>::vec(u, v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = e < n ? Load<T>::one(x + i + e) : -INFINITY;
    }
    f(v, i, n);
  }
  // f for every vector of the part, end(s) after each segment s; two steps are in flight.  (Not unrolled: several
  // such loops with a thousand instructions each do not fit the instruction cache, which halved their speed.)
  template <typename F, typename E>
  __device__ __forceinline__ void run(F&& f, E&& end) const {
    uint4 a = load(t0), b = load(t0 + 1);
    int sg = t0 / per, left = per;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      const uint4 c = load(t + 2);
      step(t, a, f);
      if (--left == 0 || t + 1 == t1) {
        end(sg++);
        left = per;
      }
      a = b;
      b = c;
    }
  }
  template <typename F>
  __device__ __forceinline__ void all(F&& f) const {
    run(f, [](int) {});
  }
  // the first reading, from HBM: six steps in flight
  template <typename F>
  __device__ __forceinline__ void first(F&& f) const {
    constexpr int D = 6;
    uint4 u[D];
#pragma unroll
    for (int d = 0; d < D; ++d) u[d] = load(t0 + d);
#pragma unroll 1
    for (int t = t0; t < t1; t += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const uint4 c = u[d];
        u[d] = load(t + d + D);
        if (t + d < t1) step(t + d, c, f);
      }
    }
  }
  // f for every `stride`-th step
  template <typename F>
  __device__ __forceinline__ void sample(int stride, F&& f) const {
    int t = t0 + (threadIdx.x >> 5) % stride;
    uint4 a = load(t);
#pragma unroll 1
    for (; t < t1; t += stride) {
      const uint4 b = load(t + stride);
      step(t, a, f);
      a = b;
    }
  }
};

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) { return cluster_map(p, rank); }
__device__ __forceinline__ void remote_add64(uint32_t a, u64 v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ u64 remote_get64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_get32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void remote_max32(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void remote_min32(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void remote_put64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// What the first CTA tells the others to do next.
enum : int { kDone = 0, kHistogram = 1, kCollect = 2, kSums = 3 };

struct Shared {
  u64 own[kList];   // places that this CTA found: candidates, then the logits of one step
  u64 list[kList];  // first CTA: those of the whole cluster
  u64 w[kShort];    // their weights
  u64 mass[kBins];          // by step: weight,
  u64 segs[kMaxSegs];       // by segment: weight above the window (first CTA, at the end: all kept weight),
  u64 part_segs[kMaxSegs];  // and between it and the step that was collected
  u64 part[kWarps];
  uint32_t count[kBins];    // and count
  u64 sample_mass[kBins];   // first CTA: those of the sample
  uint32_t sample_count[kBins];
  uint32_t table[kTable];
  u64 hist[256];
  u64 total;       // first CTA: the row's sum (weights, or 2^32 times the fp32 one)
  u64 limit;       // places kept
  u64 scan_total;
  uint32_t top, low;  // ordered keys: largest logit, smallest
  float cuts[8];      // each CTA's estimate of the cut; -inf: none
  uint32_t n;         // first CTA: entries of the list
  uint32_t own_n, own_at;
  uint32_t in_window;
  int order, bin;     // what to do next, and the step to collect
  float hi, lo, ref, scale;  // the window: logits above hi, those down to lo by (ref - x) scale
  u64 picked;
  u64 above_mass;     // first CTA: what lies above the window
  u64 above_count;
  u64 have;           // first CTA: weight of the candidates (0: they were too many)
  double drop;        // temperature ln(min_p)
  float before, behind;  // of the sample's measure: before a limit and behind it (negative: not known)
  uint32_t sampled;      // logits of the sample (first CTA: of all CTAs)
  int found;
  int pick_lo, pick_hi;
  float sq[kWarps];
  uint32_t short_n;   // candidates ranked
  int token;
  float chi, clo, c512;
  u64 found_before;
};

static_assert((kList + kShort) * sizeof(u64) == kWindow * sizeof(int), "the window's indices");

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Adds to a 64-bit counter in shared memory by its halves, the low one's carry
// going to the high one: 64-bit shared-memory atomics are loops of compare and
// swap (11 to 66 ns a warp at 512 to 8 counters and four CTAs an SM; this 3 to 6).
__device__ __forceinline__ void add64(u64* counter, u64 v) {
  uint32_t* half = reinterpret_cast<uint32_t*>(counter);
  const uint32_t lo = static_cast<uint32_t>(v);
  const uint32_t old = atomicAdd(half, lo);
  const uint32_t hi = static_cast<uint32_t>(v >> 32) + (old + lo < lo ? 1u : 0u);
  if (hi != 0) atomicAdd(half + 1, hi);
}

// Sum over the block; every thread gets it.
__device__ u64 block_sum(u64 v, Shared& sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += sh.part[w];
  return t;
}

// Exclusive prefix sum over the threads; the total in `all`.
__device__ u64 block_scan(u64 v, u64& all, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 c = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xFFFFFFFFu, c, o);
    if (lane >= o) c += t;
  }
  __syncthreads();
  if (lane == 31) sh.part[warp] = c;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all += sh.part[w];
  }
  return before + c - v;
}

// The place of the first element, in the order, at which the running measure
// (1 an element, or its weight) reaches `target` (at least 1); kAll when all of
// them stay below it.  each(f) calls f(place) for the elements, by the block.
template <bool kMass, bool kBf16, typename Each>
__device__ u64 radix_select(Each&& each, const Scale& s, u64 target, Shared& sh) {
  // the bits that all elements share are skipped (a digit that all share would have every thread add to one counter)
  u64 least = kAll, most = 0;
  each([&](u64 p) {
    least = p < least ? p : least;
    most = p > most ? p : most;
  });
  __syncthreads();
  if (threadIdx.x == 0) {
    sh.hist[0] = kAll;
    sh.hist[1] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 a = __shfl_xor_sync(0xFFFFFFFFu, least, o), b = __shfl_xor_sync(0xFFFFFFFFu, most, o);
    least = a < least ? a : least;
    most = b > most ? b : most;
  }
  if ((threadIdx.x & 31) == 0) {
    atomicMin(&sh.hist[0], least);
    atomicMax(&sh.hist[1], most);
  }
  __syncthreads();
  least = sh.hist[0];
  most = sh.hist[1];
  if (least > most) return kAll;  // no elements
  int top = 64 - __clzll(static_cast<long long>(least ^ most));  // bits not known yet
  u64 prefix = top == 64 ? 0 : most & (kAll << top), before = 0;
  while (top > 0) {
    const int shift = max(top - 8, 0);
    const u64 known = top == 64 ? 0 : kAll << top;
    const uint32_t digits = (1u << (top - shift)) - 1;
    __syncthreads();
    sh.hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.found = -1;
    __syncthreads();
    each([&](u64 p) {
      if ((p & known) != prefix) return;
      const u64 v = kMass ? weight<kBf16>(place_logit(p), s, sh.table) : 1ull;
      if (v) add64(&sh.hist[static_cast<uint32_t>(p >> shift) & digits], v);
    });
    __syncthreads();
    const u64 v = sh.hist[threadIdx.x];
    u64 all;
    const u64 b = before + block_scan(v, all, sh);
    if (b < target && target <= b + v) {
      sh.found = threadIdx.x;
      sh.found_before = b;
    }
    __syncthreads();
    if (sh.found < 0) return kAll;
    before = sh.found_before;
    prefix |= static_cast<u64>(sh.found) << shift;
    top = shift;
  }
  return prefix;
}

// A row's parameters.
struct Params {
  float temp, top_p, min_p, u;
  int top_k;
  bool valid, greedy;
};

__device__ __forceinline__ Params params_of(const SampleArgs& a, int b) {
  Params p;
  p.temp = a.temperature ? a.temperature[b] : 1.0f;
  p.top_k = a.top_k ? a.top_k[b] : 0;
  p.top_p = (a.top_p ? a.top_p[b] : 1.0f) + 0.0f;  // (-0, which lies in the range, becomes 0: fraction() takes bits)
  p.min_p = a.min_p ? a.min_p[b] : 0.0f;
  p.u = a.u[b] + 0.0f;
  p.valid = (p.temp == 0.0f || (p.temp >= 1e-6f && p.temp <= 1e6f)) && p.top_p >= 0.0f && p.min_p >= 0.0f &&
            p.min_p <= 1.0f && p.u >= 0.0f && p.u < 1.0f;
  if (p.top_k < 0 || p.top_k >= a.V) p.top_k = 0;
  p.greedy = p.temp == 0.0f;
  if (p.greedy) {  // the first of the order
    p.temp = 1.0f;
    p.top_k = 1;
    p.top_p = 1.0f;
    p.min_p = 0.0f;
  }
  return p;
}

// A row whose kept set may be larger than what is ranked on chip: three readings or more instead of two.
__device__ __forceinline__ bool may_be_long(const SampleArgs& a, int b) {
  const Params p = params_of(a, b);
  return p.top_k > kShort / 2 || (p.top_k == 0 && (p.top_p < 1.0f || p.min_p > 0.0f));
}

// The row that the n-th cluster of the grid takes when those rows go first: a
// long row that starts in the last wave is what the call would end on.
__device__ int row_at(const SampleArgs& a, int n, Shared& sh) {
  const int per = (a.B - 1) / kThreads + 1, r0 = min(a.B, static_cast<int>(threadIdx.x) * per), r1 = min(a.B, r0 + per);
  int longs = 0;
  for (int r = r0; r < r1; ++r) longs += may_be_long(a, r);
  u64 all;
  const int l = static_cast<int>(block_scan(static_cast<u64>(longs), all, sh));
  const bool want = n < static_cast<int>(all);  // one of the long rows
  const int at = want ? n : n - static_cast<int>(all);
  int before = want ? l : r0 - l;
  if (before <= at && at < before + (want ? longs : r1 - r0 - longs))
    for (int r = r0; r < r1; ++r)
      if (may_be_long(a, r) == want && before++ == at) sh.found = r;
  __syncthreads();
  return sh.found;
}

// floor(f * v) for f in [0, 1), not -0; `rest`: whether something was cut off.
__device__ __forceinline__ u64 fraction(float f, u64 v, bool& rest) {
  const uint32_t b = __float_as_uint(f);
  rest = false;
  if (b < 0x00800000u) return 0;  // 0, or below 2^-126
  const u64 m = (b & 0x7FFFFFu) | 0x800000u;
  const int e = 150 - static_cast<int>(b >> 23);  // f = m 2^-e, 24 <= e
  const u64 hi = __umul64hi(v, m), lo = v * m;
  if (e < 64) {
    rest = (lo & ((1ull << e) - 1)) != 0;
    return (hi << (64 - e)) | (lo >> e);
  }
  rest = true;
  return e < 128 ? hi >> (e - 64) : 0;
}
// The weight that ends a nucleus: the smallest integer not below top_p times base (at least 1).
__device__ __forceinline__ u64 nucleus(float top_p, u64 base) {
  bool rest;
  u64 t = fraction(top_p, base, rest);
  if (rest) ++t;
  return t < 1 ? 1 : t;
}
__device__ __forceinline__ u64 goal_of(float u, u64 mass) {
  bool rest;
  return fraction(u, mass, rest);
}

// log(a / b) of a >= b > 0: the quotient as a pair q, log1p where it is below 2 (to an ulp of fp32), else k ln 2 +
// log1p(m - 1) with q = 2^k m, m in [0.7, 1.42]: log1p is then below 0.35 and its ulp below 2^-25, whatever the whole.
__device__ __forceinline__ double log_ratio(u64 a, u64 b) {
  const float ah = __ull2float_rd(a), bh = __ull2float_rd(b);
  const float al = static_cast<float>(a - static_cast<u64>(ah)), bl = static_cast<float>(b - static_cast<u64>(bh));
  const float qh = __fdiv_rn(ah, bh);
  const float ql = __fdiv_rn(fmaf(-qh, bh, ah) + al - qh * bl, bh);
  if (qh < 2.0f) return log1pf((qh - 1.0f) + ql);
  const uint32_t bits = __float_as_uint(qh);
  int k = static_cast<int>(bits >> 23) - 127;
  float m = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
  if (m > 1.41421356f) {
    m *= 0.5f;
    ++k;
  }
  const float unit = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return static_cast<double>(k) * 0.69314718055994530942 + static_cast<double>(log1pf((m - 1.0f) + ql * unit));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleArgs a, int cluster) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int b = blockIdx.x / cluster;
  if (a.order) b = row_at(a, b, sh);
  const uint32_t rank = cluster_ctarank();
  const bool first = rank == 0;
  const Params pr = params_of(a, b);
  const int seg = kSeg * ((a.V - 1) / (kSeg * kMaxSegs) + 1);
  const int nseg = (a.V - 1) / seg + 1;
  constexpr int N = Load<T>::N;
  constexpr bool B16 = N == 8;  // bf16 logits
  const int s0 = static_cast<int>(static_cast<long long>(nseg) * rank / cluster);  // this CTA's segments
  const int s1 = static_cast<int>(static_cast<long long>(nseg) * (rank + 1) / cluster);
  const int warp = tid >> 5, per = seg / (32 * N), steps = (a.V - 1) / (32 * N) + 1;
  const Part<T> row{reinterpret_cast<const T*>(a.logits) + static_cast<long long>(b) * a.ld, a.V, per,
                    min(steps, (s0 + (s1 - s0) * warp / kWarps) * per),
                    min(steps, (s0 + (s1 - s0) * (warp + 1) / kWarps) * per)};
  for (int i = tid; i < kTable; i += kThreads) sh.table[i] = g_exp2.v[i];
  if (tid < 8) sh.cuts[tid] = -INFINITY;
  for (int i = tid; i < kBins; i += kThreads) {
    sh.count[i] = 0;
    sh.mass[i] = 0;
    sh.sample_count[i] = 0;
    sh.sample_mass[i] = 0;
  }
  if (tid == 0) {
    sh.top = 0;
    sh.low = 0xFFFFFFFFu;
    sh.n = 0;
    sh.own_n = 0;
    sh.total = 0;
    sh.sampled = 0;
    sh.token = 0x7FFFFFFF;
    // log2(e) / temperature as a pair
    constexpr double kLog2e = 1.4426950408889634074;
    constexpr float lh = static_cast<float>(kLog2e), ll = static_cast<float>(kLog2e - static_cast<double>(static_cast<float>(kLog2e)));
    const float ch = __fdiv_rn(lh, pr.temp);
    const float cl = __fdiv_rn(__fmaf_rn(-ch, pr.temp, lh) + ll, pr.temp);
    const float c16 = __uint_as_float(__float_as_uint(ch) & 0xFFFFFF00u);
    sh.chi = B16 ? c16 : ch;
    sh.clo = B16 ? __fadd_rn(__fsub_rn(ch, c16), cl) : cl;  // (ch - c16 is exact)
    sh.c512 = ch * kTable;
    sh.have = 0;
    if (pr.min_p > 0.0f) sh.drop = static_cast<double>(pr.temp) * log(static_cast<double>(pr.min_p));
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();  // every CTA's counters are set before another adds to them

  // ---- pass 1: the largest logit and the smallest
  float m = -INFINITY, lo = INFINITY;
  row.first([&](const float (&x)[N], int, int n) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      m = fmaxf(m, x[e]);
      lo = fminf(lo, e < n ? x[e] : INFINITY);
    }
  });
  m = clean(m);  // (the maximum leaves out what is not a number)
  lo = clean(lo);
  const float own = m;  // this thread's largest
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
  }
  if ((tid & 31) < cluster) {  // a lane for each CTA
    remote_max32(remote(&sh.top, tid & 31), order_key(m));
    remote_min32(remote(&sh.low, tid & 31), order_key(lo));
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  const float top = key_value(sh.top);
  if (!pr.valid || top == -INFINITY) {  // (the same in every CTA of the cluster)
    if (first && tid == 0) {
      if (!pr.valid) latch_bad_index(a.status);
      a.token[b] = -1;
      if (a.logp) a.logp[b] = -INFINITY;
      if (a.logp_kept) a.logp_kept[b] = -INFINITY;
    }
    return;
  }
  Scale s;
  s.top = top;
  s.chi = sh.chi;
  s.clo = sh.clo;
  s.c512 = sh.c512;
  s.rel = !(fabsf(top) * s.chi < 4000.0f);
  const int e0 = s.rel ? 0 : static_cast<int>(floorf(top * s.chi));  // (k >> 9 of the largest logit, or one beside it)
  // k >> 9 carries the magic number's 0x4B400000 >> 9; (w : 0) has its leading bit at 62 and the largest weight
  // at S or S + 1, S = 62 - shift
  s.bias = (0x4B400000 >> 9) + e0 + a.shift;
  const float extent = fminf(32.0f / (s.chi * 0.69314718f), top - key_value(sh.low));  // -inf logits: the first
  const float binscale = extent > 0.0f ? kBins / extent : 0.0f;
  // (+inf falls into the first step, -inf and what is not a number into the last)
  auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>(fmaxf(fminf((top - x) * binscale, 1e6f), 0.0f))); };

  const bool has_k = pr.top_k > 0, has_m = pr.min_p > 0.0f, has_p = pr.top_p < 1.0f;
  const bool truncated = has_k || has_m || has_p;
  const bool exact_total = !has_k && !has_m;
  // ---- the cut: of n logits above it, spread over t threads at random, t (1 - exp(-n / t)) threads hold one
  // or more -- so the cut is where that many threads' largest logits lie above it: the mean of the CTAs' estimates
  // (their highest one would leave less than a top-k of 50 in a row cut into 8)
  if (truncated) {
    if (a.V > kShort) {
      if (own != -INFINITY) atomicAdd(&sh.count[bin_of(own)], 1u);
      __syncthreads();
      const float t = 32.0f * min(kWarps, s1 - s0);
      const float aim = has_k ? fminf(kShort * 0.75f, pr.top_k * 1.25f + 32.0f) : static_cast<float>(kAim);
      const u64 want = static_cast<u64>(t * (1.0f - ex2(-1.4427f * aim / (cluster * t)))) + 1;
      u64 all;
      const u64 c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
      const u64 before = block_scan(c0 + c1, all, sh);
      __syncthreads();
      sh.count[2 * tid] = sh.count[2 * tid + 1] = 0;
      if (before < want && want <= before + c0 + c1) {
        const int at = 2 * tid + (want <= before + c0 ? 1 : 2);  // its step's lower edge
        const float estimate = top - static_cast<float>(at) / fmaxf(binscale, 1e-30f);
        for (int r = 0; r < cluster; ++r)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(&sh.cuts[rank], r)), "f"(estimate) : "memory");
      }
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  }

  // hands the CTA's own list to the first one, unless the lists together exceed the room (their count says so)
  auto send = [&](uint32_t room) {
    __syncthreads();
    if (tid == 0) {
      asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(sh.own_at) : "r"(remote(&sh.n, 0)), "r"(sh.own_n) : "memory");
    }
    __syncthreads();
    const uint32_t n = sh.own_n, at = sh.own_at, r_list = remote(sh.list, 0);
    if (at + n <= room)
      for (uint32_t i = tid; i < n; i += kThreads) remote_put64(r_list + 8 * (at + i), sh.own[i]);
    __syncthreads();
    if (tid == 0) sh.own_n = 0;
  };

  // ---- pass 2: the sum, the candidates, and (nothing cut off) the segments' sums
  float cut = -INFINITY;
  {
    float sum = 0.0f;
    int n = 0;
    for (int r = 0; r < cluster; ++r) {
      const float c = sh.cuts[r];
      if (c == -INFINITY) continue;
      sum += c;
      ++n;
    }
    if (n > 0) cut = fminf(sum / static_cast<float>(n), top);
  }
  {
    const uint32_t r_segs = remote(sh.segs, 0);
    u64 z = 0;
    if (exact_total && !has_p) {
      u64 v = 0;
      row.run(
          [&](const float (&x)[N], int, int) {
            u64 w[N];
            weights<B16>(x, w, s, sh.table);
#pragma unroll
            for (int e = 0; e < N; ++e) v += w[e];
          },
          [&](int sg) {
            v = warp_sum(v);
            if ((tid & 31) == 0) {
              remote_put64(r_segs + 8 * sg, v);
              z += v;
            }
            v = 0;
          });
    } else {
      auto candidates = [&](const float (&x)[N], int i, int n) {
        float most = x[0];
#pragma unroll
        for (int e = 1; e < N; ++e) most = fmaxf(most, x[e]);
        if (!(most >= cut)) return;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (x[e] >= cut && e < n) {
            const uint32_t at = atomicAdd(&sh.own_n, 1u);
            if (at < kShort) sh.own[at] = place(x[e], i + e);
          }
      };
      if (exact_total) {
        row.all([&](const float (&x)[N], int i, int n) {
          u64 w[N];
          weights<B16>(x, w, s, sh.table);
#pragma unroll
          for (int e = 0; e < N; ++e) z += w[e];
          candidates(x, i, n);
        });
      } else {
        float zf = 0.0f;
        const float c1 = s.c512 * (1.0f / kTable);  // log2(e) / temperature
        row.all([&](const float (&x)[N], int i, int n) {
          // (what is not a number: 0; +inf, the top: 1)
#pragma unroll
          for (int e = 0; e < N; ++e) zf += __saturatef(ex2((x[e] - top) * c1));
          candidates(x, i, n);
        });
        z = __float2ull_rn(zf * 4294967296.0f);
      }
    }
    z = block_sum(z, sh);
    if (tid == 0) remote_add64(remote(&sh.total, 0), z);
    if (truncated) send(kShort);
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();

  // ---- the first CTA ranks the candidates
  u64 limit = kAll;  // places kept
  u64 mass = 0;      // their weight
  u64 edge = kAll;   // places that min_p allows
  if (has_m) {
    // w >= min_p  <=>  x >= top + temperature ln(min_p)
    const double e = static_cast<double>(top) + sh.drop;
    float f = static_cast<float>(e);
    if (static_cast<double>(f) < e) f = nextafterf(f, INFINITY);
    edge = (static_cast<u64>(~order_key(clean(f))) << 32) | 0xFFFFFFFFull;
  }
  auto tell = [&](int order, int bin) {  // the first CTA, a thread for each of the cluster's
    if (tid >= cluster) return;
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.order, tid)), "r"(order) : "memory");
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.bin, tid)), "r"(bin) : "memory");
    remote_put64(remote(&sh.limit, tid), limit);
  };
  auto tell_window = [&](float hi, float lo, float ref, float scale) {  // likewise
    if (tid >= cluster) return;
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(&sh.hi, tid)), "f"(hi) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(&sh.lo, tid)), "f"(lo) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(&sh.ref, tid)), "f"(ref) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(&sh.scale, tid)), "f"(scale) : "memory");
  };
  auto heard = [&] {  // every CTA: the first one's order
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    return sh.order;
  };
  auto finish = [&](int token) {  // two threads, one for each logarithm
    // log w_token - log w_top = (x - top) / temperature, from an exact difference
    const float x = clean(Load<T>::one(row.x + token));
    const u64 w_top = weight<B16>(top, s, sh.table);
    const double d = (static_cast<double>(x) - static_cast<double>(top)) * (static_cast<double>(s.chi) + s.clo) * 0.69314718055994530942;
    if (tid == 0) {
      a.token[b] = token;
      u64 z = sh.total, unit = w_top;
      if (!exact_total) unit = 1ull << 32;
      if (a.logp) a.logp[b] = static_cast<float>(d - log_ratio(z, unit));
    } else if (a.logp_kept) {
      a.logp_kept[b] = pr.greedy ? 0.0f : static_cast<float>(d - log_ratio(mass, w_top));
    }
  };

  if (first) {
    const int n = static_cast<int>(sh.n);
    int next = truncated ? kHistogram : kDone;
    if (truncated && n <= kShort) {
      // thread t holds candidates t and t + kThreads
      u64 p[2], w[2], before[2] = {0, 0};
      uint32_t cnt[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = tid + e * kThreads;
        p[e] = i < n ? sh.list[i] : kAll;
        w[e] = i < n ? weight<B16>(place_logit(p[e]), s, sh.table) : 0;
        if (i < n) sh.w[i] = w[e];
      }
      __syncthreads();
      auto rank = [&](int e) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const u64 pj = sh.list[j], wj = sh.w[j];
          if (pj < p[e]) {
            ++cnt[e];
            before[e] += wj;
          }
        }
      };
      const u64 ranked = block_sum(w[0] + w[1], sh);
      // the set that top-k and min-p leave, if it lies above the cut; a top-p alone: of the whole row
      const u64 lowest = cut == -INFINITY ? kAll : (static_cast<u64>(~order_key(cut)) << 32) | 0xFFFFFFFFull;
      const bool inside = n == a.V || (exact_total ? ranked >= nucleus(pr.top_p, sh.total)
                                                   : (has_k && n >= pr.top_k) || (has_m && edge <= lowest));
      if (inside) {
        rank(0);
        if (n > kThreads) rank(1);
      }
      if (tid == 0) {
        sh.have = ranked;
        sh.short_n = static_cast<uint32_t>(n);
      }
      bool in[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        in[e] = tid + e * kThreads < n && (!has_k || cnt[e] < static_cast<uint32_t>(pr.top_k)) && p[e] <= edge;
      if (inside) {
        const u64 base = exact_total ? sh.total : block_sum((in[0] ? w[0] : 0) + (in[1] ? w[1] : 0), sh);
        const u64 target = has_p ? nucleus(pr.top_p, base) : kAll;
        const u64 have = exact_total ? ranked : base;
        if (!has_p || have >= target || n == a.V) {
#pragma unroll
          for (int e = 0; e < 2; ++e) in[e] = in[e] && before[e] < target;
          mass = block_sum((in[0] ? w[0] : 0) + (in[1] ? w[1] : 0), sh);
          const u64 goal = goal_of(pr.u, mass);
          // running kept weight in vocabulary order
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (tid + e * kThreads < n && !in[e]) sh.w[tid + e * kThreads] = 0;
          __syncthreads();
          u64 upto[2] = {0, 0};
          auto run = [&](int e) {
            const uint32_t ie = static_cast<uint32_t>(p[e]);
#pragma unroll 4
            for (int j = 0; j < n; ++j)
              if (static_cast<uint32_t>(sh.list[j]) <= ie) upto[e] += sh.w[j];
          };
          run(0);
          if (n > kThreads) run(1);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (in[e] && w[e] != 0 && upto[e] > goal) atomicMin(&sh.token, static_cast<int>(static_cast<uint32_t>(p[e])));
          __syncthreads();
          if (tid == 0 || tid == 32) finish(sh.token);
          next = kDone;
        }
      }
    } else if (!truncated) {
      mass = sh.total;
    }
    tell(next, n <= kShort ? 1 : 0);
  }
  int order = heard();

  if (order == kHistogram) {
    // ---- the kept set is larger.  A sample (of what lies below the cut, when the candidates' weight is known)
    const float below = sh.bin ? cut : INFINITY;
    auto gather = [&](u64* mass_to, uint32_t* count_to) {  // the first CTA: the sums of all CTAs' steps
      if (cluster > 1) cluster_sync();
      else __syncthreads();
      if (first) {
        for (int k = tid; k < kBins; k += kThreads) {
          u64 v = sh.mass[k];
          uint32_t c = sh.count[k];
          for (int r = 1; r < cluster; ++r) {
            v += remote_get64(remote(&sh.mass[k], r));
            c += remote_get32(remote(&sh.count[k], r));
          }
          mass_to[k] = v;
          count_to[k] = c;
        }
        __syncthreads();
      }
      // (the others keep theirs until the first CTA's next order)
    };
    auto clear = [&] {
      for (int k = tid; k < kBins; k += kThreads) {
        sh.mass[k] = 0;
        sh.count[k] = 0;
      }
      __syncthreads();
    };
    uint32_t sampled = 0;
    row.sample(steps >= 128 ? 8 : 1, [&](const float (&x)[N], int, int n) {
      sampled += max(n, 0);
      u64 w[N];
      weights<B16>(x, w, s, sh.table);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (!(x[e] < below) || e >= n) continue;
        const int k = bin_of(x[e]);
        atomicAdd(&sh.count[k], 1u);
        if (w[e]) add64(&sh.mass[k], w[e]);
      }
    });
    sampled = __reduce_add_sync(0xFFFFFFFFu, sampled);
    if ((tid & 31) == 0)
      asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(remote(&sh.sampled, 0)), "r"(sampled) : "memory");
    gather(sh.sample_mass, sh.sample_count);

    int* window = reinterpret_cast<int*>(sh.list);  // indices of the CTA's logits in the window
    // the limits in turn: top-k, the weight that min-p leaves, top-p
    u64 base = 0;
    int collected = -1;  // the step whose logits the list holds
    for (int stage = 0; stage < 3; ++stage) {
      // the same in every CTA (stage 1 after a top-k: only if the first CTA says that min-p cuts deeper)
      const bool on = stage == 0 ? has_k : stage == 1 ? has_m : has_p;
      if (!on) continue;
      u64 target = 0;
      bool skip = false;
      if (first) {
        clear();
        float hi = INFINITY, lo = -INFINITY, ref = top, scale = binscale;  // the whole row
        if (stage == 1) {
          if (edge >= limit) skip = true;  // (base is known from the top-k stage)
          else limit = edge;
          hi = lo = ref = place_logit(limit);
          scale = 0.0f;
        } else {
          if (stage == 2 && exact_total) base = sh.total;
          target = stage == 0 ? static_cast<u64>(pr.top_k) : nucleus(pr.top_p, base);
          // Where the target may lie, by the sample's steps.  A sum over the sampled logits above a step's edge has
          // the whole sum's share phi as its mean and less than the sum of their squares as its variance; so does
          // the sum below the edge, which is the better one where a few large weights lie above.  An edge bounds the
          // target when either sum says so by 4 sigma (a step's weights are nearly equal; four logits of the largest
          // weight stand for what the sample may have missed).
          const bool ranked = sh.have != 0;
          u64 v[2];
          float sq[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t n = sh.sample_count[2 * tid + e];
            v[e] = stage == 0 ? n : sh.sample_mass[2 * tid + e];
            const float w = static_cast<float>(v[e]);
            sq[e] = n > 0 ? w / static_cast<float>(n) * w : 0.0f;
          }
          u64 all;
          const u64 c = block_scan(v[0] + v[1], all, sh);
          const float w_top = static_cast<float>(weight<B16>(top, s, sh.table));
          if (tid == 0) {
            const u64 known = !ranked ? 0 : stage == 0 ? sh.short_n : sh.have;
            const float phi = static_cast<float>(sh.sampled) / static_cast<float>(a.V);
            sh.before = target > known ? static_cast<float>(target - known) * phi : 0.0f;
            // (a row's fp32 sum is in units of the largest weight)
            const float behind = exact_total ? static_cast<float>(sh.total - target)
                                             : static_cast<float>(sh.total) * 0x1p-32f * w_top - static_cast<float>(target);
            sh.behind = stage == 0 ? -1.0f : fmaxf(behind, 0.0f) * phi;
            sh.pick_lo = kBins;
            sh.pick_hi = 0;
          }
          // squares above the thread's first step, and below its last
          float up = sq[0] + sq[1], down = up;
          const int lane = tid & 31;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xFFFFFFFFu, up, o), y = __shfl_down_sync(0xFFFFFFFFu, down, o);
            if (lane >= o) up += x;
            if (lane + o < 32) down += y;
          }
          if (lane == 31) sh.sq[warp] = up;
          up -= sq[0] + sq[1];
          float after = __shfl_down_sync(0xFFFFFFFFu, down, 1);
          if (lane == 31) after = 0.0f;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            if (w < warp) up += sh.sq[w];
            if (w > warp) after += sh.sq[w];
          }
          const float slack = 1e-4f * static_cast<float>(all), c1 = s.c512 * (1.0f / kTable);
          const float most = stage == 0 ? 1.0f : ranked ? w_top * ex2((cut - top) * c1) : w_top;
          int pick_hi = 0, pick_lo = kBins;
          auto edge_at = [&](int j, u64 above, float sq_above, float sq_below) {
            const float least = stage == 0 ? 1.0f : w_top * ex2(-static_cast<float>(j) / fmaxf(binscale, 1e-30f) * c1);
            const float over = static_cast<float>(above), below = static_cast<float>(all - above);
            const float d0 = 4.0f * sqrtf(sq_above + 4.0f * most * most) + slack;
            const float d1 = 4.0f * sqrtf(sq_below + 4.0f * least * least) + slack;
            const bool known = sh.behind >= 0.0f;
            if (over + d0 <= sh.before || (known && below - d1 >= sh.behind)) pick_hi = max(pick_hi, j);
            if (over - d0 >= sh.before || (known && below + d1 <= sh.behind)) pick_lo = min(pick_lo, j);
          };
          edge_at(2 * tid, c, up, after + sq[0] + sq[1]);
          edge_at(2 * tid + 1, c + v[0], up + sq[0], after + sq[1]);
          pick_hi = __reduce_max_sync(0xFFFFFFFFu, pick_hi);
          pick_lo = __reduce_min_sync(0xFFFFFFFFu, pick_lo);
          if (lane == 0) {
            atomicMax(&sh.pick_hi, pick_hi);
            atomicMin(&sh.pick_lo, pick_lo);
          }
          __syncthreads();
          if (sh.before <= 0.0f && ranked) {  // among the candidates
            lo = cut;
            scale = top > cut ? kBins / (top - cut) : 0.0f;
          } else if (sh.pick_hi < sh.pick_lo && binscale > 0.0f) {
            if (sh.pick_hi > 0) hi = top - static_cast<float>(sh.pick_hi) / binscale;
            if (ranked) hi = fminf(hi, cut);  // (the sample starts below the cut)
            if (sh.pick_lo < kBins) lo = top - static_cast<float>(sh.pick_lo) / binscale;
            ref = fminf(hi, top);
            const float range = ref - fmaxf(lo, top - extent);
            scale = range > 0.0f ? kBins / range : 0.0f;
          }
        }
        if (tid == 0) {
          sh.above_mass = 0;
          sh.above_count = 0;
        }
        if (!skip) tell_window(hi, lo, ref, scale);
        tell(skip ? kDone : kHistogram, 0);
      }
      if (heard() == kDone) {  // nothing to look for in this stage (and every thread knows it before the next order)
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        continue;
      }
      for (int attempt = 0; attempt < 2; ++attempt) {
        const float hi = sh.hi, lo = sh.lo, ref = sh.ref, scale = sh.scale;
        auto step_of = [&](float x) { return min(kBins - 1, static_cast<int>(fminf(fmaxf((ref - x) * scale, 0.0f), 1e6f))); };
        if (!first) clear();
        if (tid == 0) sh.in_window = 0;
        __syncthreads();
        // what lies above the window is added up, what lies in it listed: few logits, which threads of their own
        // then take one each
        u64 n_above = 0, w_above = 0;
        u64 v = 0;
        row.run(
            [&](const float (&x)[N], int i, int n) {
              float most = x[0];
#pragma unroll
              for (int e = 1; e < N; ++e) most = fmaxf(most, x[e]);
              uint32_t in = 0;  // by element
              if (most >= lo) {
                u64 w[N];
                weights<B16>(x, w, s, sh.table);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                  v += x[e] > hi ? w[e] : 0;
                  n_above += x[e] > hi ? 1 : 0;
                  in |= x[e] >= lo && x[e] <= hi && e < n ? 1u << e : 0;
                }
              }
              if (!__any_sync(0xFFFFFFFFu, in != 0)) return;
              const int lane = tid & 31;
              uint32_t at = __popc(in);
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, at, o);
                if (lane >= o) at += t;
              }
              uint32_t from = 0;
              if (lane == 31) from = atomicAdd(&sh.in_window, at);
              at += __shfl_sync(0xFFFFFFFFu, from, 31) - __popc(in);
              for (; in != 0; in &= in - 1, ++at)
                if (at < kWindow) window[at] = i + __ffs(static_cast<int>(in)) - 1;
            },
            [&](int sg) {
              v = warp_sum(v);
              if ((tid & 31) == 0) {
                sh.segs[sg] = v;
                w_above += v;
              }
              v = 0;
            });
        w_above = block_sum(w_above, sh);
        n_above = block_sum(n_above, sh);
        const uint32_t n_window = sh.in_window;
        const bool listed_all = n_window <= kWindow;  // (else this CTA reads its part again)
        auto count_in = [&](float x) {
          const int k = step_of(x);
          const u64 w = weight<B16>(x, s, sh.table);
          if (stage == 0) atomicAdd(&sh.count[k], 1u);
          if (w) add64(&sh.mass[k], w);
        };
        if (listed_all) {
#pragma unroll 4
          for (uint32_t j = tid; j < n_window; j += kThreads) count_in(Load<T>::one(row.x + window[j]));
        } else {
          row.all([&](const float (&x)[N], int, int n) {
#pragma unroll 1
            for (int e = 0; e < min(n, N); ++e)
              if (x[e] >= lo && x[e] <= hi) count_in(x[e]);
          });
        }
        if (tid == 0) {
          remote_add64(remote(&sh.above_mass, 0), w_above);
          remote_add64(remote(&sh.above_count, 0), n_above);
        }
        gather(sh.mass, sh.count);
        u64 before = 0;
        if (first) {
          const u64 over = stage == 0 ? sh.above_count : sh.above_mass;
          const u64 v0 = stage == 0 ? sh.count[2 * tid] : sh.mass[2 * tid];
          const u64 v1 = stage == 0 ? sh.count[2 * tid + 1] : sh.mass[2 * tid + 1];
          u64 all;
          const u64 c = over + block_scan(v0 + v1, all, sh);
          __syncthreads();
          if (tid == 0) sh.found = stage == 1 ? 0 : -1;
          if (tid == 0) sh.found_before = over;
          __syncthreads();
          if (stage != 1 && c < target && target <= c + v0 + v1) {
            sh.found = target <= c + v0 ? 2 * tid : 2 * tid + 1;
            sh.found_before = target <= c + v0 ? c : c + v0;
          }
          __syncthreads();
          before = sh.found_before;
          const int step = sh.found;
          // not in the window: once more with the whole row (where nothing lies above it)
          const bool again = step < 0 && (hi < INFINITY || lo > -INFINITY);
          if (stage == 0) {  // the weight of the steps before
            u64 m0 = 0;
            for (int k = tid; k < (step < 0 ? kBins : step); k += kThreads) m0 += sh.mass[k];
            base = sh.above_mass + block_sum(m0, sh);
          }
          if (again) clear();
          if (tid == 0) {
            sh.n = 0;
            if (again) {
              sh.above_mass = 0;
              sh.above_count = 0;
            }
          }
          if (again) tell_window(INFINITY, -INFINITY, top, binscale);
          tell(again ? kHistogram : kCollect, step);
        }
        if (heard() == kHistogram) continue;
        const int want = collected = sh.bin;
        if (want >= 0) {
          // the step's logits, and the segments' weight between the window's upper end and the step
          for (int sg = s0 + tid; sg < s1; sg += kThreads) sh.part_segs[sg] = 0;
          __syncthreads();
          auto sort_in = [&](float x, int i) {
            const int k = step_of(x);
            if (k < want) add64(&sh.part_segs[i / seg], weight<B16>(x, s, sh.table));
            if (k == want) {
              const uint32_t at = atomicAdd(&sh.own_n, 1u);
              if (at < kList) sh.own[at] = place(x, i);
            }
          };
          if (listed_all) {
#pragma unroll 4
            for (uint32_t j = tid; j < n_window; j += kThreads) {
              const int i = window[j];
              sort_in(Load<T>::one(row.x + i), i);
            }
          } else {
            row.all([&](const float (&x)[N], int i, int n) {
#pragma unroll 1
              for (int e = 0; e < min(n, N); ++e)
                if (x[e] >= lo && x[e] <= hi) sort_in(x[e], i + e);
            });
          }
          if (cluster > 1) cluster_sync();  // the first CTA's window is read: `list` takes the step's logits
          send(kList);
        }
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        if (first && want >= 0) {
          const int n = static_cast<int>(sh.n);
          auto listed = [&](auto&& f) {
            for (int i = tid; i < n; i += kThreads) f(sh.list[i]);
          };
          auto whole = [&](auto&& f) {  // more logits in the step than the list holds (many equal ones): the row again
            for (int i = tid; i < a.V; i += kThreads) {
              const float x = Load<T>::one(row.x + i);
              if (x >= lo && x <= hi && step_of(x) == want) f(place(x, i));
            }
          };
          if (stage != 1) {
            u64 l = kAll;
            if (n <= kThreads) {  // ranked against each other
              const u64 p = tid < n ? sh.list[tid] : kAll;
              const u64 w = tid >= n ? 0 : stage == 0 ? 1 : weight<B16>(place_logit(p), s, sh.table);
              if (tid < n) sh.w[tid] = w;
              if (tid == 0) sh.picked = kAll;
              __syncthreads();
              u64 c = before;
#pragma unroll 4
              for (int j = 0; j < n; ++j)
                if (sh.list[j] < p) c += sh.w[j];
              if (c < target && target <= c + w) sh.picked = p;
              __syncthreads();
              l = sh.picked;
            } else if (stage == 0)
              l = n <= kList ? radix_select<false, B16>(listed, s, target - before, sh) : radix_select<false, B16>(whole, s, target - before, sh);
            else
              l = n <= kList ? radix_select<true, B16>(listed, s, target - before, sh) : radix_select<true, B16>(whole, s, target - before, sh);
            if (l < limit) limit = l;
          }
          if (stage != 2) {  // what the limit leaves
            u64 v = 0;
            auto add = [&](u64 p) {
              if (p <= limit) v += weight<B16>(place_logit(p), s, sh.table);
            };
            if (n <= kList) listed(add);
            else whole(add);
            base = (stage == 1 ? sh.above_mass : base) + block_sum(v, sh);
          }
        }
        break;
      }
    }
    // ---- the kept weight of every segment: above the last window, between it and the step, and of the step
    const int n_last = first ? static_cast<int>(sh.n) : 0;
    if (first) tell(kSums, collected >= 0 && n_last <= kList ? 1 : 0);
    order = heard();
    const bool quick = sh.bin == 1;
    limit = sh.limit;
    const float hi = sh.hi;
    const uint32_t r_segs = remote(sh.segs, 0);
    if (quick) {
      if (first)
        for (int sg = s0 + tid; sg < s1; sg += kThreads) sh.segs[sg] += sh.part_segs[sg];
      else
        for (int sg = s0 + tid; sg < s1; sg += kThreads) remote_put64(r_segs + 8 * sg, sh.segs[sg] + sh.part_segs[sg]);
    } else {  // (a step of more logits than the list holds)
      const float least = limit == kAll ? -INFINITY : place_logit(limit);
      u64 v = 0;
      row.run(
          [&](const float (&x)[N], int i, int n) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (x[e] <= hi && x[e] >= least && e < n && place(x[e], i + e) <= limit) v += weight<B16>(x[e], s, sh.table);
          },
          [&](int sg) {
            v = warp_sum(v);
            if ((tid & 31) == 0) remote_put64(r_segs + 8 * sg, sh.segs[sg] + v);
            v = 0;
          });
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    if (first && quick) {
      for (int i = tid; i < n_last; i += kThreads) {
        const u64 p = sh.list[i];
        if (p <= limit) add64(&sh.segs[static_cast<int>(static_cast<uint32_t>(p)) / seg], weight<B16>(place_logit(p), s, sh.table));
      }
      __syncthreads();
    }
  }

  // ---- the token's segment, then the token
  if (first && (order == kSums || !truncated)) {
    const u64 v0 = 2 * tid < nseg ? sh.segs[2 * tid] : 0;
    const u64 v1 = 2 * tid + 1 < nseg ? sh.segs[2 * tid + 1] : 0;
    u64 c = block_scan(v0 + v1, mass, sh);
    const u64 goal = goal_of(pr.u, mass);
    if (c <= goal && goal < c + v0 + v1) {
      const bool second = goal >= c + v0;
      sh.found = 2 * tid + (second ? 1 : 0);
      sh.found_before = second ? c + v0 : c;
    }
    __syncthreads();
    const int sg = sh.found;
    u64 run = sh.found_before;
    const int end = static_cast<int>(min(static_cast<long long>(sg + 1) * seg, static_cast<long long>(a.V)));
    for (int i0 = sg * seg; i0 < end && run <= goal; i0 += kThreads) {
      const int i = i0 + tid;
      u64 w = 0;
      if (i < end) {
        const float x = Load<T>::one(row.x + i);
        if (place(x, i) <= limit) w = weight<B16>(x, s, sh.table);
      }
      u64 all;
      c = run + block_scan(w, all, sh);
      if (c <= goal && goal < c + w) sh.token = i;
      run += all;
    }
    __syncthreads();
    if (tid == 0 || tid == 32) finish(sh.token);
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a_in, bool f32, int num_sms, cudaStream_t st) {
  SampleArgs a = a_in;
  a.shift = 1;  // ceil(log2 V) + 1
  while ((1LL << (a.shift - 1)) < a.V) ++a.shift;
  // CTAs a row, each with 2048 logits at least: as many as fill the SMs' four places; twice that with a top-p or min-p,
  // whose rows need very different work, and parts of 40960 logits at most, whose windows fit the list (us at 1 | 2 |
  // 4 | 8 CTAs a row: 256 x 131072, mixed limits 228 | 130 | 90 | 104, top-p 0.95 at temperature 0.8 181 | 157 | 146 |
  // 173, top-k 50 46 | 47 | 57 | 81, no limits 59 | 57 | 61 | 73, greedy 42 | 42 | 50 | 70; mixed limits, 128 x 131072
  // 198 | 105 | 88 | 75, 512 x 32000 111 | 79 | 104 | 172, 700 x 50257 130 | 113 | 155 | 251)
  const bool uneven = a.top_p || a.min_p;
  int cluster = 1;
  while (cluster < 8 && a.V / (cluster * 2) >= 2048 &&
         (static_cast<long long>(a.B) * cluster * 2 <= (uneven ? 8LL : 4LL) * num_sms || (uneven && a.V / cluster > 40960)))
    cluster *= 2;
  // more rows than fit at once: those that may be long first (256 x 131072, mixed limits, when it was built: 98 us, 111 in row order; the
  // look at every row's parameters costs a CTA about a microsecond at 256 rows)
  a.order = uneven && static_cast<long long>(a.B) * cluster > 4LL * num_sms && a.B <= 4096;
  auto* kern = f32 ? sample_kernel<float> : sample_kernel<__nv_bfloat16>;
  static bool attr_done[64][2] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev][f32]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
    if (e != cudaSuccess) return e;
    // (the default split of an SM's memory need not leave room for four CTAs)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done[dev][f32] = true;
  }
  return launch_pdl_cluster(kern, cluster, dim3(static_cast<unsigned>(a.B) * cluster), dim3(kThreads), sizeof(Shared), st, a,
                            cluster);
}

}  // namespace qurl
