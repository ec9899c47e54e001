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
// A row is worked on by a cluster of 1 to 8 CTAs, as many as fill the GPU with
// the batch.  Pass 1 takes the maximum; the threads' own maxima give a cut above
// which about 300 logits lie.  Pass 2 (the row now comes from L2)
// takes the sum and sends the logits above the cut to the cluster's first CTA,
// which ranks them against each other and draws -- all there is to do unless the
// kept set is larger.  Then a histogram of the whole row by equal steps of x
// (count and weight) finds the step in which a limit falls, the step's logits
// alone are collected, and a radix select among them gives the limit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qurl {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTable = 512;
constexpr int kSeg = 1024;       // logits per segment: a warp's step, and the unit of the final search
constexpr int kMaxSegs = 512;    // segments (of a multiple of kSeg logits) a row is cut into at most
constexpr int kShort = 512;      // candidates ranked against each other
constexpr int kAim = 320;        // candidates the cut aims at
constexpr int kList = 4096;      // logits of one histogram step collected for the radix select
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
  return (static_cast<u64>(~order_key(x)) << 32) | static_cast<uint32_t>(i);
}
__device__ __forceinline__ float place_logit(u64 p) { return key_value(~static_cast<uint32_t>(p >> 32)); }

// What turns a row's logits into weights.
struct Scale {
  float top;       // the largest logit
  float chi, clo;  // log2(e) / temperature as a pair
  float zero;      // exponents up to this weigh less than a unit: 0
  int bias;        // position of the weights' leading bit, see weight()
  bool rel;        // logits of large magnitude: their difference to the top is taken first
};

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

// w as an integer: 2^(x log2(e) / temperature - E + S) with E the integer part of
// that exponent for the largest logit (in relative rows of x - top).
__device__ __forceinline__ u64 weight(float x, const Scale& s, const uint32_t* table) {
  float d = x, dl = 0.0f;
  if (s.rel) {  // x - top as an exact pair (two-sum)
    d = __fsub_rn(x, s.top);
    const float bb = __fsub_rn(d, x);
    dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fadd_rn(s.top, bb)) * s.chi;
  }
  const float ph = __fmul_rn(d, s.chi);
  const float pl = fmaf(d, s.clo, fmaf(d, s.chi, -ph)) + dl;
  // ph + pl = k / 512 + r, |r| <= 2^-10 and a little
  const float t = fmaf(ph, static_cast<float>(kTable), kMagic);
  const int k = static_cast<int>(__float_as_uint(t));  // 0x4B400000 + k
  const float r = fmaf(t - kMagic, -1.0f / kTable, ph) + pl;
  // 2^r - 1 = y + y^2 / 2 + y^3 / 6, y = r ln 2: the next term is below 2^-43
  const float y = r * 0.693147180559945309f;
  const float q = fmaf(y * y, fmaf(y, 1.0f / 6.0f, 0.5f), y);
  const int qi = static_cast<int>(__float_as_uint(fmaf(q, 4294967296.0f, kMagic))) - 0x4B400000;
  const uint32_t tj = table[k & (kTable - 1)];
  const uint32_t w = tj + static_cast<uint32_t>(__mulhi(static_cast<int>(tj), qi));
  const int n = min(s.bias - (k >> 9), 63);  // bits to shift (w : 0) down by
  const u64 v = (static_cast<u64>(w) << 32) >> (n & 63);
  return ph > s.zero ? v : 0;  // (false for what is not a number)
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
  static __device__ __forceinline__ float one(const float* p) { return clean(__ldg(p)); }
  static __device__ __forceinline__ void vec(const uint4 u, float (&x)[4]) {
    x[0] = clean(__uint_as_float(u.x));
    x[1] = clean(__uint_as_float(u.y));
    x[2] = clean(__uint_as_float(u.z));
    x[3] = clean(__uint_as_float(u.w));
  }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return clean(__bfloat162float(*p));
  }
  static __device__ __forceinline__ void vec(const uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = clean(__uint_as_float(w[e] << 16));
      x[2 * e + 1] = clean(__uint_as_float(w[e] & 0xFFFF0000u));
    }
  }
};

// A CTA's part of a row: segments s0 .. s1 of `seg` logits, its warps in turn.
template <typename T>
struct Part {
  const T* x;
  int V, seg, s0, s1;

  // f(x, i) for every logit of segment s, by the calling warp
  template <typename F>
  __device__ __forceinline__ void segment(int s, F&& f) const {
    constexpr int N = Load<T>::N, U = 4;  // U vectors in flight a lane
    const int lane = threadIdx.x & 31;
    const int end = static_cast<int>(min(static_cast<long long>(s + 1) * seg, static_cast<long long>(V)));
    int i = s * seg;
    for (; i + 32 * N * U <= end; i += 32 * N * U) {
      uint4 u[U];
#pragma unroll
      for (int e = 0; e < U; ++e) u[e] = __ldg(reinterpret_cast<const uint4*>(x + i) + e * 32 + lane);
#pragma unroll
      for (int e = 0; e < U; ++e) {
        float v[N];
        Load<T>::vec(u[e], v);
#pragma unroll
        for (int j = 0; j < N; ++j) f(v[j], i + (e * 32 + lane) * N + j);
      }
    }
    for (i += lane; i < end; i += 32) f(Load<T>::one(x + i), i);
  }
  // f for every logit of the part
  template <typename F>
  __device__ __forceinline__ void all(F&& f) const {
    for (int s = s0 + (threadIdx.x >> 5); s < s1; s += kWarps) segment(s, f);
  }
};

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) { return cluster_map(p, rank); }
__device__ __forceinline__ void remote_add64(uint32_t a, u64 v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_add32(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_take(uint32_t a) {
  uint32_t r;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(r) : "r"(a) : "memory");
  return r;
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
  u64 list[kList];  // first CTA: places of the candidates, then of one histogram step
  u64 w[kShort];    // their weights
  u64 mass[kBins];
  u64 segs[kMaxSegs];
  u64 part[kWarps];
  uint32_t count[kBins];
  uint32_t table[kTable];
  u64 hist[256];
  u64 total;       // first CTA: the row's sum (weights, or 2^32 times the fp32 one)
  u64 limit;       // places kept
  u64 scan_total;
  uint32_t top, low;  // ordered keys: largest logit, smallest
  uint32_t cut;       // ordered key
  uint32_t n;         // first CTA: entries of the list
  int order, bin;     // the next step, and its histogram step
  int found;
  int token;
  float chi, clo;
  u64 found_before;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
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
template <bool kMass, typename Each>
__device__ u64 radix_select(Each&& each, const Scale& s, u64 target, Shared& sh) {
  u64 prefix = 0, before = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
    sh.hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.found = -1;
    __syncthreads();
    const u64 known = shift == 56 ? 0 : kAll << (shift + 8);
    each([&](u64 p) {
      if ((p & known) != prefix) return;
      const u64 v = kMass ? weight(place_logit(p), s, sh.table) : 1ull;
      if (v) atomicAdd(&sh.hist[(p >> shift) & 255], v);
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
  p.top_p = a.top_p ? a.top_p[b] : 1.0f;
  p.min_p = a.min_p ? a.min_p[b] : 0.0f;
  p.u = a.u[b];
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

// The weight that ends a nucleus: the smallest integer not below top_p times base (at least 1).
__device__ __forceinline__ u64 nucleus(float top_p, u64 base) {
  const u64 t = static_cast<u64>(ceil(static_cast<double>(top_p) * static_cast<double>(base)));
  return t < 1 ? 1 : t;
}
__device__ __forceinline__ u64 goal_of(float u, u64 mass) {
  return static_cast<u64>(static_cast<double>(u) * static_cast<double>(mass));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleArgs a, int cluster) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / cluster;
  const uint32_t rank = cluster_ctarank();
  const bool first = rank == 0;
  const Params pr = params_of(a, b);
  const int seg = kSeg * ((a.V - 1) / (kSeg * kMaxSegs) + 1);
  const int nseg = (a.V - 1) / seg + 1;
  const Part<T> row{reinterpret_cast<const T*>(a.logits) + static_cast<long long>(b) * a.ld, a.V, seg,
                    static_cast<int>(static_cast<long long>(nseg) * rank / cluster),
                    static_cast<int>(static_cast<long long>(nseg) * (rank + 1) / cluster)};
  for (int i = tid; i < kTable; i += kThreads) sh.table[i] = g_exp2.v[i];
  for (int i = tid; i < kBins; i += kThreads) {
    sh.count[i] = 0;
    sh.mass[i] = 0;
  }
  if (tid == 0) {
    sh.top = 0;
    sh.low = 0xFFFFFFFFu;
    sh.cut = 0;
    sh.n = 0;
    sh.total = 0;
    sh.token = 0x7FFFFFFF;
    const double c = 1.4426950408889634074 / static_cast<double>(pr.temp);
    sh.chi = static_cast<float>(c);
    sh.clo = static_cast<float>(c - static_cast<double>(sh.chi));
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();  // every CTA's counters are set before another adds to them

  // ---- pass 1: the largest logit and the smallest
  float m = -INFINITY, lo = INFINITY;
  row.all([&](float x, int) {
    m = fmaxf(m, x);
    lo = fminf(lo, x);
  });
  const float own = m;  // this thread's largest
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
  }
  if ((tid & 31) == 0) {
    const uint32_t km = order_key(m), kl = order_key(lo);
    for (int r = 0; r < cluster; ++r) {
      remote_max32(remote(&sh.top, r), km);
      remote_min32(remote(&sh.low, r), kl);
    }
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  const float top = key_value(sh.top);
  if (!pr.valid || top == -INFINITY) {  // (the same in every CTA of the cluster)
    if (first && tid == 0) {
      if (!pr.valid) atomicCAS(a.status, kDevOk, kDevBadIndex);
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
  s.rel = !(fabsf(top) * s.chi < 4000.0f);
  const int e0 = s.rel ? 0 : static_cast<int>(floorf(top * s.chi));  // (k >> 9 of the largest logit, or one beside it)
  // k >> 9 carries the magic number's 0x4B400000 >> 9; (w : 0) has its leading bit at 62 and the largest weight
  // at S or S + 1, S = 62 - shift
  s.bias = (0x4B400000 >> 9) + e0 + a.shift;
  s.zero = s.rel ? -70.0f : top * s.chi - 70.0f;
  const float extent = fminf(32.0f / (s.chi * 0.69314718f), top - key_value(sh.low));  // -inf logits: the first
  const float binscale = extent > 0.0f ? kBins / extent : 0.0f;
  auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>(fminf((top - x) * binscale, 1e6f))); };

  const bool has_k = pr.top_k > 0, has_m = pr.min_p > 0.0f, has_p = pr.top_p < 1.0f;
  const bool truncated = has_k || has_m || has_p;
  const bool exact_total = !has_k && !has_m;
  // ---- the cut: of n logits above it, spread over t threads at random, t (1 - exp(-n / t)) threads hold one
  // or more -- so the cut is where that many threads' largest logits lie above it
  if (truncated) {
    if (a.V > kShort) {
      if (own != -INFINITY) atomicAdd(&sh.count[bin_of(own)], 1u);
      __syncthreads();
      const float t = 32.0f * min(kWarps, row.s1 - row.s0);
      const u64 want = static_cast<u64>(t * (1.0f - ex2(-1.4427f * kAim / (cluster * t)))) + 1;
      u64 all;
      const u64 c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
      const u64 before = block_scan(c0 + c1, all, sh);
      __syncthreads();
      sh.count[2 * tid] = sh.count[2 * tid + 1] = 0;
      if (before < want && want <= before + c0 + c1) {
        const int at = 2 * tid + (want <= before + c0 ? 1 : 2);  // its step's lower edge
        const uint32_t key = order_key(top - static_cast<float>(at) / fmaxf(binscale, 1e-30f));
        for (int r = 0; r < cluster; ++r) remote_max32(remote(&sh.cut, r), key);
      }
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  }

  // ---- pass 2: the sum, the candidates, and (nothing cut off) the segments' sums
  const float cut = sh.cut == 0 ? -INFINITY : key_value(sh.cut);
  {
    const uint32_t r_n = remote(&sh.n, 0), r_list = remote(sh.list, 0), r_segs = remote(sh.segs, 0);
    u64 z = 0;
    if (exact_total && !has_p) {
      for (int sg = row.s0 + (tid >> 5); sg < row.s1; sg += kWarps) {
        u64 v = 0;
        row.segment(sg, [&](float x, int) { v += weight(x, s, sh.table); });
        v = warp_sum(v);
        if ((tid & 31) == 0) {
          remote_put64(r_segs + 8 * sg, v);
          z += v;
        }
      }
    } else {
      auto candidate = [&](float x, int i) {
        if (x >= cut) {
          const uint32_t at = remote_take(r_n);
          if (at < kShort) remote_put64(r_list + 8 * at, place(x, i));
        }
      };
      if (exact_total) {
        row.all([&](float x, int i) {
          z += weight(x, s, sh.table);
          candidate(x, i);
        });
      } else {
        float zf = 0.0f;
        row.all([&](float x, int i) {
          zf += ex2((x - top) * s.chi);
          candidate(x, i);
        });
        z = __float2ull_rn(zf * 4294967296.0f);
      }
    }
    z = block_sum(z, sh);
    if (tid == 0) remote_add64(remote(&sh.total, 0), z);
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();

  // ---- the first CTA ranks the candidates
  u64 limit = kAll;  // places kept
  u64 mass = 0;      // their weight
  u64 edge = kAll;   // places that min_p allows
  if (has_m) {
    // w >= min_p  <=>  x >= top + temperature ln(min_p)
    const double e = static_cast<double>(top) + static_cast<double>(pr.temp) * log(static_cast<double>(pr.min_p));
    float f = static_cast<float>(e);
    if (static_cast<double>(f) < e) f = nextafterf(f, INFINITY);
    edge = (static_cast<u64>(~order_key(clean(f))) << 32) | 0xFFFFFFFFull;
  }
  auto tell = [&](int order, int bin) {  // thread 0 of the first CTA
    for (int r = 0; r < cluster; ++r) {
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.order, r)), "r"(order) : "memory");
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.bin, r)), "r"(bin) : "memory");
      remote_put64(remote(&sh.limit, r), limit);
    }
  };
  auto heard = [&] {  // every CTA: the first one's order
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    return sh.order;
  };
  auto finish = [&](int token) {  // one thread
    a.token[b] = token;
    const double x = Load<T>::one(row.x + token);
    const double ln2 = 0.69314718055994530942;
    const double zt = (s.rel ? x - static_cast<double>(top) : x) / static_cast<double>(pr.temp);
    const double unit = ln2 * (e0 - (62 - a.shift));
    double z = static_cast<double>(sh.total);
    if (!exact_total) z = z * 0x1p-32 * static_cast<double>(weight(top, s, sh.table));
    if (a.logp) a.logp[b] = static_cast<float>(zt - (log(z) + unit));
    if (a.logp_kept) a.logp_kept[b] = pr.greedy ? 0.0f : static_cast<float>(zt - (log(static_cast<double>(mass)) + unit));
  };

  if (first) {
    const int n = static_cast<int>(sh.n);
    int next = truncated ? kHistogram : kDone;
    if (truncated && n <= kShort) {
      // thread t holds candidates t and t + kThreads
      u64 p[2], w[2], cnt[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = tid + e * kThreads;
        p[e] = i < n ? sh.list[i] : kAll;
        w[e] = i < n ? weight(place_logit(p[e]), s, sh.table) : 0;
        if (i < n) sh.w[i] = w[e];
      }
      __syncthreads();
      for (int j = 0; j < n; ++j) {
        const u64 pj = sh.list[j], wj = sh.w[j];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (pj < p[e]) {
            ++cnt[e];
            before[e] += wj;
          }
      }
      // the set that top-k and min-p leave, if it lies above the cut
      const u64 lowest = cut == -INFINITY ? kAll : (static_cast<u64>(~order_key(cut)) << 32) | 0xFFFFFFFFull;
      bool inside = (has_k && n >= pr.top_k) || (has_m && edge <= lowest) || n == a.V;
      bool in[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        in[e] = tid + e * kThreads < n && (!has_k || cnt[e] < static_cast<u64>(pr.top_k)) && p[e] <= edge;
      u64 base = 0;
      if (exact_total) {
        base = sh.total;
        inside = true;
      } else if (inside) {
        base = block_sum((in[0] ? w[0] : 0) + (in[1] ? w[1] : 0), sh);
      }
      if (inside) {
        const u64 target = has_p ? nucleus(pr.top_p, base) : kAll;
        const u64 have = exact_total ? block_sum(w[0] + w[1], sh) : base;  // weight of what is ranked
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
          const uint32_t i0 = static_cast<uint32_t>(p[0]), i1 = static_cast<uint32_t>(p[1]);
          for (int j = 0; j < n; ++j) {
            const uint32_t ij = static_cast<uint32_t>(sh.list[j]);
            const u64 wj = sh.w[j];
            if (ij <= i0) upto[0] += wj;
            if (ij <= i1) upto[1] += wj;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (in[e] && w[e] != 0 && upto[e] > goal) atomicMin(&sh.token, static_cast<int>(static_cast<uint32_t>(p[e])));
          __syncthreads();
          if (tid == 0) finish(sh.token);
          next = kDone;
        }
      }
    } else if (!truncated) {
      mass = sh.total;
    }
    if (tid == 0) tell(next, 0);
  }
  int order = heard();

  if (order == kHistogram) {
    // ---- the kept set is larger: count and weight of the row by equal steps of x
    row.all([&](float x, int) {
      const u64 w = weight(x, s, sh.table);
      const int k = bin_of(x);
      atomicAdd(&sh.count[k], 1u);
      if (w) atomicAdd(&sh.mass[k], w);
    });
    __syncthreads();
    if (!first) {
      for (int k = tid; k < kBins; k += kThreads)
        if (sh.count[k]) {
          remote_add32(remote(&sh.count[k], 0), sh.count[k]);
          remote_add64(remote(&sh.mass[k], 0), sh.mass[k]);
        }
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    // the limits in turn: top-k, the weight that min-p leaves, top-p; each looks into one step
    u64 base = 0;
    for (int stage = 0; stage < 3; ++stage) {
      // (uniform over the cluster: stages depend on the row's parameters alone)
      const bool on = stage == 0 ? has_k : stage == 1 ? !exact_total : has_p;
      if (!on) continue;
      u64 before = 0;  // count (stage 0) or weight of the steps before the one looked into
      u64 target = 0;
      int step = 0;
      if (first) {
        if (stage == 2 && exact_total) base = sh.total;
        if (stage == 0) target = static_cast<u64>(pr.top_k);
        if (stage == 2) target = nucleus(pr.top_p, base);
        if (stage == 1) {
          // the step of the limit so far (min-p's edge, or the top-k element found)
          if (edge < limit) limit = edge;
          step = bin_of(place_logit(limit));
        }
        const u64 v0 = stage == 0 ? sh.count[2 * tid] : sh.mass[2 * tid];
        const u64 v1 = stage == 0 ? sh.count[2 * tid + 1] : sh.mass[2 * tid + 1];
        u64 all;
        const u64 c = block_scan(v0 + v1, all, sh);
        __syncthreads();
        if (tid == 0) sh.found = -1;
        __syncthreads();
        if (stage == 1) {
          if (step >> 1 == tid) {
            sh.found = step;
            sh.found_before = (step & 1) ? c + v0 : c;
          }
        } else if (c < target && target <= c + v0 + v1) {
          sh.found = target <= c + v0 ? 2 * tid : 2 * tid + 1;
          sh.found_before = target <= c + v0 ? c : c + v0;
        }
        __syncthreads();
        step = sh.found;
        before = sh.found_before;
        if (tid == 0) {
          sh.n = 0;
          tell(kCollect, step);
        }
      }
      heard();
      const int want = sh.bin;
      if (want >= 0) {
        const uint32_t r_n = remote(&sh.n, 0), r_list = remote(sh.list, 0);
        row.all([&](float x, int i) {
          if (bin_of(x) != want) return;
          const uint32_t at = remote_take(r_n);
          if (at < kList) remote_put64(r_list + 8 * at, place(x, i));
        });
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
            if (bin_of(x) == want) f(place(x, i));
          }
        };
        if (stage == 1) {
          u64 v = 0;
          auto add = [&](u64 p) {
            if (p <= limit) v += weight(place_logit(p), s, sh.table);
          };
          if (n <= kList) listed(add);
          else whole(add);
          base = before + block_sum(v, sh);
        } else {
          u64 l;
          if (stage == 0)
            l = n <= kList ? radix_select<false>(listed, s, target - before, sh) : radix_select<false>(whole, s, target - before, sh);
          else
            l = n <= kList ? radix_select<true>(listed, s, target - before, sh) : radix_select<true>(whole, s, target - before, sh);
          if (l < limit) limit = l;
        }
      }
    }
    if (first && tid == 0) tell(kSums, 0);
    order = heard();
    // ---- the kept weight of every segment
    limit = sh.limit;
    const uint32_t r_segs = remote(sh.segs, 0);
    for (int sg = row.s0 + (tid >> 5); sg < row.s1; sg += kWarps) {
      u64 v = 0;
      row.segment(sg, [&](float x, int i) {
        if (place(x, i) <= limit) v += weight(x, s, sh.table);
      });
      v = warp_sum(v);
      if ((tid & 31) == 0) remote_put64(r_segs + 8 * sg, v);
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
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
        if (place(x, i) <= limit) w = weight(x, s, sh.table);
      }
      u64 all;
      c = run + block_scan(w, all, sh);
      if (c <= goal && goal < c + w) sh.token = i;
      run += all;
    }
    __syncthreads();
    if (tid == 0) finish(sh.token);
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a_in, bool f32, int num_sms, cudaStream_t st) {
  SampleArgs a = a_in;
  a.shift = 1;  // ceil(log2 V) + 1
  while ((1LL << (a.shift - 1)) < a.V) ++a.shift;
  // CTAs a row: as many as two for every SM leave the batch, each with 2048 logits at least
  int cluster = 1;
  while (cluster < 8 && static_cast<long long>(a.B) * cluster * 2 <= 4LL * num_sms && a.V / (cluster * 2) >= 2048) cluster *= 2;
  auto* kern = f32 ? sample_kernel<float> : sample_kernel<__nv_bfloat16>;
  static bool attr_done[64][2] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev][f32]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
    if (e != cudaSuccess) return e;
    attr_done[dev][f32] = true;
  }
  return launch_pdl_cluster(kern, cluster, dim3(static_cast<unsigned>(a.B) * cluster), dim3(kThreads), sizeof(Shared), st, a,
                            cluster);
}

}  // namespace qurl
