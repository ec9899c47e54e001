// sample.cu -- the next token of each row of logits, from a given uniform
// number: temperature, top-k, top-p and min-p.
//
//   z_v = (x_v - max x) / temperature,  w_v = exp(z_v),  order: x descending, index ascending
//   kept: the first top_k of the order, with w_v >= min_p; of those, while the
//         weight before v is below top_p times their whole weight
//   token = the first kept v, in vocabulary order, at which the running kept
//         weight exceeds u times the whole kept weight
//   logp = z_token - log sum_v w_v,   logp_kept = z_token - log sum_kept w_v
//
// A choice made by comparing sums of exponentials turns on their last bits, so
// the weights are integers: w_v in fixed point, 2^S for the largest (S = 62 -
// ceil(log2 V), so the sum of V of them fits 63 bits), computed to a relative
// 2^-29 from an exact difference x_v - max x (a compensated pair) and a
// 512-entry table of 2^(j/512).  Sums of integers do not depend on their
// order: the token is the same however the work is split, and differs from
// the choice in exact arithmetic only when u or top_p lies within ~2^-29 of a
// border.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qurl {
namespace {

constexpr int kThreads = 1024;
constexpr int kTable = 512;

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

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

// A logit as the sampler takes it: +inf as the largest float, NaN as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) {
  x = x + 0.0f;
  if (!(x <= FLT_MAX)) x = x > FLT_MAX ? FLT_MAX : -INFINITY;
  return x;
}

// Monotone map of a cleaned logit to unsigned.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What turns a row's logits into weights.
struct Scale {
  float top;       // the largest logit
  float chi, clo;  // log2(e) / temperature as a pair
  int shift;       // 62 - S
};

// exp((x - top) / temperature) in units of 2^-S.
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s, const uint32_t* table) {
  // x - top as an exact pair (two-sum)
  const float d = __fsub_rn(x, s.top);
  const float bb = __fsub_rn(d, x);
  const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fadd_rn(s.top, bb));
  const float ph = __fmul_rn(d, s.chi);
  if (!(ph > -126.0f)) return 0;  // below 2^-S for every S <= 62; and what is not a number
  const float pl = fmaf(d, s.chi, -ph) + fmaf(d, s.clo, dl * s.chi);
  // ph = k / 512 + r with |r| <= 2^-10; the magic sum rounds to an integer
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const float t = fmaf(ph, static_cast<float>(kTable), kMagic);
  const int k = static_cast<int>(__float_as_uint(t)) - 0x4B400000;
  const float r = fmaf(t - kMagic, -1.0f / kTable, ph) + pl;
  // 2^r - 1 = r ln2 (1 + r ln2 / 2 (1 + r ln2 / 3)): the next term is below 2^-43
  const float y = r * 0.693147180559945309f;
  const float q = fmaf(y * y, fmaf(y, 1.0f / 6.0f, 0.5f), y);
  const int qi = static_cast<int>(__float_as_uint(fmaf(q, 4294967296.0f, kMagic))) - 0x4B400000;
  const uint32_t tj = table[k & (kTable - 1)];
  const uint32_t w = tj + static_cast<uint32_t>(__mulhi(static_cast<int>(tj), qi));
  const int n = s.shift - (k >> 9);  // w is 2^30 .. 2^31 for 2^(k >> 9)
  return n > 63 ? 0 : (static_cast<unsigned long long>(w) << 32) >> n;
}

__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

struct Shared {
  uint32_t table[kTable];
  unsigned long long hist[256];
  unsigned long long part[kThreads / 32];
  uint32_t top;
  int first;
  unsigned long long found_before, found_in;
  int found_bin;
  int token;
  uint32_t count;
};

__device__ unsigned long long block_sum64(unsigned long long v, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum64(v);
  __syncthreads();
  if (lane == 0) sh.part[warp] = v;
  __syncthreads();
  unsigned long long t = 0;
  for (int w = 0; w < kThreads / 32; ++w) t += sh.part[w];
  return t;
}

template <typename T>
struct Row {
  const T* x;
  int V;
};

// Position of an element in the order: smaller comes first.
__device__ __forceinline__ unsigned long long place(float x, int i) {
  return (static_cast<unsigned long long>(~order_key(x)) << 32) | static_cast<uint32_t>(i);
}

// The place of the first element, in the order, at which the running measure
// (1 an element, or its weight) reaches `target`; ~0 when the whole row stays
// below it.  Only elements at places <= limit count.
template <bool kMass, typename T>
__device__ unsigned long long select(const Row<T>& row, const Scale& s, unsigned long long target,
                                     unsigned long long limit, Shared& sh) {
  unsigned long long prefix = 0, before = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    __syncthreads();
    const unsigned long long known = shift == 56 ? 0 : ~0ull << (shift + 8);
    for (int i = threadIdx.x; i < row.V; i += kThreads) {
      const float x = clean(load_logit(row.x + i));
      const unsigned long long p = place(x, i);
      if ((p & known) != prefix || p > limit) continue;
      const unsigned long long v = kMass ? weight(x, s, sh.table) : 1ull;
      if (v) atomicAdd(&sh.hist[(p >> shift) & 255], v);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long c = before;
      int d = 0;
      while (d < 256 && c + sh.hist[d] < target) c += sh.hist[d++];
      sh.found_bin = d;
      sh.found_before = c;
    }
    __syncthreads();
    if (sh.found_bin == 256) return ~0ull;
    before = sh.found_before;
    prefix |= static_cast<unsigned long long>(sh.found_bin) << shift;
  }
  return prefix;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Shared sh;
  const int b = blockIdx.x;
  const Row<T> row{reinterpret_cast<const T*>(a.logits) + static_cast<long long>(b) * a.ld, a.V};
  const float temp = a.temperature ? a.temperature[b] : 1.0f;
  const int top_k = a.top_k ? a.top_k[b] : 0;
  const float top_p = a.top_p ? a.top_p[b] : 1.0f;
  const float min_p = a.min_p ? a.min_p[b] : 0.0f;
  const float u = a.u[b];
  const bool valid = (temp == 0.0f || (temp >= 1e-6f && temp <= 1e6f)) && top_p >= 0.0f && min_p >= 0.0f && min_p <= 1.0f && u >= 0.0f && u < 1.0f;
  for (int i = threadIdx.x; i < kTable; i += kThreads) sh.table[i] = g_exp2.v[i];
  if (threadIdx.x == 0) {
    sh.top = 0;
    sh.token = 0x7FFFFFFF;
  }
  __syncthreads();
  float m = -INFINITY;
  for (int i = threadIdx.x; i < a.V; i += kThreads) m = fmaxf(m, clean(load_logit(row.x + i)));
  atomicMax(&sh.top, order_key(m));
  __syncthreads();
  const float top = key_value(sh.top);
  if (!valid || top == -INFINITY) {
    if (threadIdx.x == 0) {
      if (!valid) atomicCAS(a.status, kDevOk, kDevBadIndex);
      a.token[b] = -1;
      if (a.logp) a.logp[b] = -INFINITY;
      if (a.logp_kept) a.logp_kept[b] = -INFINITY;
    }
    return;
  }
  Scale s;
  s.top = top;
  const double c = 1.4426950408889634074 / static_cast<double>(temp == 0.0f ? 1.0f : temp);
  s.chi = static_cast<float>(c);
  s.clo = static_cast<float>(c - static_cast<double>(s.chi));
  s.shift = a.shift;
  unsigned long long z = 0;
  for (int i = threadIdx.x; i < a.V; i += kThreads) z += weight(clean(load_logit(row.x + i)), s, sh.table);
  z = block_sum64(z, sh);
  // the places kept: those <= limit
  unsigned long long limit = ~0ull;
  unsigned long long mass = z;
  if (temp == 0.0f) {
    limit = select<false>(row, s, 1, limit, sh);
  } else {
    if (min_p > 0.0f) {
      // w >= min_p  <=>  x >= top + temperature ln(min_p)
      const double edge = static_cast<double>(top) + static_cast<double>(temp) * log(static_cast<double>(min_p));
      float e = static_cast<float>(edge);
      if (static_cast<double>(e) < edge) e = nextafterf(e, INFINITY);
      limit = (static_cast<unsigned long long>(~order_key(clean(e))) << 32) | 0xFFFFFFFFull;
    }
    if (top_k > 0 && top_k < a.V) {
      const unsigned long long l = select<false>(row, s, static_cast<unsigned long long>(top_k), limit, sh);
      limit = l < limit ? l : limit;
    }
    if (top_p < 1.0f) {
      unsigned long long base = 0;
      for (int i = threadIdx.x; i < a.V; i += kThreads) {
        const float x = clean(load_logit(row.x + i));
        if (place(x, i) <= limit) base += weight(x, s, sh.table);
      }
      base = block_sum64(base, sh);
      const double t = ceil(static_cast<double>(top_p) * static_cast<double>(base));
      unsigned long long target = static_cast<unsigned long long>(t);
      if (target < 1) target = 1;
      const unsigned long long l = select<true>(row, s, target, limit, sh);
      limit = l < limit ? l : limit;
    }
  }
  if (limit != ~0ull) {
    mass = 0;
    for (int i = threadIdx.x; i < a.V; i += kThreads) {
      const float x = clean(load_logit(row.x + i));
      if (place(x, i) <= limit) mass += weight(x, s, sh.table);
    }
    mass = block_sum64(mass, sh);
  }
  // the first index whose running kept weight exceeds u * mass
  const unsigned long long goal = static_cast<unsigned long long>(static_cast<double>(u) * static_cast<double>(mass));
  unsigned long long before = 0;
  for (int i0 = 0; i0 < a.V; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    unsigned long long w = 0;
    if (i < a.V) {
      const float x = clean(load_logit(row.x + i));
      if (place(x, i) <= limit) w = weight(x, s, sh.table);
    }
    // inclusive scan over the block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned long long c2 = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, c2, o);
      if (lane >= o) c2 += v;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = c2;
    __syncthreads();
    unsigned long long all = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k == warp) c2 += all;
      all += sh.part[k];
    }
    if (w != 0 && before + c2 > goal) atomicMin(&sh.token, i);
    before += all;
    if (before > goal) break;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int tok = sh.token;
    a.token[b] = tok;
    const double zt = (static_cast<double>(clean(load_logit(row.x + tok))) - static_cast<double>(top)) / static_cast<double>(temp == 0.0f ? 1.0f : temp);
    const double unit = static_cast<double>(62 - a.shift) * 0.69314718055994530942;
    if (a.logp) a.logp[b] = static_cast<float>(zt - (log(static_cast<double>(z)) - unit));
    if (a.logp_kept) a.logp_kept[b] = static_cast<float>(zt - (log(static_cast<double>(mass)) - unit));
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, bool f32, cudaStream_t st) {
  return launch_pdl(f32 ? sample_kernel<float> : sample_kernel<__nv_bfloat16>, dim3(a.B), dim3(kThreads), 0, st, a);
}

}  // namespace qurl
