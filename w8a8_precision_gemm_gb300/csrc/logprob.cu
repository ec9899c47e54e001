// logprob.cu -- log-probabilities of given tokens under a row of logits, and
// the logits' gradient: what the ACR objective reads (logp of the trained and
// of the proximal policy) and where its derivative goes.
//
//   z = x / temperature,  lse = log sum_v exp(z_v),  logp = z_target - lse
//   dx_v = scale * g / (denom * temperature) * (1[v = target] - exp(z_v - lse))
//
// Both directions stream the logits once (2 or 4 bytes in per value; the
// gradient writes as many), so HBM bounds them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qurl {
namespace {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// A running maximum m (of x) and sum s of exp((x - m) / temperature).
struct Lse {
  float m, s;
};

// Joins two of them; an empty part has m = -inf.
__device__ __forceinline__ Lse join(Lse a, Lse b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == -INFINITY ? 0.0f : m;
  return {m, a.s * ex2((a.m - ref) * c) + b.s * ex2((b.m - ref) * c)};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprob_kernel(const T* __restrict__ X, int V, long long ld,
                                                                 const long long* __restrict__ targets, float inv_t,
                                                                 float* __restrict__ logp, float* __restrict__ lse_out,
                                                                 int* status) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Vec<T>::N;
  const int t = blockIdx.x;
  const long long target = targets[t];
  if (target < 0 || target >= V) {  // padding; past the vocabulary: reported
    if (threadIdx.x == 0) {
      logp[t] = 0.0f;
      lse_out[t] = 0.0f;
      if (target >= V) atomicCAS(status, kDevOk, kDevBadIndex);
    }
    return;
  }
  const T* row = X + static_cast<long long>(t) * ld;
  const float c = kLog2e * inv_t;
  Lse a{-INFINITY, 0.0f};
  const int nvec = V / N;
  for (int i = threadIdx.x; i < nvec; i += kThreads) {
    float x[N];
    Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(row) + i), x);
    float m = a.m;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[e]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = a.s * ex2((a.m - ref) * c);
#pragma unroll
    for (int e = 0; e < N; ++e) s += ex2((x[e] - ref) * c);
    a = {m, s};
  }
  for (int i = nvec * N + threadIdx.x; i < V; i += kThreads) a = join(a, {Vec<T>::one(row + i), 1.0f}, c);
  __shared__ Lse part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, {__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)}, c);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) a = join(a, part[w], c);
    const float xt = Vec<T>::one(row + target);
    const float ls = logf(a.s);
    // nothing in the row: no probability anywhere
    logp[t] = a.m == -INFINITY ? -INFINITY : (xt - a.m) * inv_t - ls;
    lse_out[t] = a.m == -INFINITY ? -INFINITY : a.m * inv_t + ls;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprob_grad_kernel(const T* X, int V, long long ld, long long rows,
                                                                      const long long* __restrict__ targets,
                                                                      float inv_t, const float* __restrict__ lse,
                                                                      const float* __restrict__ g, float scale,
                                                                      const double* __restrict__ denom, T* dX,
                                                                      long long ldd, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Vec<T>::N;
  double w0 = static_cast<double>(scale) * inv_t;
  if (denom) {
    const double d = *denom;
    w0 = d > 0.0 ? w0 / d : 0.0;
  }
  const int nvec = V / N;
  for (long long t = blockIdx.x; t < rows; t += gridDim.x) {
    const long long target = targets[t];
    const bool ok = target >= 0 && target < V;
    if (target >= V && threadIdx.x == 0) atomicCAS(status, kDevOk, kDevBadIndex);
    const float l = lse[t];
    const float w = ok && l != -INFINITY ? static_cast<float>(w0 * g[t]) : 0.0f;
    const T* row = X + t * ld;
    T* out = dX + t * ldd;
    for (int i = threadIdx.x; i < nvec; i += kThreads) {
      float x[N];
      if (w != 0.0f) {
        Vec<T>::unpack(reinterpret_cast<const uint4*>(row)[i], x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float p = ex2((x[e] * inv_t - l) * kLog2e);
          x[e] = w * ((i * N + e == target ? 1.0f : 0.0f) - p);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = 0.0f;
      }
      reinterpret_cast<uint4*>(out)[i] = Vec<T>::pack(x);
    }
    for (int i = nvec * N + threadIdx.x; i < V; i += kThreads) {
      const float p = w != 0.0f ? ex2((Vec<T>::one(row + i) * inv_t - l) * kLog2e) : 0.0f;
      Vec<T>::put(out + i, w != 0.0f ? w * ((i == target ? 1.0f : 0.0f) - p) : 0.0f);
    }
  }
}

}  // namespace

cudaError_t launch_token_logprob(const void* X, bool f32, long long T, int V, long long ld, const long long* targets,
                                 float inv_t, float* logp, float* lse, int* status, cudaStream_t st) {
  if (f32)
    return launch_pdl(token_logprob_kernel<float>, dim3(static_cast<unsigned>(T)), dim3(kThreads), 0, st,
                      reinterpret_cast<const float*>(X), V, ld, targets, inv_t, logp, lse, status);
  return launch_pdl(token_logprob_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(T)), dim3(kThreads), 0, st,
                    reinterpret_cast<const __nv_bfloat16*>(X), V, ld, targets, inv_t, logp, lse, status);
}

cudaError_t launch_token_logprob_grad(const void* X, bool f32, long long T, int V, long long ld,
                                      const long long* targets, float inv_t, const float* lse, const float* g,
                                      float scale, const double* denom, void* dX, long long ldd, int num_sms,
                                      int* status, cudaStream_t st) {
  const long long cap = 4LL * num_sms;
  const unsigned grid = static_cast<unsigned>(T < cap ? T : cap);
  if (f32)
    return launch_pdl(token_logprob_grad_kernel<float>, dim3(grid), dim3(kThreads), 0, st,
                      reinterpret_cast<const float*>(X), V, ld, T, targets, inv_t, lse, g, scale, denom,
                      reinterpret_cast<float*>(dX), ldd, status);
  return launch_pdl(token_logprob_grad_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, st,
                    reinterpret_cast<const __nv_bfloat16*>(X), V, ld, T, targets, inv_t, lse, g, scale, denom,
                    reinterpret_cast<__nv_bfloat16*>(dX), ldd, status);
}

}  // namespace qurl
