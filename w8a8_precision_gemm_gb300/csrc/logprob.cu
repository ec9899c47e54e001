// logprob.cu -- log-probabilities of given tokens under a row of logits, and
// the logits' gradient: what the ACR objective reads (logp of the trained and
// of the proximal policy) and where its derivative goes.
//
//   z = x / temperature,  lse = log sum_v exp(z_v),  logp = z_target - lse
//   dx_v = scale * g / (denom * temperature) * (1[v = target] - exp(z_v - lse))
//
// Both directions stream the logits once (2 or 4 bytes in per value; the
// gradient writes as many), so HBM bounds them: 4096 rows of 131072 bf16 logits 154 us
// forward (7.0 TB/s, a little above the copy rate: reads alone), 336 us the gradient
// (6.4 TB/s, 0.94 of it).  93 rows of 50001 fp32 values, both: 13.5 us on the device,
// the two kernels' start and end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"

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

// One row per cluster: its CTAs take equal slices, the first one joins them.  U:
// unrolled vectors a thread, MINB: resident CTAs (4096 rows of 131072 bf16 logits,
// us at U, MINB: 1, 4 179; 2, 3 169; 4, 3 161; 4, 4 156; 93 rows of 50001 fp32 in
// clusters of 2: 4, 4 7.0; 8, 1 6.0).
template <typename T, int U, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) token_logprob_kernel(const T* __restrict__ X, int V, long long ld,
                                                                 const long long* __restrict__ targets, float inv_t,
                                                                 float* __restrict__ logp, float* __restrict__ lse_out,
                                                                 int cluster, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Vec<T>::N;
  __shared__ Lse part[kThreads / 32], slice[8];
  const int t = blockIdx.x / cluster;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long target = targets[t];
  if (target < 0 || target >= V) {  // padding; past the vocabulary: reported
    if (threadIdx.x == 0 && rank == 0) {
      logp[t] = 0.0f;
      lse_out[t] = 0.0f;
      if (target >= V) latch_bad_index(status);
    }
    return;
  }
  if (cluster > 1) cluster_arrive();  // (the target is the cluster's: all of it or nothing of it comes here)
  const T* row = X + static_cast<long long>(t) * ld;
  const float xt = Vec<T>::one(row + target);
  const float c = kLog2e * inv_t;
  Lse a{-INFINITY, 0.0f};
  const int nvec = V / N;
  const int v0 = static_cast<int>(static_cast<long long>(nvec) * rank / cluster);
  const int v1 = static_cast<int>(static_cast<long long>(nvec) * (rank + 1) / cluster);
#pragma unroll U
  for (int i = v0 + threadIdx.x; i < v1; i += kThreads) {
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
  if (rank == cluster - 1)
    for (int i = nvec * N + threadIdx.x; i < V; i += kThreads) a = join(a, {Vec<T>::one(row + i), 1.0f}, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, {__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)}, c);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    constexpr int W = kThreads / 32;
    a = threadIdx.x < W ? part[threadIdx.x] : Lse{-INFINITY, 0.0f};
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
      a = join(a, {__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)}, c);
  }
  if (cluster > 1) {
    cluster_wait();  // the first CTA runs: its shared memory may be written (the row's reading hides the wait)
    if (threadIdx.x == 0) {
      const uint32_t at = cluster_map(&slice[rank], 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(a.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(a.s) : "memory");
    }
    cluster_sync();
    if (rank != 0) return;
    a = slice[0];
    for (int r = 1; r < cluster; ++r) a = join(a, slice[r], c);
  }
  if (threadIdx.x == 0) {
    const float ls = logf(a.s);
    // nothing in the row: no probability anywhere
    logp[t] = a.m == -INFINITY ? -INFINITY : (xt - a.m) * inv_t - ls;
    lse_out[t] = a.m == -INFINITY ? -INFINITY : a.m * inv_t + ls;
  }
}

// `parts` equal parts of every row, in row order over the grid, four CTAs an SM.
// (Two to eight vectors in flight a thread measured 342 us or more against 335 on
// 4096 rows of 131072 bf16 logits: the stores keep the loads company.)
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    token_logprob_grad_kernel(const T* X, int V, long long ld, long long rows, int parts,
                              const long long* __restrict__ targets, float inv_t, const float* __restrict__ lse,
                              const float* __restrict__ g, float scale, const double* __restrict__ denom, T* dX,
                              long long ldd, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N = Vec<T>::N;
  float w0 = scale * inv_t;
  if (denom) {
    const float d = static_cast<float>(*denom);
    w0 = d > 0.0f ? __fdiv_rn(w0, d) : 0.0f;
  }
  const int nvec = V / N;
  for (long long k = blockIdx.x; k < rows * parts; k += gridDim.x) {
    const long long t = parts == 1 ? k : k / parts;
    const int part = static_cast<int>(k - t * parts);
    const int v1 = static_cast<int>(static_cast<long long>(nvec) * (part + 1) / parts);
    const T* row = X + t * ld;
    T* out = dX + t * ldd;
    const long long target = targets[t];
    if (target >= V && threadIdx.x == 0) latch_bad_index(status);
    const float l = lse[t];
    const float w = target >= 0 && target < V && l != -INFINITY && w0 != 0.0f ? w0 * g[t] : 0.0f;
    const bool live = w != 0.0f;  // (else zeros, whatever the row, lse and, in a row or call that does not count, g hold)
    for (int i = static_cast<int>(static_cast<long long>(nvec) * part / parts) + threadIdx.x; i < v1; i += kThreads) {
      float x[N];
      Vec<T>::unpack(reinterpret_cast<const uint4*>(row)[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float p = ex2((x[e] * inv_t - l) * kLog2e);
        x[e] = live ? w * ((i * N + e == target ? 1.0f : 0.0f) - p) : 0.0f;
      }
      reinterpret_cast<uint4*>(out)[i] = Vec<T>::pack(x);
    }
    if (part == parts - 1)
      for (int i = nvec * N + threadIdx.x; i < V; i += kThreads) {
        const float p = ex2((Vec<T>::one(row + i) * inv_t - l) * kLog2e);
        Vec<T>::put(out + i, live ? w * ((i == target ? 1.0f : 0.0f) - p) : 0.0f);
      }
  }
}

}  // namespace

cudaError_t launch_token_logprob(const void* X, bool f32, long long T, int V, long long ld, const long long* targets,
                                 float inv_t, float* logp, float* lse, int num_sms, int* status, cudaStream_t st) {
  // CTAs a row: as many as two for every SM leave the batch, each with 4096 logits at least
  int cluster = 1;
  while (cluster < 8 && T * cluster * 2 <= 2LL * num_sms && V / (cluster * 2) >= 4096) cluster *= 2;
  const dim3 grid(static_cast<unsigned>(T * cluster));
#define CALL(TYPE, U, B)                                                                                          \
  launch_pdl_cluster(token_logprob_kernel<TYPE, U, B>, cluster, grid, dim3(kThreads), 0, st,                      \
                     reinterpret_cast<const TYPE*>(X), V, ld, targets, inv_t, logp, lse, cluster, status)
  if (cluster > 1) return f32 ? CALL(float, 8, 1) : CALL(__nv_bfloat16, 8, 1);
  return f32 ? CALL(float, 4, 4) : CALL(__nv_bfloat16, 4, 4);
#undef CALL
}

cudaError_t launch_token_logprob_grad(const void* X, bool f32, long long T, int V, long long ld,
                                      const long long* targets, float inv_t, const float* lse, const float* g,
                                      float scale, const double* denom, void* dX, long long ldd, int num_sms,
                                      int* status, cudaStream_t st) {
  // whole rows where they fill the GPU (four CTAs an SM), else each cut into parts of a vector a thread at least
  const long long cap = 4LL * num_sms;
  const int steps = V / (f32 ? 4 : 8) / kThreads + 1;
  const long long want = (cap + T - 1) / T;
  const int parts = static_cast<int>(want < steps ? want : steps);
  const unsigned grid = static_cast<unsigned>(T * parts < cap ? T * parts : cap);
  if (f32)
    return launch_pdl(token_logprob_grad_kernel<float>, dim3(grid), dim3(kThreads), 0, st,
                      reinterpret_cast<const float*>(X), V, ld, T, parts, targets, inv_t, lse, g, scale, denom,
                      reinterpret_cast<float*>(dX), ldd, status);
  return launch_pdl(token_logprob_grad_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, st,
                    reinterpret_cast<const __nv_bfloat16*>(X), V, ld, T, parts, targets, inv_t, lse, g, scale, denom,
                    reinterpret_cast<__nv_bfloat16*>(dX), ldd, status);
}

}  // namespace qurl
