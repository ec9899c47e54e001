// residual.cu -- the residual update between two blocks of a layer, fused with
// the norms on both sides of it and the next projection's quantizer:
//
//   n  = y                          or (y * r_y) * gamma_post   (RMSNorm of the block's output)
//   t  = n * gate                   (per channel or per token and channel; optional)
//   h' = bf16_RNE(h + t * rs)       (the residual stream, stored)
//   v  = (h' * r_h) * gamma'        (the next block's RMSNorm, UAQ-folded gain)
//   codes, sx = per-token quantization of v
//
// Each product and sum is rounded to fp32 as written; r = 1 / sqrt(ms + eps)
// with ms by the RMSNorm quantizer's rule (the sum of squares as an error-free
// pair, the mean rounded once).  The second half works on the stored bf16 h', so
// its codes are those of qurl_rmsnorm_quant(h') (where the two sums' 2^-44 round
// to the same ms).
//
// Bytes: 2 (y) + 2 (h) + 2 (h') + 1 (codes) per value, against 13 for the three
// passes (norm, update, norm and quantize) it stands for.  One row per CTA, the
// row kept in registers from its only read to the codes.  8192 x 5120 FP8 with
// both norms: 70 us, 4.2 TB/s, 0.62 of the copy rate; three dependent block
// reductions a row (both means and the absmax are chains of barriers that loads of
// other rows on the SM cover only in part) and the issue slots (84
// instructions a pair of values, 63% of them taken) bound it.  64 x 5120 INT8, one
// call after the other in a graph: 4.0 us, the chain of one row (qurl_rmsnorm_quant
// alone 4.0).  Rows of more than 8192 (a CTA of 512 threads, the rest of the row read
// again): 8192 x 27648 INT8 529 us with both norms, 433 without the one behind the
// block (234 at the copy rate), 64 x 27648 10.6 and 8.8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"
#include "rowquant.cuh"

namespace qurl {
namespace {

using namespace rq;

constexpr int kNC = 8;        // 16-byte vectors cached per thread
constexpr int kThreads = 512;  // threads of a long row

struct ResidualArgs {
  const __nv_bfloat16* Y;
  const __nv_bfloat16* H;
  const __nv_bfloat16* gate;  // null: 1
  __nv_bfloat16* Hout;
  const float* gamma_post;  // null: no norm behind the block
  const float* gamma;
  long long ldy, ldh, ldg, ldo;
  float eps_post, rs, eps;
  int K, qt;
  uint8_t* Xq;
  float* sx;
  float* ms_out;
};

// h + ((y normalised) * gate) * rs of 8 values, rounded to bf16.
__device__ __forceinline__ uint4 update8(const ResidualArgs& a, const uint4 yu, const uint4 hu, const uint4* grow, int idx,
                                         float2 r2, float2 rs2) {
  float2 n[4], h[4];
  if (a.gamma_post)
    norm8(yu, reinterpret_cast<const float4*>(a.gamma_post), idx, r2, n);
  else
    bf16x8_to_f2(yu, n);
  if (grow) {
    float2 g[4];
    bf16x8_to_f2(__ldg(grow + idx), g);
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = mul2(n[e], g[e]);
  }
  bf16x8_to_f2(hu, h);
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // (scalar products and sums: the paired ones were seen to join into an FMA here)
    const float sx = __fadd_rn(h[e].x, __fmul_rn(n[e].x, rs2.x));
    const float sy = __fadd_rn(h[e].y, __fmul_rn(n[e].y, rs2.y));
    const __nv_bfloat162 p = __floats2bfloat162_rn(sx, sy);
    o[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Block reductions of the row kernel: each has scratch of its own, so nothing
// has to be read before the next one may write (one barrier fewer than the
// shared ones), and the maximum, which a warp reduces in one instruction, is
// taken by every warp itself (another one fewer).
struct RmsScratch {
  float part[2 * (1024 / 32)];
  float ms, r;
};

// (s + c) / K rounded to fp32 and 1 / sqrt(ms + eps), as mean_sq gives them, with
// the quotient as an fp32 pair (2^-47) instead of in fp64 (2^-52): the fp64
// division is a chain of slow instructions that a whole block waits for.
__device__ __forceinline__ void mean_sq_pair(float s, float c, int K, float eps, float& ms, float& r) {
  const float k = static_cast<float>(K);  // exact: these rows have at most 1024 vectors
  float lo = 0.0f, hi = s;
  two_sum_acc(hi, lo, c);
  const float q = __fdiv_rn(hi, k);
  ms = __fadd_rn(q, __fdiv_rn(__fadd_rn(__fmaf_rn(-q, k, hi), lo), k));
  r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, eps)));
}

template <int NC, bool kOwn>
__device__ __forceinline__ void row_rms_once(const uint4* row, int K, const uint4 (&cache)[NC], const float4* gain, float eps,
                                             RmsScratch& sh, float& ms, float& r) {
  float s, c;
  row_sum_sq<NC, kOwn>(row, K, cache, gain, s, c);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  warp_pair_sum(s, c);
  if (lane == 0) {
    sh.part[2 * warp] = s;
    sh.part[2 * warp + 1] = c;
  }
  __syncthreads();
  if (warp == 0) {
    s = lane < nw ? sh.part[2 * lane] : 0.0f;
    c = lane < nw ? sh.part[2 * lane + 1] : 0.0f;
    warp_pair_sum(s, c);
    if (lane == 0) mean_sq_pair(s, c, K, eps, sh.ms, sh.r);
  }
  __syncthreads();
  ms = sh.ms;
  r = sh.r;
}

__device__ __forceinline__ float warp_fmax(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float block_max_once(float v, float* part) {
  v = warp_fmax(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_fmax(lane < (blockDim.x >> 5) ? part[lane] : 0.0f);
}

// One row per CTA.  NC: vectors a thread holds; KEEP: they are all of the row
// (no thread has more), and the normalised values stay in registers between the
// absmax and the codes instead of being computed twice.
template <int NC, bool KEEP, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) residual_rmsnorm_quant_kernel(const ResidualArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ RowScratch sh;
  __shared__ RmsScratch rms[2];
  __shared__ float top[32];
  const int m = blockIdx.x;
  const uint4* yrow = reinterpret_cast<const uint4*>(a.Y + static_cast<size_t>(m) * a.ldy);
  const uint4* hrow = reinterpret_cast<const uint4*>(a.H + static_cast<size_t>(m) * a.ldh);
  const uint4* grow = a.gate ? reinterpret_cast<const uint4*>(a.gate + static_cast<size_t>(m) * a.ldg) : nullptr;
  uint4* orow = reinterpret_cast<uint4*>(a.Hout + static_cast<size_t>(m) * a.ldo);
  const int nvec = a.K >> 3;
  // h is read by plain loads: h_out may be the same rows
  uint4 yc[NC], hc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = threadIdx.x + c * blockDim.x;
    if (idx < nvec) {
      yc[c] = __ldg(yrow + idx);
      hc[c] = hrow[idx];
    }
  }
  float2 r2 = splat2(1.0f);
  if (a.gamma_post) {
    float ms, r;
    row_rms_once<NC, false>(yrow, a.K, yc, reinterpret_cast<const float4*>(a.gamma_post), a.eps_post, rms[0], ms, r);
    r2 = splat2(r);
  }
  const float2 rs2 = splat2(a.rs);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = threadIdx.x + c * blockDim.x;
    if (idx < nvec) orow[idx] = hc[c] = update8(a, yc[c], hc[c], grow, idx, r2, rs2);
  }
  if constexpr (!KEEP) {
    for (int idx = threadIdx.x + NC * blockDim.x; idx < nvec; idx += blockDim.x)
      orow[idx] = update8(a, __ldg(yrow + idx), hrow[idx], grow, idx, r2, rs2);
    const CodeSums none{};
    rmsnorm_quant_cached<NC, true>(m, orow, hc, a.K, a.gamma, a.eps, a.qt, a.Xq, a.sx, a.ms_out, nullptr, none, sh);
  } else {
    const float4* g4 = reinterpret_cast<const float4*>(a.gamma);
    float ms, r;
    row_rms_once<NC, true>(orow, a.K, hc, g4, a.eps, rms[1], ms, r);
    if (threadIdx.x == 0 && a.ms_out) a.ms_out[m] = ms;
    r2 = splat2(r);
    float2 v[NC][4];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int idx = threadIdx.x + c * blockDim.x;
      if (idx >= nvec) continue;
      norm8(hc[c], g4, idx, r2, v[c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(v[c][e].x), fabsf(v[c][e].y)));
    }
    amax = block_max_once(amax, top);
    const Enc en = make_enc(amax, a.qt);
    if (threadIdx.x == 0) a.sx[m] = en.scale;
    uint8_t* out = a.Xq + static_cast<size_t>(m) * a.K;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int idx = threadIdx.x + c * blockDim.x;
      if (idx < nvec) store8(out, nullptr, idx, v[c], en);
    }
  }
}

}  // namespace

cudaError_t launch_residual_rmsnorm_quant(const void* Y, long long ldy, const float* gamma_post, float eps_post,
                                          const void* gate, long long ldg, float rs, const void* H, long long ldh,
                                          void* Hout, long long ldo, const float* gamma, float eps, int M, int K,
                                          int qt, void* Xq, float* sx, float* ms_out, int num_sms, cudaStream_t st) {
  ResidualArgs a{};
  a.Y = reinterpret_cast<const __nv_bfloat16*>(Y);
  a.H = reinterpret_cast<const __nv_bfloat16*>(H);
  a.gate = reinterpret_cast<const __nv_bfloat16*>(gate);
  a.Hout = reinterpret_cast<__nv_bfloat16*>(Hout);
  a.gamma_post = gamma_post;
  a.gamma = gamma;
  a.ldy = ldy;
  a.ldh = ldh;
  a.ldg = ldg;
  a.ldo = ldo;
  a.eps_post = eps_post;
  a.rs = rs;
  a.eps = eps;
  a.K = K;
  a.qt = qt;
  a.Xq = reinterpret_cast<uint8_t*>(Xq);
  a.sx = sx;
  a.ms_out = ms_out;
  const int nvec = K / 8;
  auto threads = [&](int nc) { return dim3(static_cast<unsigned>(((nvec + nc - 1) / nc + 31) / 32 * 32)); };
  // Few rows, all of them at once on the GPU (two an SM, or one of more than 640
  // vectors): a vector a thread, the shortest chain; 304 rows of 5120 5.0 us, 7.2 the
  // other way; 256 of 8192, past one row an SM, 9.3 and 7.3.  (640 threads is where the
  // variant of two an SM was built and measured; between that and 1024 it was not.)
  // Else four vectors a thread: fewer warps wait at each reduction.  8192 x 5120 (FP8,
  // both norms), us at resident CTAs: 1 vector 116 (2), 108 (3); 2 vectors 90 (3),
  // 80 (4); 3 vectors 73 (5); 4 vectors 73 (5), 71 (6), 70 (7), 75 (8); 5 vectors
  // 72 (6), 70 (8).  8192 x 8192 (103 to 107 us, 77 without the norm behind the block;
  // 69 at the copy rate): 4 vectors 118 (3), 103 (4), 109 (5); 5 vectors 105 (4), 112
  // (5).  Persistent CTAs that load the next row into the registers the current one
  // leaves free measured 85 or more: the registers cost more resident rows than the
  // early loads gain.
  if (M <= 2 * num_sms && nvec <= 640)
    return launch_pdl(residual_rmsnorm_quant_kernel<1, true, 640, 2>, dim3(M), threads(1), 0, st, a);
  if (M <= num_sms && nvec <= 1024)
    return launch_pdl(residual_rmsnorm_quant_kernel<1, true, 1024, 1>, dim3(M), threads(1), 0, st, a);
  if (nvec <= 4 * 160) return launch_pdl(residual_rmsnorm_quant_kernel<4, true, 160, 7>, dim3(M), threads(4), 0, st, a);
  if (nvec <= 4 * 256) return launch_pdl(residual_rmsnorm_quant_kernel<4, true, 256, 4>, dim3(M), threads(4), 0, st, a);
  return launch_pdl(residual_rmsnorm_quant_kernel<kNC, false, kThreads, 1>, dim3(M), dim3(kThreads), 0, st, a);
}

}  // namespace qurl
