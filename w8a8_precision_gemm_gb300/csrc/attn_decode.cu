// attn_decode.cu -- attention of one new token per sequence over the paged FP8
// key/value cache that qurl_kv_cache_quant fills.
//
//   s_j = scale * ks_j * sum_d q_d k_jd,   p = softmax(s),   o_d = sum_j p_j vs_j v_jd
//
// over the cached tokens j the sequence sees (its last `window` ones, or all).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qurl {
namespace {

constexpr int kWarps = 8;

// One CTA per (sequence, query head); a warp takes every eighth token, its
// lanes the head's dimensions.
__global__ void __launch_bounds__(kWarps * 32) kv_attn_decode_kernel(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads;
  const int h = hq / (a.q_heads / a.kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hd = a.head_dim, per = hd / 16;  // lane d, d + 32, ...
  const long long room = static_cast<long long>(a.max_blocks) * a.block_size;
  long long len = a.seq_lens[b];
  if (len > room) {
    if (threadIdx.x == 0) atomicCAS(a.status, kDevOk, kDevBadIndex);
    len = room;
  }
  const long long first = a.window > 0 && len > a.window ? len - a.window : 0;
  float q[8], acc[8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = lane + 32 * e;
    q[e] = d < hd ? __bfloat162float(a.q[static_cast<long long>(b) * a.ldq + static_cast<long long>(hq) * hd + d]) * a.scale : 0.0f;
  }
  (void)per;
  float m = -INFINITY, l = 0.0f;
  for (long long j = first + warp; j < len; j += kWarps) {
    const int page = a.block_table[static_cast<long long>(b) * a.ld_table + j / a.block_size];
    const long long slot = static_cast<long long>(page) * a.block_size + j % a.block_size;
    if (page < 0 || slot >= a.num_slots) {
      if (lane == 0) atomicCAS(a.status, kDevOk, kDevBadIndex);
      continue;
    }
    const long long at = slot * a.kv_heads + h;
    const __nv_fp8_e4m3* k = reinterpret_cast<const __nv_fp8_e4m3*>(a.k_cache + at * hd);
    const __nv_fp8_e4m3* v = reinterpret_cast<const __nv_fp8_e4m3*>(a.v_cache + at * hd);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = lane + 32 * e;
      if (d < hd) s = fmaf(q[e], static_cast<float>(k[d]), s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.k_scale[at];
    const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn), pv = p * a.v_scale[at];
    l = l * c + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = lane + 32 * e;
      if (d < hd) acc[e] = fmaf(pv, static_cast<float>(v[d]), acc[e] * c);
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) so[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  float mt = -INFINITY, lt = 0.0f, o = 0.0f;
  for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float c = mt == -INFINITY ? 0.0f : expf(sm[w] - mt);
    lt += c * sl[w];
    o += c * so[w][threadIdx.x];
  }
  if (threadIdx.x < hd)
    a.out[static_cast<long long>(b) * a.ldo + static_cast<long long>(hq) * hd + threadIdx.x] =
        __float2bfloat16_rn(lt > 0.0f ? o / lt : 0.0f);
  if (threadIdx.x == 0 && a.lse) a.lse[static_cast<long long>(b) * a.q_heads + hq] = lt > 0.0f ? mt + logf(lt) : -INFINITY;
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, long long, int) { return 256; }

cudaError_t launch_kv_attn_decode(const AttnArgs& a, int, cudaStream_t st) {
  return launch_pdl(kv_attn_decode_kernel, dim3(a.B * a.q_heads), dim3(kWarps * 32), 0, st, a);
}

}  // namespace qurl
