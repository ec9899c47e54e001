// rope.cu -- rotary positions: the rotation of query and key heads, alone
// (qurl_rope, forward and inverse) and together with the FP8 quantization of
// keys and values into the paged cache (qurl_rope_kv_cache_quant).
//
// The first rot values of a head are rot / 2 pairs, (i, i + rot / 2) or
// neighbours; pair i of a token at position p is turned by the angle p f_i:
//   (a, b) -> factor (a cos - b sin,  a sin + b cos);    inverse: sin negated.
//
// Angles: in fp32 the product p f_i of a far position loses the angle (2^20
// radians are known to 1/16), and fp64 arithmetic is slow here.  f_i / 2 pi is
// taken as a 64-bit fixed-point fraction of a turn; times p modulo 2^64 the
// whole turns fall away exactly, and the top 32 bits, the signed fraction of a
// turn, go to sincospi in fp32.
//
// Bound by HBM: every value is read and written once.  A CTA takes one token:
// its threads compute each pair's cosine and sine once, in shared memory, while
// the first heads are on their way; then a lane holds the same 8 dimensions of
// every head it meets (groups of lanes per head), with their cosines and sines
// in registers, and gets the other half of a pair from its partner lane.  A
// rotary width whose halves do not fall on vectors of 8 goes through shared
// memory instead.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"
#include "rowquant.cuh"

namespace qurl {
namespace {

using namespace rq;

// How the two values of a pair lie.
constexpr int kHalf = 0;         // i and i + rot / 2, rot a multiple of 16: a lane's 8 values have one partner lane
constexpr int kHalfAny = 1;      // any even rot
constexpr int kInterleaved = 2;  // 2 i and 2 i + 1

constexpr int kInFlight = 4;  // heads a lane loads before it works on the first
constexpr int kMaxThreads = 512;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    o[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// f / 2 pi modulo 1 in units of 2^-64 (a finite f), from the bits of the quotient.
__device__ __forceinline__ uint64_t turns_per_position(double f) {
  const double t = f * 0.15915494309189533577;
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(t));
  const int e = static_cast<int>((bits >> 52) & 0x7FF);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (e != 0 ? 1ull << 52 : 0);
  const int up = e - 1011;  // t = m 2^(e - 1075), in units of 2^-64: m 2^(e - 1011)
  const uint64_t u = up >= 64 || up <= -64 ? 0 : up >= 0 ? m << up : m >> -up;
  return (bits >> 63) != 0 ? 0 - u : u;
}

template <typename T, int LAYOUT, bool CACHE>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 turn[128];                              // (cos, sin) of each pair, times factor
  extern __shared__ float mix[];                            // kHalfAny: a warp's values, 256 each
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.group, sub = lane & (group - 1);      // lanes per head (a power of two), this lane's place
  const int d0 = 8 * sub, hd = a.head_dim, half = a.rot >> 1;
  const bool on = d0 < hd;
  const int per_pass = (blockDim.x >> 5) * (32 / group);
  const int h_first = warp * (32 / group) + lane / group;
  const long long m = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();

  const T* src = static_cast<const T*>(a.x) + m * a.ldx + d0;
  T* dst = static_cast<T*>(a.out) + m * a.ldo + d0;
  const int heads = CACHE ? a.heads + 2 * a.kv_heads : a.heads;
  const int turned = CACHE ? a.heads + a.kv_heads : a.heads;
  const int p = __ldg(a.positions + m);
  long long slot = -1;
  if constexpr (CACHE) {
    slot = __ldg(a.slots + m);
    if (slot >= a.num_slots) {
      if (tid == 0) latch_bad_index(a.status);
      slot = -1;
    }
  }
  float x[kInFlight][8];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int h = h0 + u * per_pass;
      if (on && h < heads) load8(src + static_cast<long long>(h) * hd, x[u]);
    }
  };
  fetch(h_first);
  for (int i = tid; i < half; i += blockDim.x) {
    const uint64_t at = static_cast<uint64_t>(static_cast<long long>(p)) * turns_per_position(a.inv_freq[i]);
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
  __syncthreads();
  float co[8], si[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    const int i = LAYOUT == kInterleaved ? d >> 1 : d < half ? d : d - half;
    const float2 t = d < a.rot ? turn[i] : make_float2(1.0f, 0.0f);
    co[e] = t.x;
    // what the other value of the pair is multiplied with
    si[e] = (LAYOUT == kInterleaved ? (d & 1) == 0 : d < half) ? -t.y : t.y;
  }
  const int partner = LAYOUT == kHalf ? (d0 < half ? lane + (half >> 3) : d0 < a.rot ? lane - (half >> 3) : lane) : 0;

  for (int h0 = h_first; h0 - h_first < heads; h0 += kInFlight * per_pass) {  // (the same turns for every lane)
    if (h0 != h_first) fetch(h0);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int h = h0 + u * per_pass;
      if (h - h_first >= heads) break;
      float y[8], z[8];
      if constexpr (LAYOUT == kHalf) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(0xFFFFFFFFu, x[u][e], partner);
      } else if constexpr (LAYOUT == kHalfAny) {
        float* row = mix + warp * 256 + (lane - sub) * 8;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) row[d0 + e] = x[u][e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          z[e] = d < half ? row[d + half] : d < a.rot ? row[d - half] : 0.0f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = x[u][e ^ 1];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = h < turned && d0 + e < a.rot ? fmaf(x[u][e], co[e], z[e] * si[e]) : x[u][e];
      if (!CACHE || h < a.heads) {
        if (on && h < heads) store8(dst + static_cast<long long>(h) * hd, y);
      }
      if constexpr (CACHE) {
        // (a warp whose heads are all queries has nothing to quantize)
        if (__any_sync(0xFFFFFFFFu, h >= a.heads && h < heads) && slot >= 0) {
          float top = 0.0f;
          if (on)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
          for (int o = 1; o < group; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          if (h >= a.heads && h < heads) {
            const int kv = h - a.heads, value = kv >= a.kv_heads;
            // (a head so small that its step would be 0 is a head of zeros)
            const Enc en = make_enc(top >= 0x1p-140f ? top : 0.0f, kQFp8);
            const long long at = slot * a.kv_heads + (value ? kv - a.kv_heads : kv);
            if (on) {
              if (top < 0x1p-140f)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = 0.0f;
              *reinterpret_cast<uint2*>((value ? a.v_cache : a.k_cache) + at * hd + d0) = encode8(y, en);
            }
            if (sub == 0) (value ? a.v_scale : a.k_scale)[at] = en.scale;
          }
        }
      }
    }
  }
}

template <typename T, bool CACHE>
cudaError_t launch_typed(const RopeArgs& a, int threads, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.M)), block(static_cast<unsigned>(threads));
  if (a.interleaved) return launch_pdl(rope_kernel<T, kInterleaved, CACHE>, grid, block, 0, st, a);
  if (a.rot % 16 == 0) return launch_pdl(rope_kernel<T, kHalf, CACHE>, grid, block, 0, st, a);
  return launch_pdl(rope_kernel<T, kHalfAny, CACHE>, grid, block, static_cast<size_t>(threads) * 32, st, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, bool f32, bool cache, int num_sms, cudaStream_t st) {
  RopeArgs a = args;
  a.group = 2;
  while (a.group * 8 < a.head_dim) a.group *= 2;
  const int heads = a.heads + (cache ? 2 * a.kv_heads : 0);
  // few tokens: a warp for every group of heads; many: about kInFlight heads a lane
  const int warps = (heads + 32 / a.group - 1) / (32 / a.group);
  const int per = a.M <= num_sms ? 1 : kInFlight;
  int threads = 32 * ((warps + per - 1) / per);
  threads = threads < 64 ? 64 : threads > kMaxThreads ? kMaxThreads : threads;
  if (cache) return launch_typed<__nv_bfloat16, true>(a, threads, st);
  return f32 ? launch_typed<float, false>(a, threads, st) : launch_typed<__nv_bfloat16, false>(a, threads, st);
}

}  // namespace qurl
