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
// turn, go to sincospi in fp32 (for fp32 rows less the nearest quarter, which keeps two more bits).
//
// Bound by HBM: every value is read and written once.  A warp takes some heads of a token (all of them where there are
// many tokens), then the same of a later token: a lane holds the same 8 dimensions of every head it meets (groups of
// lanes per head), so that it turns them by angles that it computes itself, 8 a token, from the turns per position of each
// pair, which a CTA works out once.  No warp waits for another.  The other half of a pair comes from the partner lane; a
// rotary width whose halves do not fall on vectors of 8 goes through shared memory instead.
//
// Measured (GB300): 8192 tokens of 48 heads of 128 in bf16, 201 MB: 36 us, 5.5 TB/s; with the cache, 8192 tokens of 40 + 8 + 8
// heads, 218 MB: 59 us, 3.7 TB/s, where instructions bound it (0.67 of a scheduler's slots issue: the 16 quantized heads of
// a token take as many as its 40 others).  A CTA for each token, its angles in shared memory, took 75 and 108 us; turns kept
// in registers 38 and 61.  At 80 registers (kResident) six of the nine instances spill 8 to 44 bytes, the two measured here 12 and 20.
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

constexpr int kInFlight = 4;  // vectors a lane loads before it works on the first
constexpr int kThreads = 256;
constexpr int kResident = 3;  // CTAs of an SM (4: 39 and 62 us)

// 8 values as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float2 (&x)[4]) const { bf16x8_to_f2(v, x); }
  __device__ __forceinline__ Raw from(int lane) const {
    return {make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, lane), __shfl_sync(0xFFFFFFFFu, v.y, lane),
                       __shfl_sync(0xFFFFFFFFu, v.z, lane), __shfl_sync(0xFFFFFFFFu, v.w, lane))};
  }
};
template <>
struct Raw<float> {
  float4 u, v;
  __device__ __forceinline__ void load(const float* p) {
    u = reinterpret_cast<const float4*>(p)[0];
    v = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void values(float2 (&x)[4]) const {
    x[0] = make_float2(u.x, u.y), x[1] = make_float2(u.z, u.w);
    x[2] = make_float2(v.x, v.y), x[3] = make_float2(v.z, v.w);
  }
  __device__ __forceinline__ Raw from(int lane) const {
    auto get = [&](float a) { return __shfl_sync(0xFFFFFFFFu, a, lane); };
    return {make_float4(get(u.x), get(u.y), get(u.z), get(u.w)), make_float4(get(v.x), get(v.y), get(v.z), get(v.w))};
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&x)[4]) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __float22bfloat162_rn(x[e]);
    o[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(float* p, const float2 (&x)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
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

// Sine and cosine of `at` units of 2^-32 of a turn (signed).  fp32 has 24 bits for them, 2^-26 of a turn; where the results are
// rounded to 8 bits or fewer that is enough.  FINE (fp32 rows): what is left of the nearest quarter of a turn, 2^-28.
template <bool FINE>
__device__ __forceinline__ void sine_cosine(uint32_t at, float& s, float& c) {
  if constexpr (!FINE) {
    sincospif(static_cast<float>(static_cast<int>(at)) * 0x1p-31f, &s, &c);
  } else {
    const uint32_t quarter = (at + 0x20000000u) >> 30;
    float u, v;
    sincospif(static_cast<float>(static_cast<int>(at - (quarter << 30))) * 0x1p-31f, &u, &v);
    s = (quarter & 1) != 0 ? v : u;
    c = (quarter & 1) != 0 ? u : v;
    if ((quarter & 2) != 0) s = -s;
    if (((quarter + 1) & 2) != 0) c = -c;
  }
}

template <typename T, int LAYOUT, bool CACHE>
__global__ void __launch_bounds__(kThreads, kResident) rope_kernel(const RopeArgs a) {
  __shared__ uint64_t turns[128];                           // per position, of each pair
  extern __shared__ float mix[];                            // kHalfAny: a warp's values, 256 each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group, sub = lane & (group - 1);      // lanes per head (a power of two), this lane's place
  const int d0 = 8 * sub, hd = a.head_dim, half = a.rot >> 1;
  const bool on = d0 < hd;
  const int per_pass = 32 / group;                          // heads of a warp side by side
  const int heads = CACHE ? a.heads + 2 * a.kv_heads : a.heads;
  const int turned = CACHE ? a.heads + a.kv_heads : a.heads;
  const int passes = (heads + per_pass - 1) / per_pass, passes_per_part = (passes + a.parts - 1) / a.parts;
  const int partner = LAYOUT == kHalf ? (d0 < half ? lane + (half >> 3) : d0 < a.rot ? lane - (half >> 3) : lane) : 0;
  griddep_wait();
  griddep_launch_dependents();

  constexpr int kPairs = LAYOUT == kInterleaved ? 4 : 8;    // pairs that this lane's values belong to
  const int pair0 = LAYOUT == kInterleaved ? d0 >> 1 : d0 < half ? d0 : d0 - half;
  for (int i = threadIdx.x; i < 128; i += kThreads) turns[i] = i < half ? turns_per_position(a.inv_freq[i]) : 0;
  __syncthreads();
  const long long items = a.M * a.parts, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp; item < items; item += step) {
    // (the tokens' last heads first: keys and values take longer)
    const int part = static_cast<int>(item / a.M);
    const long long m = item - part * a.M;
    const int first = (a.parts - 1 - part) * passes_per_part, last = min(first + passes_per_part, passes);
    const T* src = static_cast<const T*>(a.x) + m * a.ldx + d0;
    T* dst = static_cast<T*>(a.out) + m * a.ldo + d0;
    Raw<T> x[kInFlight];
    auto fetch = [&](int pass) {
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int h = (pass + u) * per_pass + lane / group;
        if (on && pass + u < last && h < heads) x[u].load(src + static_cast<long long>(h) * hd);
      }
    };
    fetch(first);
    const int p = __ldg(a.positions + m);
    long long slot = -1;
    if constexpr (CACHE) {
      slot = __ldg(a.slots + m);
      if (slot >= a.num_slots) {
        if (lane == 0) latch_bad_index(a.status);
        slot = -1;
      }
    }
    float2 co[4], si[4];  // si: what the other value of the pair is multiplied with
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      // the top 32 bits of p times the turns, modulo 2^64
      int i = pair0 + e;
      if (LAYOUT == kHalfAny && d0 < half && i >= half) i -= half;  // (the halves' border within this lane's values)
      const uint64_t per = turns[i & 127];
      const uint32_t pu = static_cast<uint32_t>(p), low = static_cast<uint32_t>(per);
      const uint32_t at = __umulhi(pu, low) + pu * static_cast<uint32_t>(per >> 32) - (p < 0 ? low : 0);
      float s, c;
      sine_cosine<sizeof(T) == 4>(at, s, c);
      c *= a.factor;
      s = (a.inverse ? -s : s) * a.factor;
      if constexpr (LAYOUT == kInterleaved) {
        co[e] = make_float2(c, c);
        si[e] = make_float2(-s, s);
      } else {
        if (d0 + e < half) s = -s;
        (e & 1 ? co[e >> 1].y : co[e >> 1].x) = c;
        (e & 1 ? si[e >> 1].y : si[e >> 1].x) = s;
      }
    }

    for (int pass = first; pass < last; pass += kInFlight) {
      if (pass != first) fetch(pass);
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (pass + u >= last) break;
        const int h = (pass + u) * per_pass + lane / group;
        float2 v[4], y[4];
        x[u].values(v);
        if (CACHE && (pass + u) * per_pass >= turned) {  // values only
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = v[e];
        } else {
          float2 z[4];
          if constexpr (LAYOUT == kHalf) {
            x[u].from(partner).values(z);
          } else if constexpr (LAYOUT == kHalfAny) {
            float* row = mix + warp * 256 + (lane - sub) * 8;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(row + d0 + 2 * e) = v[e];
            __syncwarp();
            auto other = [&](int d) { return d < half ? row[d + half] : d < a.rot ? row[d - half] : 0.0f; };
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = make_float2(other(d0 + 2 * e), other(d0 + 2 * e + 1));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = make_float2(v[e].y, v[e].x);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = __ffma2_rn(v[e], co[e], __fmul2_rn(z[e], si[e]));
          if (a.rot < hd) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (d0 + 2 * e >= a.rot) y[e] = v[e];
            }
          }
          if (CACHE && (pass + u + 1) * per_pass > turned) {  // the last keys beside the first values
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (h >= turned) y[e] = v[e];
            }
          }
        }
        if (!CACHE || h < a.heads) {
          if (on && h < heads) store8(dst + static_cast<long long>(h) * hd, y);
        }
        if constexpr (CACHE) {
          // (where all heads are queries there is nothing to quantize)
          if ((pass + u + 1) * per_pass > a.heads && slot >= 0) {
            float top = 0.0f;
            if (on)
#pragma unroll
              for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              if (o < group) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            }
            if (h >= a.heads && h < heads) {
              const int kv = h - a.heads, value = kv >= a.kv_heads;
              // (a head so small that its step would be 0 is a head of zeros, but for what is no number: `top` passes that over)
              const Enc en = make_enc(top >= 0x1p-140f ? top : 0.0f, kQFp8);
              const long long at = slot * a.kv_heads + (value ? kv - a.kv_heads : kv);
              if (on) {
                if (top < 0x1p-140f)
#pragma unroll
                  for (int e = 0; e < 4; ++e) y[e] = make_float2(isnan(y[e].x) ? y[e].x : 0.0f, isnan(y[e].y) ? y[e].y : 0.0f);
                *reinterpret_cast<uint2*>((value ? a.v_cache : a.k_cache) + at * hd + d0) = encode8_f8(y, en);
              }
              if (sub == 0) (value ? a.v_scale : a.k_scale)[at] = en.scale;
            }
          }
        }
      }
    }
  }
}

template <typename T, bool CACHE>
cudaError_t launch_typed(const RopeArgs& a, int grid, cudaStream_t st) {
  if (a.interleaved) return launch_pdl(rope_kernel<T, kInterleaved, CACHE>, dim3(grid), dim3(kThreads), 0, st, a);
  if (a.rot % 16 == 0) return launch_pdl(rope_kernel<T, kHalf, CACHE>, dim3(grid), dim3(kThreads), 0, st, a);
  return launch_pdl(rope_kernel<T, kHalfAny, CACHE>, dim3(grid), dim3(kThreads), static_cast<size_t>(kThreads) * 32, st, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, bool f32, bool cache, int num_sms, cudaStream_t st) {
  RopeArgs a = args;
  a.group = 2;
  while (a.group * 8 < a.head_dim) a.group *= 2;
  const int heads = a.heads + (cache ? 2 * a.kv_heads : 0), passes = (heads + 32 / a.group - 1) / (32 / a.group);
  const long long warps = static_cast<long long>(num_sms) * kResident * (kThreads / 32);
  // (the angles of an item cost about as much as three passes; the last round of items may leave warps without one)
  a.parts = 1;
  long long best = -1;
  for (int parts = 1; parts <= passes && parts <= 256; ++parts) {
    const long long cost = (a.M * parts + warps - 1) / warps * ((passes + parts - 1) / parts + 3);
    if (best < 0 || cost < best) {
      best = cost;
      a.parts = parts;
    }
  }
  const int per_part = (passes + a.parts - 1) / a.parts;
  a.parts = (passes + per_part - 1) / per_part;  // (none is empty)
  const long long ctas = (a.M * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = static_cast<int>(ctas < num_sms * kResident ? ctas : num_sms * kResident);
  if (cache) return launch_typed<__nv_bfloat16, true>(a, grid, st);
  return f32 ? launch_typed<float, false>(a, grid, st) : launch_typed<__nv_bfloat16, false>(a, grid, st);
}

}  // namespace qurl
