// rollout.h -- declarations shared by the kernels around the quantized linears:
// attention over the FP8 cache, the residual update, the sampler, token
// log-probabilities.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace qurl {

// launch_pdl for a kernel whose CTAs work in clusters of `cluster` (which divides grid.x).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                               cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

#ifdef __CUDACC__
// An index or a parameter that a kernel read and found out of range: reported by
// the next look at the status, in the word that no wait looks at (a wait that ends
// for it would break the handoff of a fused linear, whose counters then stay).
__device__ __forceinline__ void latch_bad_index(int* status) { atomicExch(status + 1, kDevBadIndex); }

// The halves of a cluster barrier that orders no memory: every thread of the
// cluster's CTAs arrives, and has arrived once one of them returns from the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
#endif

// attn_decode.cu: attention of one new token per sequence over the paged FP8 cache
// (qurl_kv_attn_decode), and the workspace it needs.
struct AttnArgs {
  const __nv_bfloat16* q;
  long long ldq;
  int B, q_heads, kv_heads, head_dim;
  const uint8_t* k_cache;
  const float* k_scale;
  const uint8_t* v_cache;
  const float* v_scale;
  long long num_slots;
  const int* block_table;
  long long ld_table;
  int max_blocks, block_size;
  const int* seq_lens;
  int window;
  float scale;
  __nv_bfloat16* out;
  long long ldo;
  float* lse;  // null: not wanted
  void* ws;
  int* status;
};
size_t attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int num_sms);
cudaError_t launch_kv_attn_decode(const AttnArgs& a, int num_sms, cudaStream_t st);

// sample.cu: one token per row of logits from a given uniform number (qurl_sample).
struct SampleArgs {
  const void* logits;
  int B, V;
  long long ld;
  const float* temperature;  // null: 1
  const int* top_k;          // null: off
  const float* top_p;        // null: off
  const float* min_p;        // null: off
  const float* u;
  long long* token;
  float* logp;       // null: not wanted
  float* logp_kept;  // null: not wanted
  int shift;         // ceil(log2 V) + 1, set by the launch
  bool order;        // rows that may take long first, set by the launch
  int* status;
};
cudaError_t launch_sample(const SampleArgs& a, bool f32, int num_sms, cudaStream_t st);

// logprob.cu: log-probabilities of given tokens and the logits' gradient.
cudaError_t launch_token_logprob(const void* X, bool f32, long long T, int V, long long ld, const long long* targets,
                                 float inv_t, float* logp, float* lse, int num_sms, int* status, cudaStream_t st);
cudaError_t launch_token_logprob_grad(const void* X, bool f32, long long T, int V, long long ld,
                                      const long long* targets, float inv_t, const float* lse, const float* g,
                                      float scale, const double* denom, void* dX, long long ldd, int num_sms,
                                      int* status, cudaStream_t st);

// residual.cu: residual update with the norms on both sides and the quantizer behind it.
cudaError_t launch_residual_rmsnorm_quant(const void* Y, long long ldy, const float* gamma_post, float eps_post,
                                          const void* gate, long long ldg, float rs, const void* H, long long ldh,
                                          void* Hout, long long ldo, const float* gamma, float eps, int M, int K,
                                          int qt, void* Xq, float* sx, float* ms_out, int num_sms, cudaStream_t st);

}  // namespace qurl
