// pages.cu -- pages of the paged cache, handed out and taken back on the GPU:
// qurl_kv_append places a step's new tokens, qurl_kv_release returns pages.
//
//   need_b = ceil((c_b + n_b) / block) - ceil(c_b / block)      pages that request b takes
//   page j of all that are taken = free[n_free - 1 - j]         (the end of the list first)
//   slot of a token at position p = page of block p / block, times block, plus p % block
//
// Nothing here is large: a step's bookkeeping is a few bytes a token (12 written)
// and a prefix sum over the requests, so what counts is the number of dependent
// steps.  One cluster of up to 8 CTAs does a call in one launch: every CTA reads
// the lengths and forms the sums for itself (no exchange), keeps them in shared
// memory, and finds a token's request there by bisection.  A page that is taken
// in the same call is looked up in the free list rather than in the table, so
// tokens need not wait for the table's entries.  The barrier of the cluster
// stands between the last read of what a caller may hand in as an output too
// (n_free, the lengths) and its write.
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "rollout.h"

namespace qurl {
namespace {

constexpr int kPageThreads = 1024;

// Exclusive prefix sum over the block's threads; `total` gets the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* red, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // (red may still be read from the sum before)
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += u;
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[31];
  return inc - v + (warp > 0 ? red[warp - 1] : T(0));
}

// The last b in [0, n) with first[b] <= i (first[0] = 0, not decreasing).
__device__ __forceinline__ int owner(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(int tokens, int block) {
  return tokens / block + (tokens % block != 0 ? 1 : 0);
}

// The number of free pages, within the list.
__device__ __forceinline__ int free_pages_of(const int* n_free, int capacity, bool report, int* status) {
  int n = *n_free;
  if (n > capacity) {
    if (report) latch_bad_index(status);
    n = capacity;
  }
  return n < 0 ? 0 : n;
}

__global__ void __launch_bounds__(kPageThreads, 1) kv_append_kernel(const KvAppendArgs a) {
  extern __shared__ int sm_pages[];
  __shared__ long long red64[32];
  __shared__ int red[32];
  int* cu = sm_pages;              // [B + 1] new tokens before a request
  int* need = cu + a.B + 1;        // [B + 1] pages taken before it
  int* held = need + a.B + 1;      // [B] tokens it has
  const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
  griddep_wait();
  griddep_launch_dependents();

  const int room = a.max_blocks * a.block_size;
  const int nf = free_pages_of(a.n_free, a.capacity, rank == 0 && tid == 0, a.status);
  const int chunk = (a.B + kPageThreads - 1) / kPageThreads;
  const int b0 = min(tid * chunk, a.B), b1 = min(b0 + chunk, a.B);
  bool bad = false;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    int c = max(a.cached[b], 0), n = max(a.fresh[b], 0);
    if (c > room) c = room, bad = true;
    if (n > room - c) n = room - c, bad = true;
    held[b] = c;
    need[b] = n;
    sum += n;
  }
  long long total64;
  long long before = block_scan(sum, red64, &total64);
  // tokens past the M rows of this step are cut
  if (total64 > a.M) bad = true;
  const int total = static_cast<int>(min(total64, static_cast<long long>(a.M)));
  int pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int at = static_cast<int>(min(before, static_cast<long long>(a.M)));
    before += need[b];
    const int n = static_cast<int>(min(before, static_cast<long long>(a.M))) - at;
    cu[b] = at;
    need[b] = blocks_of(held[b] + n, a.block_size) - blocks_of(held[b], a.block_size);
    pages += need[b];
  }
  int taken;
  int first = block_scan(pages, red, &taken);
  for (int b = b0; b < b1; ++b) {
    const int n = need[b];
    need[b] = first;
    first += n;
  }
  if (tid == 0) {
    cu[a.B] = total;
    need[a.B] = taken;
  }
  if (bad && rank == 0) latch_bad_index(a.status);
  __syncthreads();
  // This CTA has read the lengths and the number of free pages: an arrival that orders those reads (release), as the
  // writes behind the wait (acquire) may be to the same words.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  auto page_of = [&](int j) { return j < nf ? __ldg(a.free_pages + (nf - 1 - j)) : -1; };
  // (unsigned: a step past the last row may be past 2^31)
  const unsigned begin = rank * kPageThreads + tid, step = ranks * kPageThreads;
  for (unsigned u = begin; u < static_cast<unsigned>(taken); u += step) {
    const int j = static_cast<int>(u), b = owner(need, a.B, j);
    const int k = blocks_of(held[b], a.block_size) + j - need[b];
    a.table[static_cast<long long>(b) * a.ld_table + k] = page_of(j);
  }
#pragma unroll 4
  for (unsigned u = begin; u < static_cast<unsigned>(a.M); u += step) {
    const int i = static_cast<int>(u);
    long long slot = -1;
    int pos = 0;
    if (i < total) {
      const int b = owner(cu, a.B, i);
      pos = held[b] + i - cu[b];
      const int k = pos / a.block_size, have = blocks_of(held[b], a.block_size);
      const int page = k < have ? a.table[static_cast<long long>(b) * a.ld_table + k] : page_of(need[b] + k - have);
      if (page >= 0) slot = static_cast<long long>(page) * a.block_size + (pos - k * a.block_size);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has
  for (int b = static_cast<int>(begin); b <= a.B; b += static_cast<int>(step)) {
    a.cu[b] = cu[b];
    if (b < a.B) a.seq_lens[b] = held[b] + cu[b + 1] - cu[b];
  }
  if (rank == 0 && tid == 0) *a.n_free_out = nf - taken;
}

__device__ __forceinline__ int peer_value(int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_map(p, rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kPageThreads, 1) kv_release_kernel(const KvReleaseArgs a) {
  extern __shared__ int sm_pages[];
  __shared__ int red[32];
  __shared__ int mine;             // pages that this CTA's entries return
  int* first = sm_pages;           // [B + 1] entries to look at before a request
  int* from = first + a.B + 1;     // [B] its first block that is returned
  const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
  griddep_wait();
  griddep_launch_dependents();

  const int room = a.max_blocks * a.block_size;
  const int nf = free_pages_of(a.n_free, a.capacity, rank == 0 && tid == 0, a.status);
  const int chunk = (a.B + kPageThreads - 1) / kPageThreads;
  const int b0 = min(tid * chunk, a.B), b1 = min(b0 + chunk, a.B);
  bool bad = false;
  int entries = 0;
  for (int b = b0; b < b1; ++b) {
    int n = max(a.lens[b], 0);
    const int keep = a.keep ? max(a.keep[b], 0) : 0;
    if (n > room) n = room, bad = true;
    from[b] = keep < n ? blocks_of(keep, a.block_size) : 0;
    first[b] = entries;  // (within the thread's requests)
    entries += keep < n ? blocks_of(n, a.block_size) - from[b] : 0;
  }
  int total;
  const int before = block_scan(entries, red, &total);
  for (int b = b0; b < b1; ++b) first[b] += before;
  if (tid == 0) first[a.B] = total;
  __syncthreads();

  // this CTA's entries, a run of them each thread: counted, then written in order
  const int lo = static_cast<int>(static_cast<long long>(total) * rank / ranks);
  const int hi = static_cast<int>(static_cast<long long>(total) * (rank + 1) / ranks);
  const int run = (hi - lo + kPageThreads - 1) / kPageThreads;
  const int e0 = min(lo + tid * run, hi), e1 = min(e0 + run, hi);
  const int start = e0 < e1 ? owner(first, a.B, e0) : 0;
  auto each = [&](auto&& f) {
    int b = start;
    for (int e = e0; e < e1; ++e) {
      while (first[b + 1] <= e) ++b;
      const int page = a.table[static_cast<long long>(b) * a.ld_table + from[b] + e - first[b]];
      if (page >= 0) f(page);
    }
  };
  int count = 0;
  each([&](int) { ++count; });
  int all;
  int at = block_scan(count, red, &all);
  if (tid == 0) mine = all;
  cluster_sync();  // (every CTA has read n_free, too)
  long long put = nf, sum = nf;
  for (int r = 0; r < ranks; ++r) {
    const int n = peer_value(&mine, r);
    if (r < rank) put += n;
    sum += n;
  }
  put += at;
  each([&](int page) {
    if (put < a.capacity) a.free_pages[put] = page;
    ++put;
  });
  if (sum > a.capacity) bad = true;
  if (bad && rank == 0) latch_bad_index(a.status);
  if (rank == 0 && tid == 0) *a.n_free_out = static_cast<int>(min(sum, static_cast<long long>(a.capacity)));
  cluster_sync();  // no CTA leaves while another may read its count
}

// One CTA per so many items, up to a cluster of 8.
int page_ranks(long long items) {
  return items <= 4 * kPageThreads ? 1 : items <= 8 * kPageThreads ? 2 : items <= 16 * kPageThreads ? 4 : 8;
}

template <typename A>
cudaError_t launch_pages(void (*kern)(A), const A& a, int ranks, size_t smem, bool (&attr_done)[64], cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * kMaxRequests + 2) * 4);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl_cluster(kern, ranks, dim3(ranks), dim3(kPageThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t st) {
  static bool attr_done[64] = {};
  return launch_pages(kv_append_kernel, a, page_ranks(a.M > a.B ? a.M : a.B), (3 * static_cast<size_t>(a.B) + 2) * 4,
                      attr_done, st);
}

cudaError_t launch_kv_release(const KvReleaseArgs& a, cudaStream_t st) {
  static bool attr_done[64] = {};
  const long long entries = static_cast<long long>(a.B) * a.max_blocks;
  return launch_pages(kv_release_kernel, a, page_ranks(entries), (2 * static_cast<size_t>(a.B) + 1) * 4, attr_done, st);
}

}  // namespace qurl
