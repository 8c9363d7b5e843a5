// kv_pages.cu -- pages for the new tokens of a batch of requests:
//   need_b = ceil((kv_b + new_b) / page) - ceil(kv_b / page),
//   the pages of request b are free[used + sum_{a<b} need_a ..], its token rows
//   start at sum_{a<b} new_a.
// Bound by latency: some loads, a scan over the requests, some stores (a token for
// each of 64 requests 3.2 us in a graph, 512 prompts with 26,000 tokens 8.0).
//
// One cluster of CTAs does it in one launch.  Every CTA reads the lengths and
// scans them into its own shared memory; after a cluster barrier (the inputs
// may be the outputs) the CTAs share out the entries, slots and positions, each
// found by a binary search over the sums.
#include <cooperative_groups.h>

#include "cache_device.cuh"
#include "tma_host.h"

namespace gdn {
namespace {

struct Sums {
  long long tokens, pages;
};
__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, v.tokens, d), __shfl_up_sync(0xffffffffu, v.pages, d)};
}

// The last i in [0, n) with at[i] <= x (at[0] = 0 <= x).
__device__ __forceinline__ int last_not_above(const int *at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) kv_pages_kernel(const PagesArgs a) {
  extern __shared__ int arrays[];
  int *const kv_of = arrays, *const tok_of = arrays + a.B, *const page_of = arrays + 2 * a.B;
  __shared__ Sums warp_sums[32];
  __shared__ int bad;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  const int page = 1 << a.page_shift;
  if (tid == 0) bad = 0;
  __syncthreads();
  const long long used = *a.free_used;
  Sums total{0, 0};
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    Sums own{0, 0};
    if (b < a.B) {
      const long long kv = a.kv_lens[b], n = a.new_tokens[b];
      const long long need = (kv + n + page - 1) >> a.page_shift, have = (kv + page - 1) >> a.page_shift;
      if (kv < 0 || n < 0 || need > a.max_blocks || kv + n > 0x7fffffff) bad = 1;
      own = Sums{n, need - have};
      kv_of[b] = (int)kv;
    }
    Sums sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums up = shfl_up(sum, d);
      if (lane >= d) sum.tokens += up.tokens, sum.pages += up.pages;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    // each warp scans the warps' sums for itself
    Sums all = lane < nwarps ? warp_sums[lane] : Sums{0, 0};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums up = shfl_up(all, d);
      if (lane >= d) all.tokens += up.tokens, all.pages += up.pages;
    }
    Sums before = total;
    const int prev = max(warp - 1, 0);
    const long long t = __shfl_sync(0xffffffffu, all.tokens, prev), g = __shfl_sync(0xffffffffu, all.pages, prev);
    if (warp > 0) before.tokens += t, before.pages += g;
    total.tokens += __shfl_sync(0xffffffffu, all.tokens, 31);
    total.pages += __shfl_sync(0xffffffffu, all.pages, 31);
    if (b < a.B) {  // sums past 31 bits make the call fail below
      tok_of[b] = (int)(before.tokens + sum.tokens - own.tokens);
      page_of[b] = (int)(before.pages + sum.pages - own.pages);
    }
    __syncthreads();
  }
  const bool fail = bad || used < 0 || total.tokens > a.max_tokens || total.pages > a.n_free - used;
  cluster.sync();  // nobody reads the lengths or the count any more
  const int rank = (int)cluster.block_rank();
  const long long at = (long long)rank * blockDim.x + tid, step = (long long)cluster.num_blocks() * blockDim.x;
  if (at == 0) {
    if (fail) atomicOr(a.err, kErrSeqlens);
    *a.free_used_out = (int)(fail ? used : used + total.pages);
    a.cu[a.B] = fail ? 0 : (int)total.tokens;
  }
  for (long long b = at; b < a.B; b += step) {
    const int next = b + 1 < a.B ? tok_of[b + 1] : (int)total.tokens;
    a.cu[b] = fail ? 0 : tok_of[b];
    a.kv_lens_out[b] = fail ? kv_of[b] : kv_of[b] + next - tok_of[b];
  }
  const int *const fresh = a.free_pages + used;
  if (!fail)
    for (long long e = at; e < total.pages; e += step) {
      const int b = last_not_above(page_of, a.B, (int)e);
      const int have = (int)(((long long)kv_of[b] + page - 1) >> a.page_shift);
      a.table[b * a.table_ld + have + (e - page_of[b])] = fresh[e];
    }
  if (!a.slots && !a.positions) return;
  const long long tokens = fail ? 0 : total.tokens;
  for (long long t = at; t < a.max_tokens; t += step) {
    long long slot = -1;
    int pos = 0;
    if (t < tokens) {
      const int b = last_not_above(tok_of, a.B, (int)t), kv = kv_of[b];
      pos = kv + ((int)t - tok_of[b]);
      if (a.slots) {
        const int blk = pos >> a.page_shift, have = (int)(((long long)kv + page - 1) >> a.page_shift);
        const int p = blk < have ? a.table[b * a.table_ld + blk] : fresh[page_of[b] + blk - have];
        slot = ((long long)p << a.page_shift) + (pos & (page - 1));
      }
    }
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

struct PagesTag {};

}  // namespace

cudaError_t launch_kv_pages(const PagesArgs &a, cudaStream_t s) {
  const size_t smem = (size_t)a.B * 3 * sizeof(int);
  cudaError_t e = allow_smem<PagesTag>(kv_pages_kernel, (size_t)kPagesMaxB * 3 * sizeof(int));
  if (e != cudaSuccess) return e;
  // Threads and CTAs cost a start, and save on the scan and the stores (us in a graph, requests / tokens: one CTA of 256
  // threads, 8 of 512, 8 of 1024):  64/64 3.2, 3.5, 4.2;  256/256 3.5, 3.9, 4.5;  256/843 6.2, 4.0, 4.9;  64/2950 9.7, 3.7,
  // 4.5;  1024/3470 16, 5.1, 5.3;  1/18995 23, 4.3, 4.7;  512/26431 75, 8.8, 8.0;  4096/4096 27, 10.1, 10.0;
  // 16384/16384 107, 32, 27.
  const bool small = a.B <= 256 && a.max_tokens <= 256, large = a.B > 4096 || a.max_tokens > 20480;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(small ? 1 : 8);
  cfg.blockDim = dim3(small ? 256 : large ? 1024 : 512);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cfg.gridDim.x;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_pages_kernel, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace gdn
