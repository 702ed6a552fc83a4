// round.cuh -- a round's rows over a paged key/value cache, as spec_cache_append,
// spec_tree_attention and spec_cache_keep take them.
#pragma once

#include "dependent.cuh"

#include <algorithm>

namespace sv {

struct RoundParams {
  const int64_t* row0;
  const int32_t* draft_len;
  const int32_t* parents;  // null: chains
  const int32_t* ctx_len;
  const int32_t* page_table;
  int64_t ld_pages;
  int64_t n_rows;
  int64_t n_pages;
  int32_t B, max_draft_len, bonus_row;
  int32_t max_pages, page_size;
};

// The caches: element strides, the same in both.
struct CacheParams {
  __nv_bfloat16 *k, *v;
  int64_t page_stride, token_stride, head_stride;
};

struct Request {
  int64_t first;  // row of the request's row 0
  int32_t n;      // rows
  int32_t ctx;    // places filled before
};

// A request's sizes from its draft length, context and first row; false if any is out of range: the request
// is then left alone.
__device__ __forceinline__ bool round_request(const RoundParams& p, int32_t drafts, int32_t ctx,
                                              int64_t first, Request& q) {
  q.ctx = ctx;
  q.first = first;
  // (a length that max_draft_len allows fits: round_most_drafts; another may wrap, and is refused below)
  q.n = int32_t(uint32_t(drafts) + uint32_t(p.bonus_row));
  const bool ok = drafts >= 0 && drafts <= p.max_draft_len && q.ctx >= 0 && q.first >= 0 &&
                  q.first <= p.n_rows && q.n <= p.n_rows - q.first &&
                  int64_t(q.ctx) + q.n <=
                      min(int64_t(p.max_pages) * p.page_size, int64_t(INT32_MAX));
  if (!ok) q.n = 0;
  return ok;
}

__device__ __forceinline__ bool round_request(const RoundParams& p, int32_t r, Request& q) {
  return round_request(p, p.draft_len[r], p.ctx_len[r], p.row0[r], q);
}

// Page of place `at`; -1 where the table names none.
__device__ __forceinline__ int32_t round_page(const RoundParams& p, int32_t r, int32_t at) {
  const int32_t g = p.page_table[r * p.ld_pages + at / p.page_size];
  return g >= 0 && g < p.n_pages ? g : -1;
}

// ---- the status of short calls ---------------------------------------------------------------------
// A call of a few CTAs runs as one cluster, which gathers what its CTAs found and writes the word
// itself: that saves the launch that resets it.  Larger calls report to a word reset before them.
constexpr int kOneCluster = 8;  // the largest cluster every device takes

// All threads of all CTAs, at their end.  `one`: the grid is one cluster.
__device__ __forceinline__ void round_status(int32_t* status, bool bad, bool one) {
  if (!one) {
    if (bad) report(status, SV_ERR_BAD_INPUT);
    return;
  }
  __shared__ uint32_t found;
  const int any = __syncthreads_or(bad);
  if (gridDim.x == 1) {
    if (threadIdx.x == 0 && status) *status = any ? SV_ERR_BAD_INPUT : SV_OK;
    return;
  }
  if (threadIdx.x == 0) found = uint32_t(any);
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    uint32_t x = 0;
    if (threadIdx.x < gridDim.x) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&found)), "r"(threadIdx.x));
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    }
    x = __any_sync(0xffffffffu, x != 0);
    if (threadIdx.x == 0 && status) *status = x ? SV_ERR_BAD_INPUT : SV_OK;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Launches `kernel` (whose params have a member `one`) over `grid` CTAs, as one cluster if they fit,
// else behind the reset of the status word.
template <typename P>
inline sv_status launch_round(void (*kernel)(P), int64_t grid, unsigned threads, cudaStream_t s, P p) {
  if (grid > INT32_MAX) return SV_ERR_UNSUPPORTED;
  p.one = grid <= kOneCluster;
  if (!p.one) {
    const sv_status st = reset_status(p.status, s);
    return st != SV_OK ? st : launch_dependent(kernel, unsigned(grid), threads, 0, s, p);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(grid);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid > 1 ? 2 : 1;
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

// Host side: what the calls over the cache check alike.
inline bool round_sizes_ok(int32_t max_draft_len, int32_t bonus_row, int32_t B, int64_t n_rows,
                           int64_t ld_pages, int32_t max_pages, int64_t n_pages,
                           int32_t page_size) {
  return max_draft_len >= 0 && (bonus_row == 0 || bonus_row == 1) && B >= 0 && n_rows >= 0 &&
         max_pages >= 0 && ld_pages >= max_pages && n_pages >= 0 && page_size >= 1;
}

// RoundParams::max_draft_len.  The rows of longer requests, and the ends of their tiles and chunks, would pass
// 32 bits: they are out of range.
inline int32_t round_most_drafts(int32_t max_draft_len) {
  return std::min(max_draft_len, INT32_MAX - 512);
}

inline bool aligned_bf16(const void* p, int64_t a, int64_t b, int64_t c) {
  return aligned16(p) && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

}  // namespace sv
