// Device-side view of a paged cache (sa_paged_args) shared by its kernels.
#pragma once

#include "common.cuh"
#include "sa.h"

namespace sa {

// Sticky status flag of the paged calls, beside those of common.cuh.
constexpr uint32_t kFlagBadPage = 16u;  // a page id outside [0, n_pages)

struct PagedView {
  int B, T, H, H_kv, P, logP, n_pages, max_pages;
  int64_t table_stride;
  const int32_t *q_seq, *q_pos, *page_table;
};

inline PagedView paged_view(const sa_paged_args &pa) {
  int logP = 0;
  while ((1 << logP) < pa.P) ++logP;
  return PagedView{pa.B,     pa.T,    pa.H,         pa.H_kv,
                   pa.P,     logP,    pa.n_pages,   pa.max_pages,
                   pa.table_stride ? pa.table_stride : pa.max_pages, pa.q_seq, pa.q_pos, pa.page_table};
}

// Sequence and position of token t; false (and flagged when `report`) when the
// token must be skipped.
__device__ __forceinline__ bool load_paged_token(const PagedView &v, int t, uint32_t *status, bool report, int &b,
                                                 int &pos) {
  b = v.q_seq[t];
  pos = v.q_pos[t];
  if (b < 0 || b >= v.B) {
    if (report) raise_flag(status, kFlagBadSeq);
    return false;
  }
  if (pos < 0 || (pos >> v.logP) >= v.max_pages) {
    if (report) raise_flag(status, kFlagBadPos);
    return false;
  }
  return true;
}

// Page id of page-table entry j of sequence b (0 <= j < max_pages), -1 (and
// flagged when `report`) when the entry is out of range.
__device__ __forceinline__ int load_page(const PagedView &v, int b, int j, uint32_t *status, bool report) {
  const int id = v.page_table[b * v.table_stride + j];
  if (id >= 0 && id < v.n_pages) return id;
  if (report) raise_flag(status, kFlagBadPage);
  return -1;
}

// Sum of `v` over the threads before this one, and over the block (`warp_s`:
// one slot per warp).  Every thread of the block calls it.
__device__ __forceinline__ long long block_prefix(long long v, long long *warp_s, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += up;
  }
  if (lane == 31) warp_s[warp] = s;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += warp_s[w];
    total += warp_s[w];
  }
  return before + s - v;
}

}  // namespace sa
