// The page-list attention kernel as its two users launch it.
#pragma once

#include "internal.h"
#include "paged.cuh"

namespace sa {

constexpr int kMaxParts = 2048;  // most parts of a claimed list
// Word of the workspace header that counts claimed parts: 0 between calls (the
// merge that ends a call resets it).
constexpr int kCounterWord = 16;

// Weighted mean of `total` parts (locate(k) gives part k's (reference, sum) and
// output row): out[e] = value kDim / 32 lane + e of the row.  kSplit warps take
// every kSplit-th part (`mine` first) and the first of them returns true with
// the result; with kSplit > 1 every thread of the block calls this.
template <int kDim, int kSplit, typename Locate>
__device__ __forceinline__ bool merge_parts(int total, int mine, int lane, const Locate &locate, float (*acc_s)[kDim + 1],
                                            float (&out)[kDim / 32]) {
  constexpr int V = kDim / 32;
  const float2 *ml;
  const float *o;
  float M = -INFINITY;
  for (int k = lane; k < total; k += 32) {
    locate(k, ml, o);
    M = fmaxf(M, ml->x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float acc[V] = {}, l = 0.f;
  for (int k0 = 0; k0 < total; k0 += 32 * kSplit) {
    float a = 0.f, la = 0.f;  // this lane's part: weight, weighted sum
    const float *row = nullptr;
    const int k = k0 + mine + kSplit * lane;
    if (k < total) {
      locate(k, ml, row);
      const float2 v = *ml;
      a = v.x == -INFINITY ? 0.f : exp2f(v.x - M);
      la = a * v.y;
    }
    const int n = min(32, (total - k0 - mine + kSplit - 1) / kSplit);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, a, i);
      l += __shfl_sync(0xffffffffu, la, i);
      const float *src =
          reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), i));
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(w, src[V * lane + e], acc[e]);
    }
  }
  if constexpr (kSplit > 1) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < V; ++e) acc_s[warp][V * lane + e] = acc[e];
    if (lane == 0) acc_s[warp][kDim] = l;
    __syncthreads();
    if (mine != 0) return false;
    for (int w = 1; w < kSplit; ++w) {
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += acc_s[warp + w][V * lane + e];
      l += acc_s[warp + w][kDim];
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) out[e] = acc[e] * inv;
  return true;
}

struct ListParams {
  PagedView pv;
  int whole;       // nonzero: the pages first_page .. of each token's sequence; else idx and the local pages
  int first_page;
  int keep;        // nonzero: every piece goes to slot unit + part, the unit's parts to info[unit]
  int parts;       // parts the tiles are cut into (at most)
  uint32_t *counter;  // claims parts (keep), or NULL: CTA c takes part c
  const int32_t *idx;
  int K, local;
  int group, gb;   // query heads per KV head, units of up to 64 heads they take
  int tpu;         // tiles per unit (list mode)
  float qk_scale;  // scale * log2(e)
  __nv_bfloat16 *out;
  float *part;     // [slot][cols][D]
  float2 *ml;      // [slot][cols]: reference maximum (log2 units), sum
  int2 *cut;       // [CTA]: the unit its range cuts (-1: none) and the last CTA of that unit
  int2 *info;      // [unit]: first and last part
  uint32_t *status;
};

// Columns (padded heads) of a unit: 16, 32 or 64.
int list_cols(const sa_paged_args &pa);
size_t list_scratch(const sa_paged_args &pa, bool keep);
cudaError_t launch_page_list(const sa_paged_args &pa, const void *q, ListParams &p, void *out, void *scratch,
                             uint32_t *status, bool pdl, cudaStream_t stream);

}  // namespace sa
