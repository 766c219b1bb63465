// The page-list attention kernel as its two users launch it.
#pragma once

#include "internal.h"
#include "paged.cuh"

namespace sa {

constexpr int kMaxParts = 1024;  // most parts of a claimed list
// Word of the workspace header that counts claimed parts: 0 between calls (the
// merge that ends a call resets it).
constexpr int kCounterWord = 16;

// The larger of the two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Running merge of parts (reference, sum, output row): a warp per row, lane l
// holding values V l .. V l + V - 1 of it.  Eight parts' loads go out together.
// A part whose reference or sum is NaN makes the row NaN, as in a unit of one part.
template <int kDim>
struct Merge {
  static constexpr int V = kDim / 32;
  float M = -INFINITY, l = 0.f, acc[V] = {};

  __device__ __forceinline__ void scale_to(float m) {
    const float f = M == -INFINITY ? 0.f : exp2f(M - m);
    l *= f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= f;
    M = m;
  }
  // Parts first, first + step, .. below total; at(k) is part k's row number in
  // ml and part.
  template <typename At>
  __device__ __forceinline__ void add(int first, int step, int total, int lane, const float2 *ml, const float *part,
                                      const At &at) {
    for (int k0 = first; k0 < total; k0 += 8 * step) {
      float2 s[8];
      float x[8][V];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = at(min(k0 + i * step, total - 1));
        s[i] = ml[row];
        if constexpr (V == 4)
          *reinterpret_cast<float4 *>(x[i]) = *reinterpret_cast<const float4 *>(part + row * kDim + V * lane);
        else
          *reinterpret_cast<float2 *>(x[i]) = *reinterpret_cast<const float2 *>(part + row * kDim + V * lane);
      }
      float m = M;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, s[i].x);
      if (m == -INFINITY) continue;
      scale_to(m);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = k0 + i * step < total && s[i].x != -INFINITY ? exp2f(s[i].x - m) : 0.f;
        l = fmaf(w, s[i].y, l);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w, w > 0.f ? x[i][e] : 0.f, acc[e]);
      }
    }
  }
  // Joins the kSplit warps that hold a row (warps kSplit r .. of the block); the
  // first of them returns true.  Every thread of the block calls it.
  template <int kSplit>
  __device__ __forceinline__ bool join(float (*s)[kDim + 2], int lane) {
    if constexpr (kSplit == 1) {
      return true;
    } else {
      const int warp = threadIdx.x >> 5;
#pragma unroll
      for (int e = 0; e < V; ++e) s[warp][V * lane + e] = acc[e];
      if (lane == 0) {
        s[warp][kDim] = M;
        s[warp][kDim + 1] = l;
      }
      __syncthreads();
      if (warp % kSplit) return false;
      float m = M;
      for (int w = 1; w < kSplit; ++w) m = max_nan(m, s[warp + w][kDim]);
      if (m == -INFINITY) return true;
      scale_to(m);
      for (int w = 1; w < kSplit; ++w) {
        const float f = s[warp + w][kDim] == -INFINITY ? 0.f : exp2f(s[warp + w][kDim] - m);
        l = fmaf(f, s[warp + w][kDim + 1], l);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(f, s[warp + w][V * lane + e], acc[e]);
      }
      return true;
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, int lane) const {
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < V; e += 2)
      *reinterpret_cast<__nv_bfloat162 *>(row + V * lane + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  }
};

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
