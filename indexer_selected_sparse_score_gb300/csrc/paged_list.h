// The page-list attention kernel as its two users launch it.
#pragma once

#include "internal.h"
#include "paged.cuh"

namespace sa {

constexpr int kMaxCtas = 256;  // most CTAs of a grid that shares tiles out

struct ListParams {
  PagedView pv;
  int whole;       // nonzero: the pages first_page .. of each token's sequence; else idx and the local pages
  int first_page;
  int keep;        // nonzero: every piece goes to part slot unit + CTA, its CTAs to info[unit]
  const int32_t *idx;
  int K, local;
  int group, gb;   // query heads per KV head, units of up to 64 heads they take
  int tpu;         // tiles per unit (list mode)
  float qk_scale;  // scale * log2(e)
  __nv_bfloat16 *out;
  float *part;     // [slot][cols][D]
  float2 *ml;      // [slot][cols]: reference maximum (log2 units), sum
  int2 *cut;       // [CTA]: the unit its range cuts (-1: none) and the last CTA of that unit
  int2 *info;      // [unit]: first and last CTA
  uint32_t *status;
};

// Columns (padded heads) of a unit: 16, 32 or 64.
int list_cols(const sa_paged_args &pa);
size_t list_scratch(const sa_paged_args &pa, bool keep);
cudaError_t launch_page_list(const sa_paged_args &pa, const void *q, ListParams &p, void *out, void *scratch,
                             uint32_t *status, bool pdl, cudaStream_t stream);

}  // namespace sa
