// The cheap score of the pages of a paged cache: scale times the product of
// the summed queries of a KV head's group with the mean key of every complete
// page.  One warp per (token, KV head, page).
#include "internal.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
page_score_kernel(const PagedView pv, const uint16_t *q, const uint16_t *k_mean, float *scores, int64_t ld, int D,
                  float scale, int local, int32_t *row_seq, int32_t *row_pos, uint32_t *status) {
  const int t = blockIdx.y, h = blockIdx.z, lane = threadIdx.x & 31;
  const int j = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (j >= pv.max_pages) return;
  int b, pos;
  const bool ok = load_paged_token(pv, t, status, threadIdx.x == 0 && blockIdx.x == 0, b, pos);
  if (row_seq && j == 0 && lane == 0) {
    const int f = ok ? max((pos >> pv.logP) + 1 - local, 0) : 0;
    row_seq[t * pv.H_kv + h] = ok ? b : -1;
    row_pos[t * pv.H_kv + h] = max(f * pv.P - 1, 0);
  }
  if (!ok) return;
  const int G = pv.H / pv.H_kv;
  float s = -INFINITY;
  if (j < (pos + 1) >> pv.logP) {
    const int page = load_page(pv, b, j, status, lane == 0);
    if (page >= 0) {
      s = 0.f;
      for (int d = lane; d < D; d += 32) {
        float qs = 0.f;
        for (int g = 0; g < G; ++g)
          qs += bf16_bits_to_float(q[(static_cast<int64_t>(t) * pv.H + h * G + g) * D + d]);
        s = fmaf(qs, bf16_bits_to_float(k_mean[(static_cast<int64_t>(page) * pv.H_kv + h) * D + d]), s);
      }
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= scale;
    }
  }
  if (lane == 0) scores[(static_cast<int64_t>(t) * pv.H_kv + h) * ld + j] = s;
}

}  // namespace

cudaError_t launch_page_scores(const sa_paged_args &pa, const void *q, const void *k_mean, float *scores, int64_t ld,
                               int local, int32_t *row_seq, int32_t *row_pos, uint32_t *status, cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  const int per = kThreads / 32;
  return launch_ex(false, page_score_kernel, dim3((pa.max_pages + per - 1) / per, pa.T, pa.H_kv), dim3(kThreads), 0,
                   stream, 1, paged_view(pa), static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k_mean),
                   scores, ld, pa.D, pa.scale, local, row_seq, row_pos, status);
}

}  // namespace sa
