// Attention over a paged cache: selected pages and a local window of pages, or
// whole sequences.  One warp per (token, query head); the lanes split 32 keys
// for the logits and the head dim for the output, with a running maximum and
// sum (online softmax).
#include "internal.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;

struct PagedAttnParams {
  PagedView pv;
  const uint16_t *q, *K, *V;
  __nv_bfloat16 *out;
  const int32_t *idx;
  int n_list, local, shared_pages, D;
  bool whole;  // every position, the first shared_pages pages from table row 0
  float scale;
  uint32_t *status;
};

__global__ void __launch_bounds__(32 * kWarps)
paged_attn_kernel(const PagedAttnParams p) {
  __shared__ float qs[kWarps][128];
  __shared__ float ps[kWarps][32];
  const PagedView &pv = p.pv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= static_cast<int64_t>(pv.T) * pv.H) return;
  const int t = static_cast<int>(row / pv.H), h = static_cast<int>(row % pv.H), hk = h / (pv.H / pv.H_kv);
  int b, pos;
  if (!load_paged_token(pv, t, p.status, lane == 0, b, pos)) return;
  if (p.whole && pos < p.shared_pages * pv.P) {
    if (lane == 0) raise_flag(p.status, kFlagBadPos);
    return;
  }
  for (int d = lane; d < p.D; d += 32) qs[warp][d] = bf16_bits_to_float(p.q[row * p.D + d]);
  __syncwarp();
  const int last = pos >> pv.logP;
  const int f = p.whole ? 0 : max(last + 1 - p.local, 0);
  const int nl = p.whole ? 0 : p.n_list;
  float m = -INFINITY, l = 0.f, acc[4] = {};
  for (int e = 0; e < nl + last + 1 - f; ++e) {
    int j = e < nl ? p.idx[(static_cast<int64_t>(t) * pv.H_kv + hk) * p.n_list + e] : f + e - nl;
    if (e < nl && (j < 0 || j >= f)) {
      if (lane == 0 && (j < -1 || j > last)) raise_flag(p.status, kFlagBadIndex);
      continue;
    }
    const int page = load_page(pv, p.whole && j < p.shared_pages ? 0 : b, j, p.status, lane == 0);
    if (page < 0) continue;
    const int64_t tile = (static_cast<int64_t>(page) * pv.H_kv + hk) * pv.P;
    const int n = min(pv.P, pos + 1 - j * pv.P);
    for (int r0 = 0; r0 < n; r0 += 32) {
      float s = -INFINITY;
      if (r0 + lane < n) {
        s = 0.f;
        const uint16_t *kr = p.K + (tile + r0 + lane) * p.D;
        for (int d = 0; d < p.D; ++d) s = fmaf(qs[warp][d], bf16_bits_to_float(kr[d]), s);
        s *= p.scale;
      }
      float mx = s;
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m, mx);
      const float a = m == -INFINITY ? 0.f : __expf(m - mn);
      const float w = s == -INFINITY ? 0.f : __expf(s - mn);
      m = mn;
      l = l * a + w;
      ps[warp][lane] = w;
      __syncwarp();
      for (int i = 0; i < 4; ++i) acc[i] *= a;
      for (int k = 0; k < min(32, n - r0); ++k) {
        const uint16_t *vr = p.V + (tile + r0 + k) * p.D;
        for (int i = 0; i < p.D / 32; ++i)
          acc[i] = fmaf(ps[warp][k], bf16_bits_to_float(vr[32 * i + lane]), acc[i]);
      }
      __syncwarp();
    }
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  for (int i = 0; i < p.D / 32; ++i)
    p.out[row * p.D + 32 * i + lane] = __float2bfloat16_rn(l > 0.f ? acc[i] / l : 0.f);
}

cudaError_t launch(const sa_paged_args &pa, PagedAttnParams &p, const void *q, void *out, uint32_t *status,
                   cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  p.pv = paged_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.K = static_cast<const uint16_t *>(pa.K);
  p.V = static_cast<const uint16_t *>(pa.V);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.D = pa.D;
  p.scale = pa.scale;
  p.status = status;
  const int64_t rows = static_cast<int64_t>(pa.T) * pa.H;
  return launch_ex(false, paged_attn_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)),
                   dim3(32 * kWarps), 0, stream, 1, p);
}

}  // namespace

size_t prefix_attn_scratch(const sa_paged_args &, int) { return 0; }

cudaError_t launch_prefix_attn(const sa_paged_args &pa, const void *q, int shared_pages, void *out, void *,
                               uint32_t *status, cudaStream_t stream) {
  PagedAttnParams p{};
  p.whole = true;
  p.shared_pages = shared_pages;
  return launch(pa, p, q, out, status, stream);
}

}  // namespace sa
