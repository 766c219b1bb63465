// C ABI of the paged cache (include/sa.h, sa_paged_args): argument checks on
// the host, workspace carve-up and the launch sequence of each entry point.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace {

using sa::set_error;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

sa_status cuda_fail(cudaError_t e, const char *what) {
  return set_error(SA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

namespace sa {

sa_status check_paged(const sa_paged_args *pa, bool need_cache) {
  if (!pa) return set_error(SA_ERR_INVALID_ARG, "paged args pointer is NULL");
  if (pa->B < 1 || pa->T < 0 || pa->H < 1 || pa->H_kv < 1 || pa->H % pa->H_kv || pa->n_pages < 1 || pa->max_pages < 1)
    return set_error(SA_ERR_INVALID_ARG,
                     "need B, H, H_kv, n_pages, max_pages >= 1, T >= 0, H_kv dividing H (got B=%d T=%d H=%d H_kv=%d "
                     "n_pages=%d max_pages=%d)",
                     pa->B, pa->T, pa->H, pa->H_kv, pa->n_pages, pa->max_pages);
  if (pa->D != 64 && pa->D != 128) return set_error(SA_ERR_UNSUPPORTED, "head dim %d: need 64 or 128", pa->D);
  if (pa->H / pa->H_kv > 128 || pa->H_kv > 65535)
    return set_error(SA_ERR_UNSUPPORTED, "%d query heads over %d KV heads: at most 128 per KV head, 65535 KV heads",
                     pa->H, pa->H_kv);
  if (pa->P != 16 && pa->P != 32 && pa->P != 64 && pa->P != 128)
    return set_error(SA_ERR_UNSUPPORTED, "%d positions per page: need 16, 32, 64 or 128", pa->P);
  if (static_cast<int64_t>(pa->max_pages) * pa->P > (int64_t{1} << 30))
    return set_error(SA_ERR_UNSUPPORTED, "max_pages * P above 2^30");
  if (static_cast<int64_t>(pa->n_pages) * pa->H_kv > ((int64_t{1} << 31) - 256) / pa->P - 1)
    return set_error(SA_ERR_UNSUPPORTED, "cache rows n_pages * H_kv * P must fit in 31 bits");
  if (static_cast<int64_t>(pa->T) * pa->H > (int64_t{1} << 30))
    return set_error(SA_ERR_UNSUPPORTED, "T * H above 2^30");
  if (pa->table_stride != 0 && pa->table_stride < pa->max_pages)
    return set_error(SA_ERR_INVALID_ARG, "table_stride %lld: need 0 or at least max_pages = %d",
                     static_cast<long long>(pa->table_stride), pa->max_pages);
  if (pa->T > 0 && (!pa->q_seq || !pa->q_pos || !pa->page_table))
    return set_error(SA_ERR_INVALID_ARG, "q_seq, q_pos and page_table must be device pointers");
  if (!aligned(pa->q_seq, 4) || !aligned(pa->q_pos, 4) || !aligned(pa->page_table, 4))
    return set_error(SA_ERR_INVALID_ARG, "q_seq, q_pos and page_table must be 4-byte aligned");
  if (!need_cache) return SA_OK;
  if (pa->T > 0 && (!pa->K || !pa->V)) return set_error(SA_ERR_INVALID_ARG, "K and V must be device pointers");
  if (!aligned(pa->K, 16) || !aligned(pa->V, 16))
    return set_error(SA_ERR_INVALID_ARG, "K and V must be 16-byte aligned");
  return SA_OK;
}

namespace {

sa_status check_stride(const char *name, int64_t stride, int64_t row) {
  if (stride != 0 && (stride < row || stride % 8))
    return set_error(SA_ERR_INVALID_ARG, "%s_stride %lld: need 0 or a multiple of 8 of at least %lld", name,
                     static_cast<long long>(stride), static_cast<long long>(row));
  return SA_OK;
}

}  // namespace

sa_status check_append(const sa_paged_args *pa, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                       const void *q, int64_t q_stride, const void *q_out, const sa_rope_args *rope, int dim_unit) {
  const int64_t kv_row = static_cast<int64_t>(pa->H_kv) * pa->D, q_row = static_cast<int64_t>(pa->H) * pa->D;
  if (sa_status s = check_stride("k", k_stride, kv_row)) return s;
  if (sa_status s = check_stride("v", v_stride, kv_row)) return s;
  if (sa_status s = check_stride("q", q_stride, q_row)) return s;
  if (pa->T > 0 && (!k || !v)) return set_error(SA_ERR_INVALID_ARG, "k and v must be device pointers");
  if ((q == nullptr) != (q_out == nullptr)) return set_error(SA_ERR_INVALID_ARG, "q and q_out go together");
  if (q && q == q_out && q_stride != 0 && q_stride != q_row)
    return set_error(SA_ERR_INVALID_ARG, "q_out may be q only when q is dense");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16))
    return set_error(SA_ERR_INVALID_ARG, "k, v, q and q_out must be 16-byte aligned");
  if (rope) {
    if (rope->dim < 0 || rope->dim > pa->D || rope->dim % dim_unit)
      return set_error(SA_ERR_INVALID_ARG, "rope dim %d: need a multiple of %d in [0, %d]", rope->dim, dim_unit, pa->D);
    if (rope->dim > 0 &&
        (!std::isfinite(rope->base) || rope->base <= 1.0 || !std::isfinite(rope->factor) || rope->factor <= 0.0 ||
         (rope->original_seq_len > 0 && !(std::isfinite(rope->beta_fast) && rope->beta_fast > 0.0 &&
                                          std::isfinite(rope->beta_slow) && rope->beta_slow > 0.0))))
      return set_error(SA_ERR_INVALID_ARG, "rope base > 1, factor > 0 and, with YaRN, beta_fast and beta_slow > 0");
  }
  return SA_OK;
}

}  // namespace sa

namespace {

using sa::check_paged;

sa_status check_scale(const sa_paged_args *pa) {
  return std::isfinite(pa->scale) ? SA_OK : set_error(SA_ERR_INVALID_ARG, "scale is not finite");
}

sa_status check_ws(void *ws, size_t ws_bytes, size_t need) {
  if (!ws) return set_error(SA_ERR_WORKSPACE, "workspace pointer is NULL");
  if (!aligned(ws, 16)) return set_error(SA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (ws_bytes < need) return set_error(SA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  return SA_OK;
}

sa_status check_lists(int32_t K, int32_t local) {
  if (K < 0 || local < 0) return set_error(SA_ERR_INVALID_ARG, "need K >= 0 and local >= 0 (got %d, %d)", K, local);
  if (K > 1 << 30) return set_error(SA_ERR_UNSUPPORTED, "K = %d above 2^30", K);
  return SA_OK;
}

sa_status check_shared(const sa_paged_args *pa, int32_t shared_pages) {
  if (shared_pages < 0 || shared_pages > pa->max_pages)
    return set_error(SA_ERR_INVALID_ARG, "shared_pages %d: need 0 .. max_pages = %d", shared_pages, pa->max_pages);
  return SA_OK;
}

// Workspace of the fused call: scores, indices and the top-k's token arrays
// (one row per token and KV head; none for K = 0), then the attention's scratch.
struct FusedLayout {
  size_t scores, idx, row_seq, row_pos, attn, total;
};
FusedLayout fused_layout(const sa_paged_args &pa, int K, int local) {
  FusedLayout L{};
  const size_t rows = K > 0 ? static_cast<size_t>(pa.T) * pa.H_kv : 0;
  size_t off = sa::kWsHeader;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round_up(bytes);
    return at;
  };
  L.scores = take(sizeof(float) * rows * pa.max_pages);
  L.idx = take(sizeof(int32_t) * rows * K);
  L.row_seq = take(sizeof(int32_t) * rows);
  L.row_pos = take(sizeof(int32_t) * rows);
  L.attn = take(sa::block_attn_scratch(pa, K, local));
  L.total = off;
  return L;
}

template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}
cudaStream_t cu(sa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

size_t sa_paged_workspace_size(const sa_paged_args *pa, int32_t K, int32_t local, int32_t shared_pages) {
  if (check_paged(pa, false) != SA_OK || check_lists(K, local) != SA_OK || check_shared(pa, shared_pages) != SA_OK)
    return 0;
  return std::max(fused_layout(*pa, K, local).total, sa::kWsHeader + round_up(sa::prefix_attn_scratch(*pa, shared_pages)));
}

sa_status sa_paged_append(const sa_paged_args *pa, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          const void *q, int64_t q_stride, void *q_out, const sa_rope_args *rope, int32_t rope_halves,
                          void *k_mean, void *ws, size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged(pa, true)) return s;
  if (sa_status s = sa::check_append(pa, k, k_stride, v, v_stride, q, q_stride, q_out, rope, 16)) return s;
  if (!aligned(k_mean, 16)) return set_error(SA_ERR_INVALID_ARG, "k_mean must be 16-byte aligned");
  if (sa_status s = check_ws(ws, ws_bytes, 256)) return s;
  cudaError_t e = sa::launch_paged_append(*pa, k, k_stride, v, v_stride, q, q_stride, q_out, rope, rope_halves != 0,
                                          k_mean, at<uint32_t>(ws, 0), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "paged append launch");
}

static sa_status check_queries(const sa_paged_args *pa, const void *q, const void *k_mean, bool need_mean) {
  if (sa_status s = check_scale(pa)) return s;
  if (pa->T > 0 && (!q || (need_mean && !k_mean)))
    return set_error(SA_ERR_INVALID_ARG, "q%s must be device pointers", need_mean ? " and k_mean" : "");
  if (!aligned(q, 16) || !aligned(k_mean, 16))
    return set_error(SA_ERR_INVALID_ARG, "q and k_mean must be 16-byte aligned");
  return SA_OK;
}

static sa_status check_out(const sa_paged_args *pa, const void *out) {
  if (pa->T > 0 && !out) return set_error(SA_ERR_INVALID_ARG, "out must be a device pointer");
  if (!aligned(out, 16)) return set_error(SA_ERR_INVALID_ARG, "out must be 16-byte aligned");
  return SA_OK;
}

sa_status sa_page_scores(const sa_paged_args *pa, const void *q, const void *k_mean, float *scores, int64_t ld,
                         void *ws, size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged(pa, false)) return s;
  if (sa_status s = check_queries(pa, q, k_mean, true)) return s;
  if (ld < pa->max_pages)
    return set_error(SA_ERR_INVALID_ARG, "score row stride ld = %lld is below max_pages = %d",
                     static_cast<long long>(ld), pa->max_pages);
  if (pa->T > 0 && !scores) return set_error(SA_ERR_INVALID_ARG, "scores must be a device pointer");
  if (!aligned(scores, 4)) return set_error(SA_ERR_INVALID_ARG, "scores must be 4-byte aligned");
  if (sa_status s = check_ws(ws, ws_bytes, 256)) return s;
  cudaError_t e = sa::launch_page_scores(*pa, q, k_mean, scores, ld, 0, nullptr, nullptr, at<uint32_t>(ws, 0), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "page score launch");
}

sa_status sa_block_attn(const sa_paged_args *pa, const void *q, const int32_t *idx, int32_t K, int32_t local,
                        void *out, void *ws, size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged(pa, true)) return s;
  if (sa_status s = check_lists(K, local)) return s;
  if (sa_status s = check_queries(pa, q, nullptr, false)) return s;
  if (sa_status s = check_out(pa, out)) return s;
  if (pa->T > 0 && K > 0 && !idx) return set_error(SA_ERR_INVALID_ARG, "idx must be a device pointer");
  if (!aligned(idx, 4)) return set_error(SA_ERR_INVALID_ARG, "idx must be 4-byte aligned");
  if (sa_status s = check_ws(ws, ws_bytes, sa::kWsHeader + sa::block_attn_scratch(*pa, K, local))) return s;
  cudaError_t e =
      sa::launch_block_attn(*pa, q, idx, K, local, out, at<void>(ws, sa::kWsHeader), at<uint32_t>(ws, 0), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "block attention launch");
}

sa_status sa_fused_block_attn(const sa_paged_args *pa, const void *q, const void *k_mean, int32_t K, int32_t local,
                              int32_t *idx_out, void *out, void *ws, size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged(pa, true)) return s;
  if (sa_status s = check_lists(K, local)) return s;
  if (local < 1) return set_error(SA_ERR_INVALID_ARG, "the fused call needs local >= 1");
  if (sa_status s = check_queries(pa, q, k_mean, K > 0)) return s;
  if (sa_status s = check_out(pa, out)) return s;
  if (!aligned(idx_out, 4)) return set_error(SA_ERR_INVALID_ARG, "idx_out must be 4-byte aligned");
  const FusedLayout L = fused_layout(*pa, K, local);
  if (sa_status s = check_ws(ws, ws_bytes, L.total)) return s;
  uint32_t *status = at<uint32_t>(ws, 0);
  int32_t *idx = idx_out ? idx_out : at<int32_t>(ws, L.idx);
  if (K > 0) {
    int32_t *row_seq = at<int32_t>(ws, L.row_seq), *row_pos = at<int32_t>(ws, L.row_pos);
    float *scores = at<float>(ws, L.scores);
    cudaError_t e = sa::launch_page_scores(*pa, q, k_mean, scores, pa->max_pages, local, row_seq, row_pos, status,
                                           cu(stream));
    if (e != cudaSuccess) return cuda_fail(e, "page score launch");
    // one top-k row per token and KV head; its visible count is the number of
    // pages before the local ones
    sa_index_args ia{};
    ia.B = pa->B;
    ia.T = pa->T * pa->H_kv;
    ia.N_c = pa->max_pages;
    ia.r = pa->P;
    ia.q_seq = row_seq;
    ia.q_pos = row_pos;
    e = sa::launch_topk(scores, pa->max_pages, ia, K, idx, status, cu(stream));
    if (e != cudaSuccess) return cuda_fail(e, "top-k launch");
  }
  cudaError_t e = sa::launch_block_attn(*pa, q, idx, K, local, out, at<void>(ws, L.attn), status, cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "block attention launch");
}

sa_status sa_prefix_attn(const sa_paged_args *pa, const void *q, int32_t shared_pages, void *out, void *ws,
                         size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged(pa, true)) return s;
  if (sa_status s = check_shared(pa, shared_pages)) return s;
  if (sa_status s = check_queries(pa, q, nullptr, false)) return s;
  if (sa_status s = check_out(pa, out)) return s;
  if (sa_status s = check_ws(ws, ws_bytes, sa::kWsHeader + sa::prefix_attn_scratch(*pa, shared_pages))) return s;
  cudaError_t e =
      sa::launch_prefix_attn(*pa, q, shared_pages, out, at<void>(ws, sa::kWsHeader), at<uint32_t>(ws, 0), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "prefix attention launch");
}

}  // extern "C"
