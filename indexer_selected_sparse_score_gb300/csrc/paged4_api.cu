// C ABI of the paged cache held in 4 bits (include/sa.h, sa_paged4_args): argument
// checks on the host, workspace carve-up and the launches of each entry point.
#include <algorithm>
#include <cmath>

#include "internal.h"

namespace {

using sa::set_error;

using sa::kWsHeader;
static_assert(sa::kWsCounters + 4 * sa::kAttn4Counters <= kWsHeader, "header");

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sa_status cuda_fail(cudaError_t e, const char *what) {
  return set_error(SA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool power_of_two(float x) {
  int e;
  return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e >= -59 && e <= 61;
}

sa_status check_paged4(const sa_paged4_args *pa, bool need_keys, bool need_values) {
  if (!pa) return set_error(SA_ERR_INVALID_ARG, "paged4 args pointer is NULL");
  if (sa_status s = sa::check_paged(&pa->p, false)) return s;
  if (!power_of_two(pa->k_gain) || !power_of_two(pa->v_gain))
    return set_error(SA_ERR_INVALID_ARG, "k_gain %g, v_gain %g: need powers of two in [2^-60, 2^60]",
                     static_cast<double>(pa->k_gain), static_cast<double>(pa->v_gain));
  if ((need_keys && (!pa->p.K || !pa->K_scale)) || (need_values && (!pa->p.V || !pa->V_scale)))
    return set_error(SA_ERR_INVALID_ARG, "the codes and scales of K%s must be device pointers", need_values ? " and V" : "");
  if (!aligned(pa->p.K, 16) || !aligned(pa->p.V, 16) || !aligned(pa->K_scale, 16) || !aligned(pa->V_scale, 16))
    return set_error(SA_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  return SA_OK;
}

sa_status check_ws(void *ws, size_t ws_bytes, size_t need) {
  if (!ws) return set_error(SA_ERR_WORKSPACE, "workspace pointer is NULL");
  if (!aligned(ws, 16)) return set_error(SA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (ws_bytes < need) return set_error(SA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  return SA_OK;
}

sa_status check_records(const sa_paged4_args *pa, const void *weight, const void *born, int64_t ld) {
  if (!aligned(weight, 4) || !aligned(born, 4))
    return set_error(SA_ERR_INVALID_ARG, "weight and born must be 4-byte aligned");
  if (ld < static_cast<int64_t>(pa->p.max_pages) * pa->p.P)
    return set_error(SA_ERR_INVALID_ARG, "record row stride ld = %lld is below max_pages * P = %lld",
                     static_cast<long long>(ld), static_cast<long long>(pa->p.max_pages) * pa->p.P);
  return SA_OK;
}

sa_status check_rows(const sa_paged4_args *pa, const void *q) {
  if (!std::isfinite(pa->p.scale)) return set_error(SA_ERR_INVALID_ARG, "scale is not finite");
  if (pa->p.T > 0 && !q) return set_error(SA_ERR_INVALID_ARG, "q must be a device pointer");
  if (!aligned(q, 16)) return set_error(SA_ERR_INVALID_ARG, "q must be 16-byte aligned");
  return SA_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

uint32_t *status_of(void *ws) { return static_cast<uint32_t *>(ws); }
void *scratch_of(void *ws) { return static_cast<char *>(ws) + kWsHeader; }
cudaStream_t cu(sa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

size_t sa_paged4_workspace_size(const sa_paged4_args *pa) {
  if (check_paged4(pa, false, false) != SA_OK) return 0;
  return kWsHeader + std::max({sa::attn4_scratch(*pa), sa::weights4_scratch(*pa), sa::evict4_scratch(*pa)});
}

sa_status sa_paged4_append(const sa_paged4_args *pa, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           const void *q, int64_t q_stride, void *q_out, const sa_rope_args *rope, int32_t rope_halves,
                           const int32_t *rope_pos, float *weight, int32_t *born, int64_t ld, void *ws, size_t ws_bytes,
                           sa_stream_t stream) {
  if (sa_status s = check_paged4(pa, pa && pa->p.T > 0, pa && pa->p.T > 0)) return s;
  if (sa_status s = sa::check_append(&pa->p, k, k_stride, v, v_stride, q, q_stride, q_out, rope, 32)) return s;
  if (!aligned(rope_pos, 4)) return set_error(SA_ERR_INVALID_ARG, "rope_pos must be 4-byte aligned");
  if ((weight == nullptr) != (born == nullptr))
    return set_error(SA_ERR_INVALID_ARG, "weight and born go together");
  if (weight)
    if (sa_status s = check_records(pa, weight, born, ld)) return s;
  if (sa_status s = check_ws(ws, ws_bytes, 256)) return s;
  cudaError_t e = sa::launch_paged4_append(*pa, k, k_stride, v, v_stride, q, q_stride, q_out, rope, rope_halves != 0,
                                           rope_pos, weight, born, ld, status_of(ws), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "4-bit append launch");
}

sa_status sa_paged4_read(const sa_paged4_args *pa, void *k_out, void *v_out, void *ws, size_t ws_bytes,
                         sa_stream_t stream) {
  if (sa_status s = check_paged4(pa, k_out != nullptr, v_out != nullptr)) return s;
  if (pa->p.T > 0 && (!pa->p.q_seq || !pa->p.q_pos || !pa->p.page_table))
    return set_error(SA_ERR_INVALID_ARG, "q_seq, q_pos and page_table must be device pointers");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return set_error(SA_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  if (sa_status s = check_ws(ws, ws_bytes, 256)) return s;
  cudaError_t e = sa::launch_paged4_read(*pa, k_out, v_out, status_of(ws), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "4-bit read launch");
}

sa_status sa_paged4_attn(const sa_paged4_args *pa, const void *q, void *out, float *lse, void *ws, size_t ws_bytes,
                         sa_stream_t stream) {
  if (sa_status s = check_paged4(pa, pa && pa->p.T > 0, pa && pa->p.T > 0)) return s;
  if (sa_status s = check_rows(pa, q)) return s;
  if (pa->p.T > 0 && !out) return set_error(SA_ERR_INVALID_ARG, "out must be a device pointer");
  if (!aligned(out, 16) || !aligned(lse, 4))
    return set_error(SA_ERR_INVALID_ARG, "out must be 16-byte aligned, lse 4-byte aligned");
  if (sa_status s = check_ws(ws, ws_bytes, kWsHeader + sa::attn4_scratch(*pa))) return s;
  cudaError_t e = sa::launch_attn4(*pa, q, out, lse, scratch_of(ws),
                                   reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + sa::kWsCounters), status_of(ws),
                                   cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "4-bit attention launch");
}

sa_status sa_paged4_weights(const sa_paged4_args *pa, const void *q, const float *lse, float *weight, int64_t ld, void *ws,
                            size_t ws_bytes, sa_stream_t stream) {
  if (sa_status s = check_paged4(pa, pa && pa->p.T > 0, false)) return s;
  if (sa_status s = check_rows(pa, q)) return s;
  if (pa->p.T > 0 && (!lse || !weight)) return set_error(SA_ERR_INVALID_ARG, "lse and weight must be device pointers");
  if (!aligned(lse, 4)) return set_error(SA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (sa_status s = check_records(pa, weight, nullptr, ld)) return s;
  if (sa_status s = check_ws(ws, ws_bytes, kWsHeader + sa::weights4_scratch(*pa))) return s;
  cudaError_t e = sa::launch_weights4(*pa, q, lse, weight, ld, scratch_of(ws), status_of(ws), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "slot weights launch");
}

sa_status sa_paged4_evict(const sa_paged4_args *pa, const int32_t *length, const int32_t *newest, int32_t budget,
                          int32_t recent, const float *weight, const int32_t *born, float *weight_out, int32_t *born_out,
                          int64_t ld, int32_t *length_out, void *ws, size_t ws_bytes, sa_stream_t stream) {
  if (!pa) return set_error(SA_ERR_INVALID_ARG, "paged4 args pointer is NULL");
  sa_paged4_args a = *pa;  // the tokens of pa are not read
  a.p.T = 0;
  if (sa_status s = check_paged4(&a, true, true)) return s;
  if (static_cast<int64_t>(a.p.B) * a.p.H_kv > (1 << 26))
    return set_error(SA_ERR_UNSUPPORTED, "B * H_kv above 2^26");
  if (!a.p.page_table || !length || !newest || !weight || !born || !weight_out || !born_out || !length_out)
    return set_error(SA_ERR_INVALID_ARG, "page_table, length, newest, the records and length_out must be device pointers");
  if (!aligned(length, 4) || !aligned(newest, 4) || !aligned(length_out, 4))
    return set_error(SA_ERR_INVALID_ARG, "length, newest and length_out must be 4-byte aligned");
  if (budget < 1 || recent < 0 || recent > budget)
    return set_error(SA_ERR_INVALID_ARG, "budget %d, recent %d: need budget >= 1 and 0 <= recent <= budget", budget, recent);
  if (sa_status s = check_records(&a, weight, born, ld)) return s;
  if (sa_status s = check_records(&a, weight_out, born_out, ld)) return s;
  const size_t bytes = static_cast<size_t>(a.p.B) * a.p.H_kv * ld * 4, lens = static_cast<size_t>(a.p.B) * 4;
  if (overlap(weight, bytes, weight_out, bytes) || overlap(born, bytes, born_out, bytes) ||
      overlap(weight, bytes, born_out, bytes) || overlap(born, bytes, weight_out, bytes) ||
      overlap(weight_out, bytes, born_out, bytes) || overlap(length, lens, length_out, lens) ||
      overlap(newest, lens, length_out, lens))
    return set_error(SA_ERR_INVALID_ARG, "the records and lengths that are written may not overlap those that are read");
  if (sa_status s = check_ws(ws, ws_bytes, kWsHeader + sa::evict4_scratch(a))) return s;
  cudaError_t e = sa::launch_evict4(a, length, newest, budget, recent, weight, born, weight_out, born_out, ld, length_out,
                                    scratch_of(ws), status_of(ws), cu(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, "eviction launch");
}

}  // extern "C"
