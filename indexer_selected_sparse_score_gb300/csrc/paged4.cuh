// Device-side view and the number formats of a paged cache held in 4 bits
// (sa_paged4_args), shared by its kernels.
#pragma once

#include <cuda_fp16.h>

#include "paged.cuh"

namespace sa {

struct Paged4View {
  PagedView v;
  uint8_t *K, *V, *Ks, *Vs;
};

inline Paged4View paged4_view(const sa_paged4_args &pa) {
  return Paged4View{paged_view(pa.p), static_cast<uint8_t *>(pa.p.K), static_cast<uint8_t *>(pa.p.V),
                    static_cast<uint8_t *>(pa.K_scale), static_cast<uint8_t *>(pa.V_scale)};
}

// Eight e2m1 codes (code i in bits 4 i .. 4 i + 3) as fp16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, __half2 (&d)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<__half2 *>(&r[i]);
}

// Two e4m3 scales (the lower byte first) as an fp16 pair, exact.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<__half2 *>(&r);
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ bool e4m3_is_nan(uint32_t byte) { return (byte & 0x7Fu) == 0x7Fu; }

// The largest power of two that brings a row whose largest magnitude is `top`
// below 2^15 (fp16 holds it then, and what is 2^-29 of it still to its last
// bit); a row of zeros or of infinities has one all the same.
__device__ __forceinline__ float to_half_factor(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // top < 2^(e + 1), e = 128 for infinities
  return __uint_as_float(static_cast<uint32_t>(127 + 14 - max(e, -100)) << 23);
}

}  // namespace sa
