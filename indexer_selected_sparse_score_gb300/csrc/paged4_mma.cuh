// Warp-level products over rows held in 4 bits, and the softmax of a few columns
// between them (see paged4_attn.cu for the layouts).
#pragma once

#include <cfloat>

#include "paged4.cuh"

namespace sa {

// Weights are 2^(logit - ref): ref is 2^kRefHead below the logit that set it,
// and is raised when a logit passes it by kRefTop (log2 units).
constexpr float kRefHead = 6.f, kRefTop = 14.f;

__device__ __forceinline__ float exp2_fast(float x) {  // relative error about 2^-22, 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), fp16.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values (lane (g, t): row g, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One warp brings a column of the queries into fragments of the K Q^T product as fp16,
// scaled by a power of two.  load_column: a lane's part of kDim bf16 at src (zeros
// unless in).
template <int kDim>
__device__ __forceinline__ void load_column(const uint16_t *src, bool in, int lane, uint32_t (&w)[kDim / 64]) {
#pragma unroll
  for (int i = 0; i < kDim / 64; ++i) w[i] = 0;
  if (in) {
    if constexpr (kDim == 128)
      *reinterpret_cast<uint2 *>(w) = reinterpret_cast<const uint2 *>(src)[lane];
    else
      w[0] = reinterpret_cast<const uint32_t *>(src)[lane];
  }
}

// stage_column: as column `col`; returns 1 / factor.  Fragment (nt, i) of lane (g, t):
// 16 bytes, the values kDim / 4 t + 8 i .. + 7 of column 8 nt + g.
template <int kDim>
__device__ __forceinline__ float stage_column(uint32_t (&w)[kDim / 64], int col, int lane, uint4 *qf) {
  constexpr int V = kDim / 32;
  float x[V], top = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = bf16_bits_to_float(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
    top = fmaxf(top, fabsf(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float f = to_half_factor(top);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) w[i] = as_u32(__floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f));
  const int at = V * (lane & 7);  // within the quarter of the row that lane >> 3 holds
  uint8_t *dst = reinterpret_cast<uint8_t *>(qf + ((col >> 3) * (kDim / 32) + (at >> 3)) * 32 + (col & 7) * 4 + (lane >> 3)) +
                 2 * (at & 7);
  if constexpr (V == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(dst) = w[0];
  return 1.f / f;
}

// Key rows g and g + 8 of 16 (codes at k, scales at ks): words of codes and, per
// block of 16 values, the scale as an fp16 pair.
template <int kDim>
struct KeyRows {
  static constexpr int kWords = kDim / 32;  // of a row, per lane
  uint32_t w[2][kWords];
  __half2 s[2][kWords / 2];
  __device__ __forceinline__ void load(const uint8_t *k, const uint8_t *ks, int g, int t) {
    k += g * (kDim / 2) + t * (kDim / 8);
    ks += g * (kDim / 16) + t * (kDim / 64);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (kDim == 128) {
        *reinterpret_cast<uint4 *>(w[r]) = *reinterpret_cast<const uint4 *>(k + 512 * r);
        const __half2 two = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(ks + 64 * r));
        s[r][0] = __low2half2(two);
        s[r][1] = __high2half2(two);
      } else {
        *reinterpret_cast<uint2 *>(w[r]) = *reinterpret_cast<const uint2 *>(k + 256 * r);
        s[r][0] = __low2half2(e4m3x2_to_half2(ks[32 * r]));
      }
    }
  }
  // Values 8 i .. 8 i + 7 of the lane's quarter of row r.
  __device__ __forceinline__ void values(int r, int i, __half2 (&d)[4]) const {
    e2m1x8_to_half2(w[r][i], d);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = __hmul2(d[j], s[r][i >> 1]);
  }
};

// A warp's columns: reference, sum (of this lane's rows) and O.
template <int kDim, int NT>
struct Columns {
  static constexpr int kMt = kDim / 16, kFr = kDim / 32;
  float o[NT][kMt][4], ref[NT][2], l[NT][2], cs[NT][2];
  int lim[NT][2];

  __device__ __forceinline__ void begin(const float2 *cols, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 c = cols[8 * nt + 2 * (lane & 3) + e];
        cs[nt][e] = c.x;
        lim[nt][e] = __float_as_int(c.y);
        ref[nt][e] = -FLT_MAX;  // (no logit yet; a finite one is larger)
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
    }
  }

  // 32 keys, slots base .. base + 31: codes and scales at k, ks, v, vs (shared
  // memory).  edge: some of them are no keys of some column: they lie past its limit
  // or past `last`, or the half that they are in has no page (bit of `held` clear; the
  // bytes of such slots may be anything).  A block of V that is NaN in a slot that
  // not every column attends is left to the caller (poison: the lowest such slot per
  // block).
  __device__ __forceinline__ void step(const uint8_t *k, const uint8_t *ks, const uint8_t *v, const uint8_t *vs, int base,
                                       bool edge, uint32_t held, int low, int last, const uint4 *qf, int *poison, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[2][NT][4] = {};
    {
      KeyRows<kDim> rows[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) rows[h].load(k + h * (8 * kDim), ks + h * kDim, g, t);
#pragma unroll
      for (int i = 0; i < kFr; ++i) {
        uint4 q[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) q[nt] = qf[(nt * kFr + i) * 32 + lane];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          __half2 a[4], b[4];
          rows[h].values(0, i, a);
          rows[h].values(1, i, b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(s[h][nt], as_u32(a[0]), as_u32(b[0]), as_u32(a[1]), as_u32(b[1]), q[nt].x, q[nt].y);
            mma_16816(s[h][nt], as_u32(a[2]), as_u32(b[2]), as_u32(a[3]), as_u32(b[3]), q[nt].z, q[nt].w);
          }
        }
      }
    }
    // logits relative to the references (the product rounded as the reference was: a
    // fused one would differ from it by all of a huge logit's last place)
    float x[2][NT][4], top = -INFINITY;
    auto relate = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[h][nt][e] = __fadd_rn(__fmul_rn(s[h][nt][e], cs[nt][e & 1]), -ref[nt][e & 1]);
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((held >> h) & 1u) || base + 16 * h + g + 4 * (e & 2) > lim[nt][e & 1]) x[h][nt][e] = -INFINITY;
      }
    };
    relate();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        top = fmaxf(fmaxf(top, fmaxf(x[h][nt][0], x[h][nt][1])), fmaxf(x[h][nt][2], x[h][nt][3]));
    if (__any_sync(0xffffffffu, top > kRefTop)) {
      raise(s, x);
      relate();
    }
    uint32_t pw[2][NT][2];  // weights of keys 0-7 and 8-15 of a half, transposed
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[h][nt][e] = exp2_fast(x[h][nt][e]);
        l[nt][0] += x[h][nt][0] + x[h][nt][2];
        l[nt][1] += x[h][nt][1] + x[h][nt][3];
        pw[h][nt][0] = transpose_8x8(as_u32(__floats2half2_rn(x[h][nt][0], x[h][nt][1])));
        pw[h][nt][1] = transpose_8x8(as_u32(__floats2half2_rn(x[h][nt][2], x[h][nt][3])));
      }
    // values: lane (g, t) has kDim / 8 values of keys 2t, 2t + 1, 2t + 8, 2t + 9
    constexpr int kVw = kDim / 64;  // words of codes
    v += 2 * t * (kDim / 2) + g * (kDim / 16);
    vs += 2 * t * (kDim / 16) + (kDim == 128 ? g : g >> 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t y[4][kVw], sc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 16 * h + (j & 1) + 4 * (j & 2);
        if constexpr (kDim == 128)
          *reinterpret_cast<uint2 *>(y[j]) = *reinterpret_cast<const uint2 *>(v + key * 64);
        else
          y[j][0] = *reinterpret_cast<const uint32_t *>(v + key * 32);
        sc[j] = vs[key * (kDim / 16)];
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int slot = base + 16 * h + 2 * t + (j & 1) + 4 * (j & 2);
          if (slot > last || !((held >> h) & 1u)) {
            sc[j] = 0;
          } else if (slot > low && e4m3_is_nan(sc[j])) {
            sc[j] = 0;
            atomicMin(&poison[kDim == 128 ? g : g >> 1], slot);
          }
        }
      }
      const __half2 s01 = e4m3x2_to_half2(sc[0] | sc[1] << 8), s23 = e4m3x2_to_half2(sc[2] | sc[3] << 8);
#pragma unroll
      for (int i = 0; i < kVw; ++i) {
        // pairs (key, key + 1) of the even and of the odd values
        const uint32_t e01 = (y[0][i] & 0x0F0F0F0Fu) | ((y[1][i] << 4) & 0xF0F0F0F0u);
        const uint32_t o01 = ((y[0][i] >> 4) & 0x0F0F0F0Fu) | (y[1][i] & 0xF0F0F0F0u);
        const uint32_t e23 = (y[2][i] & 0x0F0F0F0Fu) | ((y[3][i] << 4) & 0xF0F0F0F0u);
        const uint32_t o23 = ((y[2][i] >> 4) & 0x0F0F0F0Fu) | (y[3][i] & 0xF0F0F0F0u);
        __half2 a0[4], a1[4], a2[4], a3[4];
        e2m1x8_to_half2(e01, a0);
        e2m1x8_to_half2(o01, a1);
        e2m1x8_to_half2(e23, a2);
        e2m1x8_to_half2(o23, a3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b0 = as_u32(__hmul2(a0[j], s01)), b1 = as_u32(__hmul2(a1[j], s01));
          const uint32_t b2 = as_u32(__hmul2(a2[j], s23)), b3 = as_u32(__hmul2(a3[j], s23));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][4 * i + j], b0, b1, b2, b3, pw[h][nt][0], pw[h][nt][1]);
        }
      }
    }
  }

  // Raises the references that logits have passed; sums and O shrink in step.  s: the
  // products, x: -inf where there is no key.
  __device__ __forceinline__ void raise(const float (&s)[2][NT][4], const float (&x)[2][NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = e; k < 4; k += 2)
            if (x[h][nt][k] != -INFINITY) top = fmaxf(top, __fmul_rn(s[h][nt][k], cs[nt][e]));
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        // (passed as step() sees it: r + kRefTop would be rounded, by more than fp16 has room for
        // where a step of fp32 is 4 or more)
        const float r = ref[nt][e], nr = __fadd_rn(top, -r) > kRefTop ? top - kRefHead : r;
        const float f = r == nr ? 1.f : exp2_fast(r - nr);
        ref[nt][e] = nr;
        l[nt][e] *= f;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          o[nt][mt][e] *= f;
          o[nt][mt][e + 2] *= f;
        }
      }
  }

  // The sums over the warp's keys, in every lane of a column.
  __device__ __forceinline__ void sum_up() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
  }
};

}  // namespace sa
