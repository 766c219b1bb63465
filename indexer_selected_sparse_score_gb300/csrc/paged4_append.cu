// The writer and the reader of a paged cache held in 4 bits.
//
// append: rows in, rotated, rounded to bf16, and quantised (the angles are 64-bit
// fixed-point turns, 2^-64 of a turn off a position at most; a key whose rounding fp32 does
// not settle is carried as two floats, since one that is rounded the other way, one in
// 10^5 otherwise, may get another code or its block another scale): s = e4m3(max(amax / 6, 2^-9)) of every
// 16 values, codes = e2m1(z / s).  The gain is a power of two, so z = y / gain has
// bf16's eight significant bits and s four: z / s either is a midpoint between
// two codes or lies 2^-9 of it away (z 2^k and m s are integers below 2^8).  So
// the quotient is taken as z times the rounded 1 / s, rounded to 14 significant
// bits (which restores a midpoint and moves no other value across one), and
// the hardware's conversion rounds it as the exact quotient.
//
// Traffic per token: 4 D bytes of every key and value row pair in, 9/8 D out, 4 D
// of every query head; bound by HBM and issue for a prefill (10,907 tokens of 64 + 2 x 8
// heads 86 us, 4.9 TB/s, 62% of the issue slots), by its chain of loads for a decode step
// (64 tokens 5 us).  One CTA per token, its rows' loads issued before its page is
// known; a thread holds two chunks of eight values, the two halves of a block of
// 16, or (halves) of two blocks that it shares with its neighbour.
//
// read: a thread per 16 values (the same tokens 15 us).
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "paged4.cuh"
#include "paged_list.h"
#include "paged_turns.h"

namespace sa {
namespace {

constexpr int kThreads = 320;
constexpr int kMaxPairs = 64;

struct Turns {
  uint64_t f[kMaxPairs];  // turns per position, times 2^64
  float4 at[17];          // cosine and sine of k / 128 turns, each as two floats: c, s, the rest of c, of s
};

struct AppendParams {
  Paged4View c;
  const uint16_t *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;
  uint16_t *q_out;
  const int32_t *rope_pos;
  float *weight;
  int32_t *born;
  int64_t ld;
  float k_inv, v_inv;  // 1 / gain
  int q_heads;         // H, or 0 without queries
  int D, dim, halves;
  uint32_t *status;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// h + l = a + b exactly.
__device__ __forceinline__ void two_sum(float a, float b, float &h, float &l) {
  h = __fadd_rn(a, b);
  const float x = __fsub_rn(h, a);
  l = __fadd_rn(__fsub_rn(a, __fsub_rn(h, x)), __fsub_rn(b, x));
}

// Cosine and sine of ph 2^-64 turns to 2^-39 (2^-39.7 over 5 million angles), each as two floats.  The angle is k
// / 128 turns from the table, after whole quarters, and a rest of at most pi / 128, whose
// power series end after the fifth and the sixth power.
__device__ __forceinline__ float4 cos_sin(uint64_t ph, const float4 *at) {
  constexpr double kTurn = 6.283185307179586476925286766559 / 18446744073709551616.0;
  constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - static_cast<double>(kHi));
  const uint32_t quarter = static_cast<uint32_t>((ph + (uint64_t{1} << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(ph - (static_cast<uint64_t>(quarter) << 62));
  const int k = static_cast<int>((rest + (int64_t{1} << 56)) >> 57);  // -16 .. 16
  const int64_t d = rest - (static_cast<int64_t>(k) << 57);
  const float d_hi = __ll2float_rn(d), d_lo = __ll2float_rn(d - __float2ll_rn(d_hi));
  const float a = d_hi * kHi, a_lo = fmaf(d_hi, kHi, -a) + fmaf(d_hi, kLo, d_lo * kHi);
  const float z = a * a, z_lo = fmaf(a, a, -z) + 2.f * a * a_lo;
  const float sn_lo = fmaf(a * z, fmaf(z, 1.f / 120.f, -1.f / 6.f), a_lo);                   // sine: a + sn_lo
  const float m = -0.5f * z, m_lo = fmaf(z * z, fmaf(z, -1.f / 720.f, 1.f / 24.f), -0.5f * z_lo);  // cosine: 1 + m + m_lo
  float4 t = at[abs(k)];
  if (k < 0) {
    t.y = -t.y;
    t.w = -t.w;
  }
  // u + (u m + v sn) for (u, v) = (cosine, -sine) and (sine, cosine) of the table
  auto turned = [&](float u, float u_lo, float v, float v_lo, float &h, float &l) {
    const float p = u * m, p_lo = fmaf(u, m, -p), q = v * a, q_lo = fmaf(v, a, -q);
    float x, x_lo, y, y_lo;
    two_sum(p, q, x, x_lo);
    two_sum(u, x, y, y_lo);
    const float low = y_lo + (x_lo + (p_lo + q_lo + fmaf(u, m_lo, u_lo * m) + fmaf(v, sn_lo, v_lo * a) + u_lo));
    two_sum(y, low, h, l);
  };
  float4 o;
  turned(t.x, t.z, -t.y, -t.w, o.x, o.z);
  turned(t.y, t.w, t.x, t.z, o.y, o.w);
  if (quarter & 1) o = make_float4(-o.y, o.x, -o.w, o.z);
  if (quarter & 2) o = make_float4(-o.x, -o.y, -o.z, -o.w);
  return o;
}

// a c + b s (c, s as two floats) rounded once to fp32, but for 2^-39 of |a| + |b|: a rotated key
// whose bf16 is another one than the 64-bit value's (by way of fp32, as every conversion
// of one goes) may be given another code, or its block another scale.
__device__ __forceinline__ float exact_sum(float a, float c, float c_lo, float b, float s, float s_lo) {
  const float p = a * c, p_lo = fmaf(a, c, -p), q = b * s, q_lo = fmaf(b, s, -q);
  float x, x_lo, y, y_lo;
  two_sum(p, q, x, x_lo);
  two_sum(x, x_lo + (p_lo + q_lo + fmaf(a, c_lo, b * s_lo)), y, y_lo);
  return fabsf(y) <= 3.4028235e38f ? y : p + q;  // (infinities, NaN)
}

// What a key's rotation needs where fp32 does not settle its rounding.
struct ExactTurn {
  int64_t turn;
  const Turns *turns;
};

// (rarely called, and long)
__device__ __noinline__ float2 turn_exactly(float a, float b, uint64_t ph, const float4 *at) {
  const float4 t = cos_sin(ph, at);
  return make_float2(exact_sum(a, t.x, t.z, b, -t.y, -t.w), exact_sum(a, t.y, t.w, b, t.x, t.z));
}

// A pair (a, b) turned by c, s (fp32): y0, y1.  For keys (e): sine and cosine are off by
// 2^-23 and a step's rounding at most, products and sum by 2^-24 of the pair each, together
// by 5 2^-24 (|a| + |b|); a value that is that near a midpoint of bf16 (one in 3000 or so)
// is taken exactly.  (10,907 tokens of 64 + 2 x 8 heads, appended and read: 109 us; 99 without
// looking, 126 with every key taken exactly.)
template <bool kKey>
__device__ __forceinline__ void turn_pair(float a, float b, float2 cs, int pair, const ExactTurn &e, float &y0, float &y1) {
  y0 = a * cs.x - b * cs.y;
  y1 = a * cs.y + b * cs.x;
  if (kKey) {
    auto middle = [](float y) { return __uint_as_float((__float_as_uint(y) & 0xFFFF0000u) | 0x8000u); };
    const float err = 0x1.4p-22f * (fabsf(a) + fabsf(b));
    if (fabsf(y0 - middle(y0)) <= err || fabsf(y1 - middle(y1)) <= err) {
      const float2 y = turn_exactly(a, b, static_cast<uint64_t>(e.turn) * e.turns->f[pair], e.turns->at);
      y0 = y.x;
      y1 = y.y;
    }
  }
}

// Four adjacent pairs of one chunk, from `pair` on.
template <bool kKey>
__device__ __forceinline__ void rotate_adjacent(uint32_t (&w)[4], const float2 *cs, int pair, const ExactTurn &e) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y0, y1;
    turn_pair<kKey>(lo_f(w[i]), hi_f(w[i]), cs[pair + i], pair + i, e, y0, y1);
    w[i] = pack_bf16(y0, y1);
  }
}

// Eight pairs (u[e], w[e]) of two chunks half the rotated span apart.
template <bool kKey>
__device__ __forceinline__ void rotate_halves(uint32_t (&u)[4], uint32_t (&w)[4], const float2 *cs, int pair, const ExactTurn &e) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, x1, y0, y1;
    turn_pair<kKey>(lo_f(u[i]), lo_f(w[i]), cs[pair + 2 * i], pair + 2 * i, e, x0, y0);
    turn_pair<kKey>(hi_f(u[i]), hi_f(w[i]), cs[pair + 2 * i + 1], pair + 2 * i + 1, e, x1, y1);
    u[i] = pack_bf16(x0, x1);
    w[i] = pack_bf16(y0, y1);
  }
}

// Largest magnitude of a chunk of eight, NaN if one is.
__device__ __forceinline__ float chunk_top(const uint32_t (&w)[4], float inv) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(max_nan(m, fabsf(lo_f(w[i]) * inv)), fabsf(hi_f(w[i]) * inv));
  return m;
}

// Scale byte of a block whose largest magnitude is `top`.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  if (top != top) return 0x7Fu;
  const float s = fminf(fmaxf(__fdiv_rn(top, 6.f), 0x1p-9f), 448.f);
  return __nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3);
}

// Codes of a chunk of eight values over a scale (byte).
__device__ __forceinline__ uint32_t chunk_codes(const uint32_t (&w)[4], float inv, uint32_t scale) {
  if (scale == 0x7Fu) return 0u;
  const float r = __frcp_rn(e4m3_bits_to_float(static_cast<uint8_t>(scale)));
  auto quotient = [&](float y) {
    // 14 significant bits, to the nearest (infinities stay)
    return __uint_as_float((__float_as_uint(y * inv * r) + 0x200u) & ~0x3FFu);
  };
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t two;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tmov.b32 %0, {b, 0, 0, 0};\n\t}"
        : "=r"(two)
        : "f"(quotient(hi_f(w[i]))), "f"(quotient(lo_f(w[i]))));
    out |= two << (8 * i);
  }
  return out;
}

__global__ void __launch_bounds__(kThreads, 4)
append4_kernel(const AppendParams p, const __grid_constant__ Turns turns) {
  __shared__ float2 cs[kMaxPairs];
  const PagedView &pv = p.c.v;
  const int t = blockIdx.x, threads = blockDim.x;
  const int log_upr = p.D == 128 ? 3 : 2;  // of the units (two chunks of eight values) of a row
  const int kept = (p.D - p.dim) >> 4;     // units before the rotated span
  const int span = p.dim >> 3;             // chunks of the rotated span
  const int first = (p.D >> 3) - span;     // first rotated chunk
  const int units = (p.q_heads + 2 * pv.H_kv) << log_upr;
  // chunks of unit u within its row: two neighbours, or the two halves of eight
  // pairs; a row's last units hold its rotated span (values are rotated in
  // halves whether or not they are a value row's, so that rows are alike)
  auto chunks = [&](int u, int &c0, int &c1) {
    const int i = u & ((1 << log_upr) - 1), j = i - kept;
    const bool half = p.halves && j >= 0;
    c0 = half ? first + j : 2 * i;
    c1 = half ? c0 + (span >> 1) : 2 * i + 1;
    return half;
  };
  constexpr int kUnits = 2;
  bool ok = false, tabled = false;
  ExactTurn exact{0, &turns};
  int page = -1, slot = 0;
  for (int base = 0; base < units; base += kUnits * threads) {
    uint32_t x[kUnits][4], y[kUnits][4];
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int u = base + e * threads + threadIdx.x;
      if (u >= units) continue;
      int c0, c1;
      chunks(u, c0, c1);
      const int row = u >> log_upr, h = row - p.q_heads;
      const uint16_t *src = h < 0        ? p.q + t * p.q_stride + static_cast<int64_t>(row) * p.D
                            : h < pv.H_kv ? p.k + t * p.k_stride + static_cast<int64_t>(h) * p.D
                                          : p.v + t * p.v_stride + static_cast<int64_t>(h - pv.H_kv) * p.D;
      *reinterpret_cast<uint4 *>(x[e]) = *reinterpret_cast<const uint4 *>(src + 8 * c0);
      *reinterpret_cast<uint4 *>(y[e]) = *reinterpret_cast<const uint4 *>(src + 8 * c1);
    }
    if (!tabled) {
      const int turn = p.rope_pos ? p.rope_pos[t] : pv.q_pos[t];
      exact.turn = turn;
      int b, pos;
      ok = load_paged_token(pv, t, p.status, threadIdx.x == 0, b, pos);
      if (ok) {
        page = load_page(pv, b, pos >> pv.logP, p.status, threadIdx.x == 0);
        slot = pos & (pv.P - 1);
        if (threadIdx.x < p.dim / 2) {
          // the turn's first 32 bits in fp32, and a step along the circle by what that rounds off
          const uint64_t ph = static_cast<uint64_t>(exact.turn) * turns.f[threadIdx.x] + (uint64_t{1} << 31);
          const int32_t part = static_cast<int32_t>(ph >> 32);
          const float x = static_cast<float>(part);
          const float step = static_cast<float>(part - static_cast<int64_t>(x)) * static_cast<float>(3.14159265358979323846 * 0x1p-31);
          float sn, c;
          sincospif(x * 0x1p-31f, &sn, &c);
          cs[threadIdx.x] = make_float2(fmaf(-sn, step, c), fmaf(c, step, sn));
        }
        if (p.weight) {
          for (int h = threadIdx.x; h < pv.H_kv; h += threads) {
            const int64_t at = (static_cast<int64_t>(b) * pv.H_kv + h) * p.ld + pos;
            p.weight[at] = 0.f;
            p.born[at] = turn;
          }
        }
      }
      __syncthreads();
      tabled = true;
    }
    if (!ok) return;  // the whole CTA alike
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int u = base + e * threads + threadIdx.x;
      const bool mine = u < units;
      if (!__any_sync(0xffffffffu, mine)) continue;
      int c0, c1;
      const bool half = chunks(u, c0, c1);
      const int row = u >> log_upr, h = row - p.q_heads;
      if (mine && h < pv.H_kv && c0 >= first) {
        if (half) {
          if (h >= 0)
            rotate_halves<true>(x[e], y[e], cs, 8 * (c0 - first), exact);
          else
            rotate_halves<false>(x[e], y[e], cs, 8 * (c0 - first), exact);
        } else if (h >= 0) {
          rotate_adjacent<true>(x[e], cs, 4 * (c0 - first), exact);
          rotate_adjacent<true>(y[e], cs, 4 * (c1 - first), exact);
        } else {
          rotate_adjacent<false>(x[e], cs, 4 * (c0 - first), exact);
          rotate_adjacent<false>(y[e], cs, 4 * (c1 - first), exact);
        }
      }
      if (mine && h < 0) {
        uint16_t *dst = p.q_out + (static_cast<int64_t>(t) * pv.H + row) * p.D;
        *reinterpret_cast<uint4 *>(dst + 8 * c0) = *reinterpret_cast<uint4 *>(x[e]);
        *reinterpret_cast<uint4 *>(dst + 8 * c1) = *reinterpret_cast<uint4 *>(y[e]);
      }
      const bool held = mine && h >= 0 && page >= 0;
      if (!__any_sync(0xffffffffu, held)) continue;
      const bool key = h < pv.H_kv;
      const float inv = key ? p.k_inv : p.v_inv;
      float tx = held ? chunk_top(x[e], inv) : 0.f, ty = held ? chunk_top(y[e], inv) : 0.f;
      const float ox = __shfl_xor_sync(0xffffffffu, tx, 1), oy = __shfl_xor_sync(0xffffffffu, ty, 1);
      if (!held) continue;
      if (half) {  // the neighbour holds the blocks' other chunks
        tx = max_nan(tx, ox);
        ty = max_nan(ty, oy);
      } else {
        tx = ty = max_nan(tx, ty);
      }
      const uint32_t sx = scale_byte(tx), sy = half ? scale_byte(ty) : sx;
      const uint32_t wx = chunk_codes(x[e], inv, sx), wy = chunk_codes(y[e], inv, sy);
      const int64_t at = (static_cast<int64_t>(page) * pv.H_kv + (key ? h : h - pv.H_kv)) * pv.P + slot;
      uint8_t *codes = (key ? p.c.K : p.c.V) + at * (p.D / 2), *scales = (key ? p.c.Ks : p.c.Vs) + at * (p.D / 16);
      if (half) {
        *reinterpret_cast<uint32_t *>(codes + 4 * c0) = wx;
        *reinterpret_cast<uint32_t *>(codes + 4 * c1) = wy;
        if (!(c0 & 1)) scales[c0 >> 1] = static_cast<uint8_t>(sx);
        if (!(c1 & 1)) scales[c1 >> 1] = static_cast<uint8_t>(sy);
      } else {
        *reinterpret_cast<uint2 *>(codes + 4 * c0) = make_uint2(wx, wy);
        scales[c0 >> 1] = static_cast<uint8_t>(sx);
      }
    }
  }
}

// CTA (x): tokens; a thread per block of 16 values.
__global__ void __launch_bounds__(256)
read4_kernel(const Paged4View c, int D, float k_gain, float v_gain, uint16_t *k_out, uint16_t *v_out, int kinds,
             uint32_t *status) {
  const PagedView &pv = c.v;
  const int t = blockIdx.x;
  int b, pos;
  if (!load_paged_token(pv, t, status, threadIdx.x == 0, b, pos)) return;
  const int page = load_page(pv, b, pos >> pv.logP, status, threadIdx.x == 0);
  if (page < 0) return;
  const int log_b = D == 128 ? 3 : 2;
  for (int u = threadIdx.x; u < (kinds * pv.H_kv) << log_b; u += blockDim.x) {
    const int row = u >> log_b, blk = u & ((1 << log_b) - 1);
    const bool key = k_out && row < pv.H_kv;
    const int h = row < pv.H_kv ? row : row - pv.H_kv;
    const int64_t at = (static_cast<int64_t>(page) * pv.H_kv + h) * pv.P + (pos & (pv.P - 1));
    const uint2 w = *reinterpret_cast<const uint2 *>((key ? c.K : c.V) + at * (D / 2) + 8 * blk);
    const float s = (key ? k_gain : v_gain) * e4m3_bits_to_float((key ? c.Ks : c.Vs)[at * (D / 16) + blk]);
    __half2 d[8];
    e2m1x8_to_half2(w.x, *reinterpret_cast<__half2(*)[4]>(d));
    e2m1x8_to_half2(w.y, *reinterpret_cast<__half2(*)[4]>(d + 4));
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = __half22float2(d[i]);
      o[i] = pack_bf16(f.x * s, f.y * s);
    }
    uint4 *dst = reinterpret_cast<uint4 *>((key ? k_out : v_out) + (static_cast<int64_t>(t) * pv.H_kv + h) * D + 16 * blk);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_paged4_append(const sa_paged4_args &pa, const void *k, int64_t k_stride, const void *v,
                                 int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                 const sa_rope_args *rope, bool halves, const int32_t *rope_pos, float *weight,
                                 int32_t *born, int64_t ld, uint32_t *status, cudaStream_t stream) {
  if (pa.p.T == 0) return cudaSuccess;
  AppendParams p;
  p.c = paged4_view(pa);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.q = static_cast<const uint16_t *>(q);
  const int64_t kv_row = static_cast<int64_t>(pa.p.H_kv) * pa.p.D;
  p.k_stride = k_stride ? k_stride : kv_row;
  p.v_stride = v_stride ? v_stride : kv_row;
  p.q_stride = q_stride ? q_stride : static_cast<int64_t>(pa.p.H) * pa.p.D;
  p.q_out = static_cast<uint16_t *>(q_out);
  p.rope_pos = rope_pos;
  p.weight = weight;
  p.born = born;
  p.ld = ld;
  p.k_inv = 1.f / pa.k_gain;
  p.v_inv = 1.f / pa.v_gain;
  p.q_heads = q ? pa.p.H : 0;
  p.D = pa.p.D;
  p.dim = rope ? rope->dim : 0;
  p.halves = halves ? 1 : 0;
  p.status = status;
  // (a table of the circle, the same for every call)
  static const struct Circle {
    float4 at[17];
    Circle() {
      for (int k = 0; k <= 16; ++k) {
        const double c = std::cos(k * 3.14159265358979323846 / 64.0), s = std::sin(k * 3.14159265358979323846 / 64.0);
        const float ch = static_cast<float>(c), sh = static_cast<float>(s);
        at[k] = make_float4(ch, sh, static_cast<float>(c - ch), static_cast<float>(s - sh));
      }
    }
  } circle;
  Turns turns{};
  std::copy(circle.at, circle.at + 17, turns.at);
  const RopeRamp ramp = p.dim > 0 ? rope_ramp(*rope) : RopeRamp{0.0, 0.0};
  for (int i = 0; i < p.dim / 2; ++i) turns.f[i] = turns_of(rope_frequency(*rope, ramp, i));
  const int units = (p.q_heads + 2 * pa.p.H_kv) * (pa.p.D / 16);
  // few tokens: as many threads as may be, so that a CTA's loads go out at once; many: no more than
  // a thread has two units
  const int threads =
      pa.p.T > 4 * sm_count() ? std::min(std::max((units / 2 + 31) & ~31, kMaxPairs), kThreads) : kThreads;
  return launch_ex(false, append4_kernel, dim3(pa.p.T), dim3(threads), 0, stream, 1, p, turns);
}

cudaError_t launch_paged4_read(const sa_paged4_args &pa, void *k_out, void *v_out, uint32_t *status,
                               cudaStream_t stream) {
  const int kinds = (k_out ? 1 : 0) + (v_out ? 1 : 0);
  if (pa.p.T == 0 || kinds == 0) return cudaSuccess;
  const int units = kinds * pa.p.H_kv * (pa.p.D / 16);
  return launch_ex(false, read4_kernel, dim3(pa.p.T), dim3(std::min((units + 31) & ~31, 256)), 0, stream, 1,
                   paged4_view(pa), pa.p.D, pa.k_gain, pa.v_gain, static_cast<uint16_t *>(k_out),
                   static_cast<uint16_t *>(v_out), kinds, status);
}

}  // namespace sa
