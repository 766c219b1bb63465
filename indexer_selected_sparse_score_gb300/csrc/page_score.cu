// The cheap score of the pages of a paged cache: scale times the product of
// the summed queries of a KV head's group with the mean key of every complete
// page.
//
// The score is an fp32 number, so the summed query enters the tensor cores as
// three bf16 pieces (q = hi + mid + lo to 2^-24 of it) against the bf16 means:
// products exact, sums fp32.  Of an infinite sum or mean the lower pieces make
// NaN (0 x inf, inf - inf); there the upper pieces' product alone is the score.
// Two kernels.  With few tokens per sequence (a
// decode step) every mean key is met by one token: a stream of 2 D-byte rows
// bound by HBM; there a warp-level product takes 16 pages' rows straight from
// registers against the three pieces as columns (on the CUDA cores the unpacking
// and reducing of every row had cost more issue slots than the stream leaves).
// With many tokens per sequence (a prefill chunk) it is a product of 128 tokens
// with 128 pages at a time (tcgen05), bound by reading the queries and writing
// the scores.
//
// Measured, heads of 128, pages of 64: 64 tokens (64 over 8 heads) at 32 K to
// 64 K positions 23.8 us, 4.4 TB/s of the 104 MB it must move (5.7 TB/s once
// started: two chains of loads pass before the first mean keys arrive); a
// 4096-token chunk (64 over 4 heads) at 28 K positions 33 us, 3.1 TB/s (the
// queries' 67 MB on the 128 SMs that have a tile, then the scores, little of the
// two overlapping); 4 tokens (16 over 2 heads) at 4 K positions 6.4 to 7.3 us
// called from Python, one launch and its chain of loads.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

struct ScoreParams {
  PagedView pv;
  const uint16_t *q, *k_mean;
  float *scores;
  int64_t ld;
  float scale;
  int local;
  int32_t *row_seq, *row_pos;  // [T, H_kv] or NULL: the top-k's token arrays
  uint32_t *status;
};

__device__ __forceinline__ void add_bf16x8(float (&a)[8], uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] += __uint_as_float(w[i] << 16);
    a[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Sum of queries first, first + step, .. below G of (token t, KV head h) over 8
// dims from chunk c, kLoads in flight at a time (a loop left to the compiler
// takes what is left of its unrolling, all of a small group, one by one).
template <int kDim, int kLoads>
__device__ __forceinline__ void sum_queries(const ScoreParams &p, int64_t t, int h, int G, int c, int first, int step,
                                            float (&a)[8]) {
  const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (t * p.pv.H + static_cast<int64_t>(h) * G) * kDim) + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 0.f;
  for (int g = first; g < G; g += kLoads * step) {
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (g + i * step < G) x[i] = src[(g + i * step) * (kDim / 8)];
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) add_bf16x8(a, x[i]);
  }
}

__device__ __forceinline__ void write_row_token(const ScoreParams &p, int64_t row, bool ok, int b, int pos) {
  const int f = ok ? max((pos >> p.pv.logP) + 1 - p.local, 0) : 0;
  p.row_seq[row] = ok ? b : -1;
  p.row_pos[row] = max(f * p.pv.P - 1, 0);
}

// Product of a summed query's upper piece with a mean key; the query's 16-byte
// chunk c lies at q, or at its place in row `row` of a 128-byte-swizzled tile of
// 64-dim blocks.
template <int kDim, uint32_t kBlock = 0>
__device__ float upper_product(const void *q, int row, const uint16_t *k) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < kDim / 8; ++c) {
    const uint32_t off = kBlock ? (c >> 3) * kBlock + sw128_offset(row, 16u * (c & 7)) : 16u * c;
    float x[8] = {}, y[8] = {};
    add_bf16x8(x, *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(q) + off));
    add_bf16x8(y, reinterpret_cast<const uint4 *>(k)[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
  }
  return sum;
}

// ------------------------------------------------------- one token at a time

constexpr int kThreads = 256;
constexpr int kHeads = 8;       // KV heads of a CTA
constexpr int kSumLoads = 8;    // queries a thread has in flight
constexpr int kPass = 16;       // 16-page tiles of one pass over the shared memory

// D += A B, 16 x 8 x 16, bf16 inputs.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// CTA (t S + s, z): the s-th of S shares of the 16-page tiles that token t sees,
// for KV heads 8 z .. 8 z + 7.  (Sharing the tiles of all tokens out evenly cost
// more than the uneven tokens do: a scan of the positions first, and a second
// chain of dependent loads wherever a CTA crossed into another token.)  A warp's
// item is a tile of one head: A rows are the pages, B columns 0-2 the query's
// pieces.  The order of the dims within a product is free, so lane 4 g + i holds
// 16-byte chunks i, i + 4, .. of rows g and g + 8 as they lie in memory, two
// k-steps a chunk.
template <int kDim>
__global__ void __launch_bounds__(kThreads, 4)
score_token_kernel(const ScoreParams p, int S) {
  constexpr int kChunks = kDim / 8, kLoads = kChunks / 4;  // of a row; a lane's loads of it
  __shared__ __align__(16) uint16_t qs[kHeads][3][kDim];
  __shared__ __align__(16) float tile[kHeads][16 * kPass];
  __shared__ int page_s[16 * kPass], odd_s;  // odd_s: a score is NaN
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x / S, share = blockIdx.x - t * S;
  const int h0 = blockIdx.z * kHeads, nh = min(kHeads, p.pv.H_kv - h0), G = p.pv.H / p.pv.H_kv;
  if (tid == 0) odd_s = 0;
  // The queries' loads do not wait for the token's position.  A thread sums a
  // chunk over every parts-th query; `tile` joins the parts.
  const int sums = nh * kChunks;
  int parts = 1;
  while (parts * 2 * sums <= kThreads && parts * 2 * kSumLoads <= G) parts *= 2;
  const int part = tid / sums, h = (tid - part * sums) / kChunks, ch = tid % kChunks;
  float q[8];
  if (part < parts) sum_queries<kDim, kSumLoads>(p, t, h0 + h, G, ch, part, parts, q);
  if (parts > 1) {
    float4 *joint = reinterpret_cast<float4 *>(&tile[0][0]);  // [parts][sums][2]
    if (part > 0 && part < parts) {
      joint[2 * tid] = make_float4(q[0], q[1], q[2], q[3]);
      joint[2 * tid + 1] = make_float4(q[4], q[5], q[6], q[7]);
    }
    __syncthreads();
    for (int i = 1; part == 0 && i < parts; ++i) {
      const float4 u = joint[2 * (tid + i * sums)], w = joint[2 * (tid + i * sums) + 1];
      q[0] += u.x, q[1] += u.y, q[2] += u.z, q[3] += u.w;
      q[4] += w.x, q[5] += w.y, q[6] += w.z, q[7] += w.w;
    }
  }
  if (part == 0) {
#pragma unroll
    for (int piece = 0; piece < 3; ++piece) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = pack_bf16x2(q[2 * i], q[2 * i + 1]);
        q[2 * i] -= __uint_as_float(w[i] << 16);
        q[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
      }
      *reinterpret_cast<uint4 *>(&qs[h][piece][8 * ch]) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  int b, pos;
  const bool ok = load_paged_token(p.pv, t, p.status, tid == 0 && share == 0 && blockIdx.z == 0, b, pos);
  if (p.row_seq && share == 0 && tid < nh)
    write_row_token(p, static_cast<int64_t>(t) * p.pv.H_kv + h0 + tid, ok, b, pos);
  if (!ok) return;
  const int vis = (pos + 1) >> p.pv.logP, n = (vis + 15) >> 4;
  const int last = static_cast<int>(static_cast<int64_t>(n) * (share + 1) / S);
  const int begin = static_cast<int>(static_cast<int64_t>(n) * share / S);
  int a = begin;
  auto page_at = [&](int first) -> int {  // of this thread's page of the pass from tile `first`
    const int j = 16 * first + tid;
    return j < min(16 * min(first + kPass, last), vis) ? load_page(p.pv, b, j, p.status, blockIdx.z == 0) : -1;
  };
  int page = page_at(a);
  // the share of the columns past the pages the token sees
  {
    const int past = p.pv.max_pages - vis;
    const int c0 = vis + static_cast<int>(static_cast<int64_t>(past) * share / S);
    const int c1 = vis + static_cast<int>(static_cast<int64_t>(past) * (share + 1) / S);
    for (int h = warp; h < nh; h += kThreads / 32) {
      float *row = p.scores + (static_cast<int64_t>(t) * p.pv.H_kv + h0 + h) * p.ld;
      for (int j = c0 + lane; j < c1; j += 32) row[j] = -INFINITY;
    }
  }
  const int g = lane >> 2, ti = lane & 3;
  for (; a < last; a += kPass) {
    const int e = min(a + kPass, last), j0 = 16 * a, nj = min(16 * e, vis) - j0;
    page_s[tid] = page;
    __syncthreads();
    page = page_at(e);  // the next pass's, meanwhile
    const int items = (e - a) * nh;
    for (int it = warp; it < items; it += kThreads / 32) {
      const int jt = it / nh, h = it - jt * nh;
      uint4 v[2][kLoads];
      bool bad[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int id = page_s[16 * jt + g + 8 * r];  // -1 past the pages as well
        bad[r] = id < 0;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.k_mean + (static_cast<int64_t>(max(id, 0)) * p.pv.H_kv + h0 + h) * kDim);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) v[r][i] = bad[r] ? make_uint4(0, 0, 0, 0) : src[ti + 4 * i];
      }
      float d[4] = {};
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (g < 3) y = *reinterpret_cast<const uint4 *>(&qs[h][g][8 * (ti + 4 * i)]);
        mma_16816(d, v[0][i].x, v[1][i].x, v[0][i].y, v[1][i].y, y.x, y.y);
        mma_16816(d, v[0][i].z, v[1][i].z, v[0][i].w, v[1][i].w, y.z, y.w);
      }
      // columns 0 and 1 sit in lane 4 g, column 2 in lane 4 g + 1
      const float e0 = __shfl_down_sync(0xffffffffu, d[0], 1), e1 = __shfl_down_sync(0xffffffffu, d[2], 1);
      if (ti == 0) {
        const float s0 = (d[0] + (d[1] + e0)) * p.scale, s1 = (d[2] + (d[3] + e1)) * p.scale;
        tile[h][16 * jt + g] = bad[0] ? -INFINITY : s0;
        tile[h][16 * jt + g + 8] = bad[1] ? -INFINITY : s1;
        if (s0 != s0 || s1 != s1) odd_s = 1;
      }
    }
    __syncthreads();
    for (int h = warp; h < nh; h += kThreads / 32) {
      float *row = p.scores + (static_cast<int64_t>(t) * p.pv.H_kv + h0 + h) * p.ld + j0;
      for (int j = lane; j < nj; j += 32) row[j] = tile[h][j];
    }
    __syncthreads();  // the next pass writes tile
  }
  if (!odd_s) return;
  // NaN among the scores: an infinity in a sum or mean, perhaps, whose score is
  // the upper piece's product
  for (int h = warp; h < nh; h += kThreads / 32) {
    float *row = p.scores + (static_cast<int64_t>(t) * p.pv.H_kv + h0 + h) * p.ld;
    // (the columns of the passes above, by the same threads)
    for (int j = 16 * begin + lane; j < min(16 * last, vis); j += 32) {
      if (row[j] == row[j]) continue;
      const int id = load_page(p.pv, b, j, nullptr, false);
      const uint16_t *k = p.k_mean + (static_cast<int64_t>(max(id, 0)) * p.pv.H_kv + h0 + h) * kDim;
      row[j] = p.scale * upper_product<kDim>(qs[h][0], 0, k);
    }
  }
}

// ------------------------------------------------------ 128 tokens at a time

constexpr int kTile = 128;  // tokens, and pages, of a product
constexpr int kTileThreads = 512;  // and one warp that issues the products
constexpr int kPieces = 3;  // bf16 pieces of a summed query

template <int kDim>
struct ScoreSmem {
  static constexpr uint32_t kBlock = kTile * 128;          // one 64-dim block of 128 rows
  static constexpr uint32_t kRows = kBlock * (kDim / 64);
  static constexpr size_t q = 0;                           // [piece][D / 64][128 tokens][128 B]
  static constexpr size_t k = kPieces * kRows;             // [2][D / 64][128 pages][128 B]
  static constexpr size_t stage = k + 2 * kRows;           // [16 warps][32][16] f32
  static constexpr size_t pages = stage + 16 * 2048;           // [2][128] page ids of a block
  static constexpr size_t tok = pages + 2 * kTile * 4;     // [128] int2: sequence (-1: skip), visible pages
  static constexpr size_t bars = tok + kTile * 8;
  static constexpr size_t misc = bars + 2 * 8;
  static constexpr size_t total = misc + 32;
  static_assert(total + 1024 <= 232448, "shared memory budget");
};

template <int kDim>
__device__ __noinline__ float upper_product_of_tile(const uint8_t *qs, int row, const uint16_t *k) {
  return upper_product<kDim, ScoreSmem<kDim>::kBlock>(qs, row, k);
}

// CTA (x, h): tokens 128 x .. 128 x + 127, KV head h, every page.  Per
// sequence among the tokens: blocks of 128 pages, two in flight, the next
// block's product running and the one after being gathered while the current
// one's scores are written.
template <int kDim>
__global__ void __launch_bounds__(kTileThreads + 32, 1)
score_tile_kernel(const ScoreParams p) {
  using L = ScoreSmem<kDim>;
  constexpr int kChunks = kDim / 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *qs = smem + L::q, *ks = smem + L::k;
  int *page_s = reinterpret_cast<int *>(smem + L::pages);
  int2 *tok_s = reinterpret_cast<int2 *>(smem + L::tok);
  uint64_t *ready = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + L::misc);
  int *seq_s = reinterpret_cast<int *>(smem + L::misc + 8);  // sequence and page bound of the pass
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * kTile, nt = min(kTile, p.pv.T - t0), h = blockIdx.y, G = p.pv.H / p.pv.H_kv;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&ready[i], 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_base_s, 256);
    tmem_relinquish();
  }
  if (tid < kTile) {
    int b = -1, pos = -1;
    bool ok = false;
    if (tid < nt) {
      ok = load_paged_token(p.pv, t0 + tid, p.status, h == 0, b, pos);
      if (p.row_seq) write_row_token(p, static_cast<int64_t>(t0 + tid) * p.pv.H_kv + h, ok, b, pos);
    }
    tok_s[tid] = make_int2(ok ? b : -1, ok ? (pos + 1) >> p.pv.logP : 0);
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const bool worker = warp < kTileThreads / 32;    // not the issuer, which only joins the barriers
  const int row = 32 * (warp & 3) + lane;          // this thread's token
  const int2 mine = tok_s[row];
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const int64_t row_step = static_cast<int64_t>(p.pv.H_kv) * p.ld;  // scores of a token
  float *rows = p.scores + (t0 + 32 * (warp & 3)) * row_step + h * p.ld;
  float4 *stage = reinterpret_cast<float4 *>(smem + L::stage + warp * 2048);
  const bool vec = (p.ld & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scores) & 15) == 0;
  const int nblk = (p.pv.max_pages + kTile - 1) / kTile;
  int n = 0;  // blocks issued so far (of all passes)
  // the summed queries, split into bf16 pieces (round to nearest: each piece
  // takes at least 8 bits of what is left), while the first mean keys come in
  auto sum_all = [&]() {
    for (int i = worker ? tid : kTile * kChunks; i < kTile * kChunks; i += kTileThreads) {
      const int r = i / kChunks, ch = i % kChunks;
      float a[8] = {};
      if (r < nt) sum_queries<kDim, 16>(p, t0 + r, h, G, ch, 0, 1, a);
      const uint32_t off = (ch >> 3) * L::kBlock + sw128_offset(r, 16u * (ch & 7));
#pragma unroll
      for (int piece = 0; piece < kPieces; ++piece) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = pack_bf16x2(a[2 * e], a[2 * e + 1]);
          a[2 * e] -= __uint_as_float(w[e] << 16);
          a[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint4 *>(qs + piece * L::kRows + off) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    fence_proxy_async();
    __syncthreads();
  };
  bool summed = false;
  int prev = -1;  // sequences are taken in rising order
  while (true) {
    if (warp == 0) {
      // the next sequence among the tokens and the most pages any of them sees
      int next = INT32_MAX;
      for (int i = lane; i < kTile; i += 32) {
        const int b = tok_s[i].x;
        if (b > prev) next = min(next, b);
      }
      next = __reduce_min_sync(0xffffffffu, next);
      int most = 0;
      for (int i = lane; i < kTile; i += 32)
        if (tok_s[i].x == next) most = max(most, tok_s[i].y);
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) {
        seq_s[0] = next;
        seq_s[1] = most;
      }
    }
    __syncthreads();
    const int b = seq_s[0], seen = seq_s[1], used = (seen + kTile - 1) / kTile;
    if (b == INT32_MAX) break;
    __syncthreads();  // everyone has read the pass before the next one is written
    prev = b;
    // block i of the pass (block n + i of all) into buffer (n + i) & 1; pages
    // that do not exist or lie past the tokens' sight read row 0 and are masked
    // when written
    // Row r of the block is copied by threads 4 r .. 4 r + 3, 16 bytes at a
    // time into the swizzle (gathered TMA loads take 70 ns each to issue).
    // The page ids are looked up a block ahead.
    auto look_up = [&](int i) -> int {
      const int j = i * kTile + (tid >> 2);
      return worker && j < seen ? load_page(p.pv, b, j, p.status, h == 0) : -1;
    };
    int page_ahead = look_up(0);
    auto gather = [&](int i) {
      if (!worker) return;
      const int bf = (n + i) & 1, r = tid >> 2, page = page_ahead;
      page_ahead = look_up(i + 1);
      if ((tid & 3) == 0) page_s[bf * kTile + r] = page;
      const uint16_t *src = p.k_mean + (static_cast<int64_t>(max(page, 0)) * p.pv.H_kv + h) * kDim;
#pragma unroll
      for (int e = 0; e < kChunks / 4; ++e) {
        const int ch = (tid & 3) + 4 * e;
        cp_async16_plain(ks + bf * L::kRows + (ch >> 3) * L::kBlock + sw128_offset(r, 16u * (ch & 7)), src + 8 * ch);
      }
    };
    // The copies of every thread have landed and are visible to the tensor core.
    auto landed = [&]() {
      cp_async_wait_all();
      fence_proxy_async();
      __syncthreads();
    };
    auto multiply = [&](int i) {
      const int bf = (n + i) & 1;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t db = desc_sw128_kmajor(smem_u32(ks + bf * L::kRows));
#pragma unroll
        for (int piece = 0; piece < kPieces; ++piece) {
          const uint64_t da = desc_sw128_kmajor(smem_u32(qs + piece * L::kRows));
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint64_t o = ((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4;
            mma_f16(tmem + kTile * bf, da + o, db + o, idesc_bf16(128, kTile), piece + kk > 0);
          }
        }
        mma_commit(&ready[bf]);
      }
      __syncwarp();
    };
    if (used > 0) gather(0);
    if (!summed) {
      sum_all();
      summed = true;
    }
    if (used > 0) {
      landed();
      if (!worker) multiply(0);
      if (used > 1) gather(1);
    }
    const uint32_t ours = __ballot_sync(0xffffffffu, mine.x == b);  // rows of the warp's tokens
    for (int i = 0; i < nblk; ++i) {
      const int u = n + i, bf = u & 1;
      const bool live = i < used;
      float v[32];
      const int c0 = 32 * (warp >> 2), j0 = i * kTile + c0;
      if (!worker) {
        if (live) {
          landed();
          if (i + 1 < used) multiply(i + 1);
        }
        continue;
      }
      if (live) {
        if (!mbar_wait_warp(&ready[bf], (u >> 1) & 1) && lane == 0) raise_flag(p.status, kFlagTimeout);
        tc_fence_after();
        tmem_load(tmem + lanes + kTile * bf + c0, reinterpret_cast<uint32_t(&)[32]>(v));
        tmem_ld_wait();
        tc_fence_before();
        const int pg = page_s[bf * kTile + c0 + lane];
        // columns that exist and that this row's token sees
        const int sees = mine.y - j0;
        const uint32_t cols = __ballot_sync(0xffffffffu, pg >= 0) &
                              (sees >= 32 ? 0xffffffffu : sees > 0 ? (1u << sees) - 1 : 0u);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= p.scale;
        if (cols != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((cols >> e) & 1u)) v[e] = -INFINITY;
        }
        // NaN: an infinity among the sums or means, perhaps (the three pieces'
        // products share the accumulator)
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 32; ++e) odd |= v[e] != v[e];
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int id = __shfl_sync(0xffffffffu, pg, e);
            if (v[e] != v[e])  // (a masked column is -inf here: the page exists)
              v[e] = p.scale * upper_product_of_tile<kDim>(
                                   qs, row, p.k_mean + (static_cast<int64_t>(id) * p.pv.H_kv + h) * kDim);
          }
        }
        landed();  // block i + 1 is in; buffer bf (keys, page ids, accumulator) is free
        if (i + 2 < used) gather(i + 2);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = -INFINITY;
      }
      // 32 rows x 32 columns of the warp, transposed through shared memory 16
      // columns at a time so that a store covers 64 contiguous bytes of each of
      // eight rows, or, where rows are not 16-byte aligned or end, of each of two
      const bool whole = vec && j0 + 32 <= p.pv.max_pages;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          stage[4 * lane + (e ^ ((lane >> 1) & 3))] =
              make_float4(v[16 * half + 4 * e], v[16 * half + 4 * e + 1], v[16 * half + 4 * e + 2],
                          v[16 * half + 4 * e + 3]);
        __syncwarp();
        const int j = j0 + 16 * half;
        if (whole) {
          float *dst = rows + (lane >> 2) * row_step + j + 4 * (lane & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e, dst += 8 * row_step) {
            const int r = 8 * e + (lane >> 2);
            const float4 x = stage[4 * r + ((lane & 3) ^ ((r >> 1) & 3))];
            if ((ours >> r) & 1u) *reinterpret_cast<float4 *>(dst) = x;
          }
        } else {
          const int col = lane & 15;
          float *dst = rows + (lane >> 4) * row_step + j + col;
          const uint32_t write = j + col < p.pv.max_pages ? ours >> (lane >> 4) : 0u;
#pragma unroll 4
          for (int e = 0; e < 16; ++e, dst += 2 * row_step) {
            const int r = 2 * e + (lane >> 4);
            const float x = reinterpret_cast<const float *>(stage + 4 * r + ((col >> 2) ^ ((r >> 1) & 3)))[col & 3];
            if ((write >> (2 * e)) & 1u) *dst = x;
          }
        }
      }
      __syncwarp();
    }
    n += used;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int kDim>
cudaError_t launch_tile(const sa_paged_args &pa, const ScoreParams &p, cudaStream_t stream) {
  auto kern = score_tile_kernel<kDim>;
  const size_t smem = ScoreSmem<kDim>::total + 1024;
  static bool attr_done[64] = {};
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3((pa.T + kTile - 1) / kTile, pa.H_kv), dim3(kTileThreads + 32), smem, stream, 1, p);
}

}  // namespace

cudaError_t launch_page_scores(const sa_paged_args &pa, const void *q, const void *k_mean, float *scores, int64_t ld,
                               int local, int32_t *row_seq, int32_t *row_pos, uint32_t *status, cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  const ScoreParams p{paged_view(pa),
                      static_cast<const uint16_t *>(q),
                      static_cast<const uint16_t *>(k_mean),
                      scores,
                      ld,
                      pa.scale,
                      local,
                      row_seq,
                      row_pos,
                      status};
  // The kernel whose time is the lower by the measured costs (us): of the token
  // kernel a CTA per token and 8 heads and an item per 16 pages and head; of the
  // tile kernel, per wave of CTAs, a start, the queries' sum and the blocks of 128
  // pages, once for every sequence among a tile's tokens.  Measured (tile, token):
  // 4096 tokens, 4 KV heads, 512 pages 35 and 195; 1300 tokens, 8 heads, 1121
  // pages 48 and 239; 300, 8 heads, 958 pages 31 and 49; 2048, 2 heads, 147 pages
  // 14 and 25; 1300, 1 head of 64 queries, 1121 pages 61 and 50; 600, 4 heads, 44
  // pages 14 and 12; 475 tokens of two sequences, 14 pages 27 and 8.
  const int groups = (pa.H_kv + kHeads - 1) / kHeads;
  const double T = pa.T, items = T * pa.H_kv * ((pa.max_pages + 15) / 16);
  const double token_us = 5.5 + 0.0065 * T * groups + 0.33e-3 * items;
  const int64_t tiles = (static_cast<int64_t>(pa.T) + kTile - 1) / kTile * pa.H_kv;
  const double blocks = (pa.max_pages + kTile - 1) / kTile * (1.0 + (pa.B - 1.0) * kTile / T);
  const double tile_us = static_cast<double>((tiles + sm_count() - 1) / sm_count()) *
                         (9.0 + 0.5 * (pa.H / pa.H_kv) + 3.0 * blocks);
  if (tile_us < token_us)
    return pa.D == 128 ? launch_tile<128>(pa, p, stream) : launch_tile<64>(pa, p, stream);
  // shares of a token: three CTAs per SM over all (four run at once; shares for all
  // four measured 28 us against 25 on a decode batch of 64), no
  // more than it has tiles
  const int64_t target = std::max<int64_t>(1, 3LL * sm_count() / (static_cast<int64_t>(pa.T) * groups));
  const int S = static_cast<int>(std::min<int64_t>(target, (pa.max_pages + 15) / 16));
  const dim3 grid(static_cast<unsigned>(pa.T) * S, 1, groups);
  return pa.D == 128 ? launch_ex(false, score_token_kernel<128>, grid, dim3(kThreads), 0, stream, 1, p, S)
                     : launch_ex(false, score_token_kernel<64>, grid, dim3(kThreads), 0, stream, 1, p, S);
}

}  // namespace sa
