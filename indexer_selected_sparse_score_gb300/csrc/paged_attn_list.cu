// Attention of single tokens over lists of pages, on the 5th-generation tensor
// cores: the selected and local pages of sa_block_attn, and the pages past the
// shared ones of sa_prefix_attn.
//
// A unit is one token's group of query heads over one KV head (64 heads at
// most): few rows against many keys.  So the products are taken transposed,
// the keys in the 128 lanes of the accumulator and the heads in its columns,
// and no row of the tensor core is spent on padding:
//   S^T = K Q^T     M = 128 keys, N = heads (16, 32 or 64), K = D
//   P^T             one thread per key, or two with half of the heads each: p =
//                   2^(c s - m_ref[h]), bf16, to shared memory with the heads
//                   contiguous (the MN-major B operand)
//   O^T += V^T P^T  M = D, N = heads, K = 128 keys
// The pages land by TMA in the 128-byte swizzle, which is K-major for the
// first product and MN-major for the second, so K and V are copied once and
// never rearranged.  The reference maximum m_ref is the first tile's and is
// raised only when a logit passes it by 2^8 (one vote per tile); sums of p stay
// in registers per key and head and are reduced once per unit.  Weights are
// rounded to bf16 for the second product (2^-8 of each at most, against an
// output that is itself rounded to bf16); logits, sums and O are fp32.
//
// Work: the tiles of all units (128 keys each) form one list, cut evenly into
// parts, at the units' ends where that costs a CTA little: one part for each CTA,
// one CTA per SM, two with up to 16 heads (a decode step reads each page once, so
// HBM is the bound and every SM must stream to the end); beside the product with
// the shared pages, whose CTAs leave their SMs at different times, four per SM
// that CTAs claim, shrinking towards the end.  A unit that falls into several
// CTAs leaves its parts (m_ref, sum, O) in scratch for a merge kernel.  (A
// cluster per unit that merges over distributed shared memory instead: 33.5 us
// against 31.0 for 64 tokens of 64 heads over 2112 keys, and 16.5 against 14.2
// for a single token.)  Entries that name no page are dropped before tiles are
// formed; positions past the token's own are masked, and the V rows they hold
// are zeroed in shared memory, since 0 x NaN would reach the sum.
//
// Warps: 0-3 or 0-7 softmax and output; the next two issue S^T and O^T; then one
// resolves the lists, copies K and publishes one record per tile; the last
// copies V.  Every wait is bounded; on expiry the kernel flags the status word,
// drains its copies and products and returns.
//
// Measured, heads of 128: 64 tokens of 64 heads over one KV head, 34 pages of 64
// each: 27 us, 2.7 TB/s of the 72 MB it must read, by two CTAs to a unit, so on
// 128 of the SMs (about 3 us to the first tile, 8.5 tiles of 64 KB, 1.25 us each at
// HBM's rate, and 5 us of merge with its launch: 19 us; the rest are waits that no
// measurement has placed).  966 tokens of 32 over 4 heads, 13
// pages of 128 each: 205 us; a page is copied once for every token that lists it,
// so 3.4 GB pass from L2 to the SMs at 16 TB/s (about 60 bytes a clock and SM),
// which bounds work cut by tokens as it is here (cut by pages it would move less).  One token of 16 over 2
// heads, 34 pages of 64: 12 us, two launches and their chains of loads.  Units
// of a tile or two cost about 2 us each and CTA, half of it the walk of the
// list, half the chain of a tile: 306 tokens of 64 over 8 heads at the start of
// a sequence 51 us.
#include <cudaTypedefs.h>

#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "paged_bounds.h"
#include "paged_list.h"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;      // keys per tile
// Tiles that a CTA saves by not crossing into another unit (64 tokens of 64 heads,
// 17 tiles each: 30.3 us cut evenly over 152 CTAs, 28.0 over two for each unit),
// and that a call saves without a merge (26 units of two tiles: 13.9 us in halves,
// 12.4 whole).
constexpr int kCross = 2, kMerge = 2;
constexpr int kFewBlocks = 640; // of a merge (four per SM are resident)
constexpr int kQueue = 40;      // page entries the loader holds: under a tile's and one batch of 32
// The reference a weight is taken against lies kHead above the maximum that
// set it (log2 units), and is raised once a logit passes that maximum by kLazy:
// unnormalised sums of weights up to 2^(kLazy - kHead) times any bf16 values
// stay finite, and weights down to 2^-106 of the largest are kept.
constexpr float kLazy = 8.f, kHead = 20.f;
enum : int { kFirst = 1, kLast = 2, kEnd = 4, kMasked = 8, kDirect = 16 };

struct Record {
  int flags;     // bits 0-7; the unit's heads from bit 8
  int row;       // first output row of the unit (t * H + head)
  int slot;      // part slot of the piece
  uint32_t cnt[2];  // byte g: keys present among keys 16 g .. 16 g + 15
  uint32_t y[8];    // cache row of each page slot (past the end: an empty slot)
};

template <int N, int kDim>
struct ListSmem {
  // One ring holds the K and V tiles, in the order K(0), K(1), V(0), K(2), V(1),
  // ..: a V tile is needed a softmax later than its K, and with three slots it
  // takes the very slot that its K leaves.  Up to 16 heads two CTAs share an SM,
  // half a ring each: a tile's chain of waits (logits, weights, product) is then
  // longer than its work, and the other CTA's tiles fill it.
  static constexpr int kCtas = N == 16 ? 2 : 1;
  // Softmax warps: a thread takes one key and all heads (up to 16) or half of
  // them; then the two issuers and the two loaders.
  static constexpr int kSoftmaxWarps = N == 16 ? 4 : 8;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kSlots = (kDim == 128 ? 6 : 12) / kCtas;
  // P^T: rows of 64 heads in the 128-byte swizzle, with up to 32 heads a second
  // buffer in the upper half of the rows; up to 16 heads both buffers in rows
  // of 32 in the 64-byte swizzle.
  static constexpr int kPBufs = N <= 32 ? 2 : 1;
  static constexpr uint32_t kPRow = N == 16 ? 64 : 128;
  static constexpr int kRecs = list_records(kSlots);       // tile records
  static constexpr uint32_t kBlock = kTile * 128;          // one 64-dim block of a tile
  static constexpr uint32_t kKv = kBlock * (kDim / 64);
  static constexpr size_t ring = 0;
  static constexpr size_t p = ring + kSlots * kKv;         // [128 keys][kPRow]
  static constexpr size_t q = p + kTile * kPRow;           // [D / 64][N][128 B]
  static constexpr size_t recs = q + N * kDim * 2;
  static constexpr size_t red = (recs + kRecs * sizeof(Record) + 15) & ~size_t(15);   // [4][N]
  static constexpr size_t fac = red;                       // [N], over the reduction's first row (see below)
  static constexpr size_t mref = red + 4 * N * 4;          // [N]
  static constexpr size_t queue = mref + N * 4;            // [kQueue] page entries waiting for a tile
  static constexpr size_t bars = (queue + kQueue * 4 + 7) & ~size_t(7);
  static constexpr int kBars = 2 * kSlots + 2 + 4 + 2 * kPBufs + 2 + kRecs + 2;
  static constexpr size_t misc = bars + kBars * 8;
  static constexpr size_t used = misc + 16;
  // O^T at dim 64 reads a second block past a V tile (lanes nobody reads)
  static constexpr size_t total = kDim == 128 || used > p + kBlock ? used : p + kBlock;
  static_assert(kCtas * (total + 1024) <= 233472, "shared memory budget");
  static_assert(red % 16 == 0 && mref % 16 == 0 && queue % 4 == 0 && bars % 8 == 0 && misc % 8 == 0, "alignment");
  static constexpr uint32_t kCols = N == 16 ? 64 : N == 32 ? 128 : 256;  // tensor memory: S^T twice, O^T
};

// Byte of a P^T buffer's row `key` at which head `h` of the buffer begins.
template <int N>
__device__ __forceinline__ uint32_t p_offset(int key, int buf, int h) {
  if (N > 16) return sw128_offset(key, 64u * buf + 2u * h);
  const uint32_t b = 32u * buf + 2u * h;
  return static_cast<uint32_t>(key) * 64u + ((((b >> 4) ^ (static_cast<uint32_t>(key) >> 1)) & 3u) << 4) + (b & 15u);
}

// Barrier of the softmax warps.
template <int kSoftmax>
__device__ __forceinline__ void group_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
}

template <int N, int kDim>
__global__ void __launch_bounds__(ListSmem<N, kDim>::kThreads, ListSmem<N, kDim>::kCtas)
page_list_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const ListParams p) {
  using L = ListSmem<N, kDim>;
  constexpr int kSl = L::kSlots, kB = kDim / 64, kPb = L::kPBufs, kRecs = L::kRecs;
  constexpr uint32_t kColO = 2 * N;
  constexpr int kSoftmax = 32 * L::kSoftmaxWarps, kThreads = L::kThreads;
  constexpr int kWarpS = L::kSoftmaxWarps, kWarpO = kWarpS + 1, kWarpK = kWarpS + 2, kWarpV = kWarpS + 3;
  extern __shared__ __align__(1024) uint8_t smem[];  // (its alignment is checked below)
  uint8_t *ring = smem + L::ring, *ps = smem + L::p, *qs = smem + L::q;
  Record *recs = reinterpret_cast<Record *>(smem + L::recs);
  float *red_s = reinterpret_cast<float *>(smem + L::red);
  float *mref_s = reinterpret_cast<float *>(smem + L::mref);
  // fac[h] overwrites red[0][h], which only the thread that writes it has read;
  // a vote or a barrier of the softmax warps lies between a read of fac and the
  // next write of red
  float *fac_s = reinterpret_cast<float *>(smem + L::fac);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *full = bars, *empty = full + kSl;  // per ring slot
  uint64_t *qfull = empty + kSl, *qempty = qfull + 1, *sfull = qempty + 1, *sempty = sfull + 2;
  uint64_t *pfull = sempty + 2, *pempty = pfull + kPb, *ofull = pempty + kPb, *oempty = ofull + 1;
  uint64_t *rfull = oempty + 1, *done = rfull + kRecs;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  volatile int *issued_s = reinterpret_cast<volatile int *>(smem + L::misc + 8);  // tiles whose K and whose V were copied

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
    if (tid == 0) raise_flag(p.status, kFlagTimeout);
    return;
  }
  pdl_trigger();
  if (p.counter) {
    // a CTA that starts when every part has been claimed leaves at once (not
    // CTA 0, which reports the tokens it skips)
    const bool late = tid == 0 && blockIdx.x > 0 &&
                      *static_cast<volatile uint32_t *>(p.counter) >= static_cast<uint32_t>(p.parts);
    if (__syncthreads_or(late)) return;
  }
  // parts are claimed by the loader of K, the first while the block sets up
  int claim = 0;
  if (p.counter && warp == kWarpK && lane == 0) claim = static_cast<int>(atomicAdd(p.counter, 1u));
  if (tid == 0) {
    for (int i = 0; i < kSl; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], kSoftmax / 32);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < kPb; ++i) {
      mbar_init(&pfull[i], kSoftmax / 32);
      mbar_init(&pempty[i], 1);
    }
    mbar_init(ofull, 1);
    mbar_init(oempty, kSoftmax / 32);
    for (int i = 0; i < kRecs; ++i) mbar_init(&rfull[i], 1);
    *abort_s = 0;
    issued_s[0] = issued_s[1] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_base_s, L::kCols);
    tmem_relinquish();
  }
  // tiles of token t's units in whole-sequence mode (0 for a token to skip)
  const int spt = kTile >> p.pv.logP;  // pages per tile
  const int upt = p.pv.H_kv * p.gb;    // units per token
  auto count_of = [&](int t, bool report) -> int {
    int b, pos;
    if (!load_paged_token(p.pv, t, p.status, report, b, pos)) return 0;
    const int n = (pos >> p.pv.logP) + 1 - p.first_page;
    if (n <= 0) {
      if (report) raise_flag(p.status, kFlagBadPos);
      return 0;
    }
    return (n + spt - 1) / spt;
  };
  long long tot = static_cast<long long>(p.pv.T) * upt * p.tpu;
  if (p.whole) {
    // sequence lengths are known to the device only: every CTA sums the tiles
    // of all tokens (shared memory of the ring as scratch)
    long long own = 0;
    for (int t = tid; t < p.pv.T; t += kThreads) own += count_of(t, blockIdx.x == 0);
    block_prefix(own, reinterpret_cast<long long *>(ring), tot);
    tot *= upt;
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  // parts the tiles are cut into: no more than there are tiles, so that every
  // part between a unit's first and last holds a piece of it
  const int G = static_cast<int>(min(static_cast<long long>(p.parts), max(tot, 1ll)));
  // Place of K(n) and V(n) in the ring's order, the slot of place m and the
  // parity of its phase there.
  auto place_k = [](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto place_v = [](int n) { return 2 * n + 2; };
  auto slot_of = [](int m) { return m % kSl; };
  auto phase_of = [](int m) { return static_cast<uint32_t>((m / kSl) & 1); };
  auto fail = [&]() {
    raise_flag(p.status, kFlagTimeout);
    *abort_s = 1;
  };

  if (warp == kWarpV) {
    // ------------------------------------------------------------ loader of V
    // follows the records
    const int slot = lane / kB, kb = lane % kB;  // this lane's copy: page slot, 64-dim block
    const uint32_t dst = kb * L::kBlock + slot * p.pv.P * 128;
    if (lane == 0) prefetch_tmap(&vmap);
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      ok = mbar_wait_warp(&rfull[n % kRecs], (n / kRecs) & 1);
      if (!ok) break;
      const Record &rec = recs[n % kRecs];
      if (rec.flags & kEnd) break;
      const uint32_t y = rec.y[min(slot, 7)];
      const int m = place_v(n), s = slot_of(m);
      ok = mbar_wait_warp(&empty[s], phase_of(m) ^ 1);
      if (!ok || *abort_s) break;
      if (lane == 0) mbar_expect_tx(&full[s], L::kKv);
      __syncwarp();
      if (slot < spt) tma_load_2d(ring + s * L::kKv + dst, &vmap, &full[s], 64 * kb, static_cast<int>(y));
      if (lane == 0) issued_s[1] = n + 1;
    }
    if (lane == 0 && !ok) fail();
    __syncwarp();
  } else if (warp == kWarpK) {
    // ---------------------------------------------- loader of K, Q; the lists
    int *queue = reinterpret_cast<int *>(smem + L::queue);
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&qmap);
    }
    int n = 0, qn = 0;
    bool ok = true;
    const uint32_t rows_total = static_cast<uint32_t>(p.pv.n_pages) * p.pv.H_kv * p.pv.P;
    const int slot = lane / kB, kb = lane % kB;
    const uint32_t dst = kb * L::kBlock + slot * p.pv.P * 128;
    int t = 0, sub = 0, cnt = p.tpu;  // token, unit of the token, tiles of the unit
    long long base = 0;               // tiles before the unit
    // whole sequences: moves on to the token that holds tile x (x is not before
    // the current token's), 32 tokens at a time
    auto seek = [&](long long x) {
      base -= static_cast<long long>(sub) * cnt;
      sub = 0;
      for (;;) {
        const int own = t + lane < p.pv.T ? count_of(t + lane, false) : 0;
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += up;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, x < base + static_cast<long long>(sum) * upt);
        const int at = m ? __ffs(m) - 1 : 31;
        const int incl = __shfl_sync(0xffffffffu, sum, at), mine = __shfl_sync(0xffffffffu, own, at);
        if (m) {
          t += at;
          base += static_cast<long long>(incl - mine) * upt;
          cnt = mine;
          return;
        }
        base += static_cast<long long>(incl) * upt;
        t += 32;
      }
    };
    // First tile of part c.  Claimed parts shrink towards the end, from twice the
    // mean to one tile, so that CTAs that start late share what is left.
    auto part_begin = [&](int c) -> long long {
      if (!p.counter) return tot * c / G;
      // c (2 G - c) / G^2 in steps of 2^-11, and a tile for every part
      static_assert(kMaxParts <= 1024, "32 bits");
      const uint32_t w = (static_cast<uint32_t>(c * (2 * G - c)) << 11) / static_cast<uint32_t>(G * G);
      return c + ((tot - G) * w >> 11);
    };
    int c = blockIdx.x;  // the part being worked on
    int b = 0, pos = 0, at = -1;  // sequence and position of token `at`
    bool tok = false;
    for (bool again = false; ok; again = true) {
      if (p.counter) {
        if (again && lane == 0) claim = static_cast<int>(atomicAdd(p.counter, 1u));
        c = __shfl_sync(0xffffffffu, claim, 0);
        if (c >= G) break;
      }
      const long long x_begin = part_begin(min(c, G)), x_end = part_begin(min(c + 1, G));
      int cut_unit = -1, cut_last = 0;
      long long x = x_begin;
      if (x < x_end) {
        if (p.whole) {
          seek(x);
          sub = static_cast<int>((x - base) / cnt);
          base += static_cast<long long>(sub) * cnt;
        } else {
          const long long u = x / p.tpu;
          t = static_cast<int>(u / upt);
          sub = static_cast<int>(u % upt);
          base = u * p.tpu;
        }
      }
      while (ok && x < x_end) {
        const int u = t * upt + sub;
        const int a = static_cast<int>(x - base);
        const int e = static_cast<int>(min(static_cast<long long>(cnt), x_end - base));
        const bool starts = a == 0, ends = e == cnt;
        const int hk = p.gb == 1 ? sub : sub / p.gb, nlist = p.whole ? 0 : p.K;
        // (the list's entries do not wait for the token's position)
        auto entry = [&](int i) -> int {
          return i < nlist ? p.idx[(static_cast<int64_t>(t) * p.pv.H_kv + hk) * p.K + i] : 0;
        };
        int entry_ahead = entry(a * spt + lane);
        if (t != at) tok = load_paged_token(p.pv, t, p.status, lane == 0 && sub == 0 && starts && !p.whole, b, pos);
        at = t;
        if (tok) {
          const int h0 = hk * p.group + (sub - hk * p.gb) * 64;
          const int last = pos >> p.pv.logP;
          const int own = pos + 1 - last * p.pv.P;  // positions of the token's own page that it sees
          const int f = p.whole ? p.first_page : max(last + 1 - p.local, 0);
          const int r1 = min(e * spt, nlist + last + 1 - f);
          int r = a * spt, qh = 0, qe = 0;  // raw entries, queue head and end
          if (p.keep) {
            if (lane == 0 && starts) p.info[u].x = c;
            if (lane == 0 && ends) p.info[u].y = c;
          } else if (starts && !ends) {
            // the part of tile y is floor(((y + 1) G - 1) / tot)
            cut_unit = u;
            cut_last = static_cast<int>(((base + cnt) * G - 1) / tot);
          }
          // page entry i of the list (page id, bit 30 set for the token's own
          // page, whose later positions are masked), -1 when it names no page
          auto resolve = [&](int i, int j) -> int {
            if (i >= r1) return -1;
            if (i < nlist) {
              if (j < 0 || j >= f) {
                if (j < -1 || j > last) raise_flag(p.status, kFlagBadIndex);
                return -1;
              }
            } else {
              j = f + i - nlist;
            }
            const int page = load_page(p.pv, b, j, p.status, true);
            return page < 0 ? -1 : page | (j == last ? 1 << 30 : 0);
          };
          bool first = true, more = true;
          int ahead = resolve(r + lane, entry_ahead);  // the next batch, resolved while earlier tiles are copied
          while (more) {
            while (qe - qh <= spt && r < r1) {  // enough for this tile and to know whether another follows
              const int rest = qe - qh, ent = ahead;
              r += 32;
              ahead = -1;
              if (r < r1) ahead = resolve(r + lane, entry(r + lane));
              const int keep = lane < rest ? queue[qh + lane] : 0;
              const uint32_t m = __ballot_sync(0xffffffffu, ent >= 0);
              __syncwarp();
              if (lane < rest) queue[lane] = keep;
              if (ent >= 0) queue[rest + __popc(m & ((1u << lane) - 1))] = ent;
              __syncwarp();
              qh = 0;
              qe = rest + __popc(m);
            }
            const int take = min(spt, qe - qh);
            more = qe - qh > take;
            const int ent = slot < take ? queue[qh + slot] : -1;
            const int m = place_k(n), s = slot_of(m);
            // keys present among each 16: lane g's own granule, its page slot
            // held by the lanes of that slot
            const int g = lane & 7, sg = (16 * g) >> p.pv.logP;
            const int eg = __shfl_sync(0xffffffffu, ent, sg * kB);
            int have = eg >= 0 ? 16 : 0;
            if (eg >= 0 && (eg >> 30)) have = min(max(own - (16 * g - (sg << p.pv.logP)), 0), 16);
            const bool masked = __any_sync(0xffffffffu, eg >= 0 && have < 16);
            const uint32_t byte = lane < 8 ? static_cast<uint32_t>(have) << (8 * (g & 3)) : 0u;
            const uint32_t cn0 = __reduce_or_sync(0xffffffffu, g < 4 ? byte : 0u);
            const uint32_t cn1 = __reduce_or_sync(0xffffffffu, g < 4 ? 0u : byte);
            // a slot without a page reads past the tensor's end: the copy fills zeros
            const uint32_t y = ent >= 0 ? ((static_cast<uint32_t>(ent) & 0x3FFFFFFFu) * p.pv.H_kv + hk) * p.pv.P
                                        : rows_total;
            // With an odd number of slots the phase before V(n - 3)'s in this
            // slot is K(n - 3)'s: the parity tells them apart once V(n - 3) has
            // been issued.
            bool mine = true;
            if ((kSl & 1) != 0 && n >= 3) {
              if (issued_s[1] < n - 2) {
                const long long since = clock64();
                while (mine && issued_s[1] < n - 2) mine = clock64() - since < kWaitBudgetCycles && !*abort_s;
              }
              mine = __all_sync(0xffffffffu, mine);
            }
            if (!mine || !mbar_wait_warp(&empty[s], phase_of(m) ^ 1) || *abort_s) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_expect_tx(&full[s], L::kKv);
            __syncwarp();
            if (slot < spt) tma_load_2d(ring + s * L::kKv + dst, &kmap, &full[s], 64 * kb, static_cast<int>(y));
            Record &rec = recs[n % kRecs];
            if (slot < 8 && kb == 0) rec.y[slot] = y;
            if (lane == 0) {
              rec.flags = (first ? kFirst : 0) | (more ? 0 : kLast) | (masked ? kMasked : 0) |
                          (!p.keep && starts && ends ? kDirect : 0) | min(64, (hk + 1) * p.group - h0) << 8;
              rec.row = t * p.pv.H + h0;
              rec.slot = p.keep ? u + c : 2 * c + (starts ? 1 : 0);
              rec.cnt[0] = cn0;
              rec.cnt[1] = cn1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rfull[n % kRecs]);
            ++n;
            if (first) {
              // the queries, once the previous unit's last product has read its own
              if (lane == 0) {
                ok = mbar_wait(qempty, (qn & 1) ^ 1);
                if (ok) {
                  mbar_expect_tx(qfull, N * kDim * 2);
                  for (int i = 0; i < kB; ++i)
                    tma_load_2d(qs + i * N * 128, &qmap, qfull, 64 * i, t * p.pv.H + h0);
                }
              }
              ok = __shfl_sync(0xffffffffu, ok, 0);
              if (!ok) break;
              ++qn;
            }
            qh += take;
            first = false;
          }
        }
        x = base + e;
        if (ends && x < x_end) {
          if (++sub < upt) {
            base += cnt;
          } else if (p.whole) {
            --sub;
            seek(x);
          } else {
            base += cnt;
            sub = 0;
            ++t;
          }
        }
      }
      if (!p.counter) {
        if (lane == 0) p.cut[c] = make_int2(cut_unit, cut_last);
        break;
      }
    }
    if (lane == 0) {
      if (ok) {
        recs[n % kRecs].flags = kEnd;
        mbar_arrive(&rfull[n % kRecs]);
      } else {
        fail();
      }
      issued_s[0] = n;
      if (qn > 0) mbar_wait(qfull, (qn - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpS) {
    // ---------------------------------------------------------- S^T = K Q^T
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16(128, N);
    bool ok = true;
    int qn = 0;
    for (int n = 0;; ++n) {
      ok = mbar_wait_warp(&rfull[n % kRecs], (n / kRecs) & 1);
      if (!ok) break;
      const int flags = recs[n % kRecs].flags;
      if (flags & kEnd) break;
      const int m = place_k(n), s = slot_of(m), bf = n & 1;
      if (flags & kFirst) ok = mbar_wait_warp(qfull, (qn++) & 1);
      ok = ok && mbar_wait_warp(&full[s], phase_of(m)) && mbar_wait_warp(&sempty[bf], ((n >> 1) & 1) ^ 1);
      if (!ok || *abort_s) break;
      tc_fence_after();
      if (leader) {
        const uint64_t da = desc_sw128_kmajor(smem_u32(ring + s * L::kKv)), db = desc_sw128_kmajor(smem_u32(qs));
#pragma unroll
        for (int kk = 0; kk < kDim / 16; ++kk) {
          const uint64_t ao = ((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4;
          const uint64_t bo = ((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4;
          mma_f16(tmem + N * bf, da + ao, db + bo, idesc, kk > 0);
        }
        mma_commit(&sfull[bf]);
        mma_commit(&empty[s]);
        if (flags & kLast) mma_commit(qempty);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) fail();
    if (leader) {
      mma_commit(&done[0]);
      if (!mbar_wait(&done[0], 0)) raise_flag(p.status, kFlagTimeout);
    }
    __syncwarp();
  } else if (warp == kWarpO) {
    // ------------------------------------------------------- O^T += V^T P^T
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16(128, N) | (1u << 15) | (1u << 16);  // MN-major A and B
    bool ok = true;
    int pieces = 0;
    for (int n = 0;; ++n) {
      ok = mbar_wait_warp(&rfull[n % kRecs], (n / kRecs) & 1);
      if (!ok) break;
      const int flags = recs[n % kRecs].flags;
      if (flags & kEnd) break;
      const int m = place_v(n), s = slot_of(m), pb = n % kPb;
      if (flags & kFirst) ok = mbar_wait_warp(oempty, (pieces++ & 1) ^ 1);
      // (the weights first: they say that K(n), perhaps the slot's phase before,
      // is done with)
      ok = ok && mbar_wait_warp(&pfull[pb], (n / kPb) & 1) && mbar_wait_warp(&full[s], phase_of(m));
      if (!ok || *abort_s) break;
      tc_fence_after();
      if (leader) {
        const uint64_t da = desc_mn(smem_u32(ring + s * L::kKv), L::kBlock);
        const uint64_t db = N == 16 ? desc_mn64(smem_u32(ps) + 32 * pb) : desc_mn(smem_u32(ps) + 64 * pb, 16384);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
          mma_f16(tmem + kColO, da + ((kk * 2048) >> 4), db + ((kk * 16 * L::kPRow) >> 4), idesc, !((flags & kFirst) && kk == 0));
        }
        mma_commit(&empty[s]);
        mma_commit(&pempty[pb]);
        if (flags & kLast) mma_commit(ofull);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) fail();
    if (leader) {
      mma_commit(&done[1]);
      if (!mbar_wait(&done[1], 0)) raise_flag(p.status, kFlagTimeout);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------------- softmax
    // Thread: one key of the tile (the accumulator lane) and NH of the heads.
    // The logits' arguments are formed once, tested against the reference, and
    // only then raised to weights.
    constexpr int NH = 4 * N / L::kSoftmaxWarps;
    const int quarter = warp & 3, key = tid & 127, hb = warp >= 4 ? NH : 0;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const float cs = p.qk_scale;
    const float2 cs2 = make_float2(cs, cs);
    float *red_w = red_s + N * quarter + hb;
    float l[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) l[h] = 0.f;
    int pieces = 0;
    for (int n = 0;; ++n) {
      bool ok = mbar_wait_warp(&rfull[n % kRecs], (n / kRecs) & 1);
      Record rec{};
      if (ok) rec = recs[n % kRecs];
      const bool end = (rec.flags & kEnd) != 0;
      const int bf = n & 1, s = slot_of(place_v(n));
      const bool first = (rec.flags & kFirst) != 0;
      const uint32_t word = key < 64 ? rec.cnt[0] : rec.cnt[1];
      const bool present = static_cast<uint32_t>(key & 15) < ((word >> (8 * ((key >> 4) & 3))) & 0xFFu);
      ok = ok && (end || mbar_wait_warp(&sfull[bf], (n >> 1) & 1));
      float v[NH];  // logits, then c s - m_ref
      bool over = first;
      if (ok && !end) {
        tc_fence_after();
        tmem_load(tmem + lanes + N * bf + hb, reinterpret_cast<uint32_t(&)[NH]>(v));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[bf]);
        if (!first) {
          float top = -INFINITY;
#pragma unroll
          for (int h = 0; h < NH; h += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(mref_s + hb + h);
            float2 *w = reinterpret_cast<float2 *>(v + h);
            w[0] = fma2(w[0], cs2, make_float2(-m.x, -m.y));
            w[1] = fma2(w[1], cs2, make_float2(-m.z, -m.w));
            top = max3(max3(top, w[0].x, w[0].y), w[1].x, w[1].y);
          }
          over = present && top > kLazy - kHead;
        }
      }
      if (!ok && lane == 0) fail();
      // one vote per tile; only when it passes, a second one tells a raise of
      // the reference from the end or a failure (all warps leave together)
      const bool leave = !ok || end || *abort_s;
      if (barrier_any(2, kSoftmax, over || leave)) {
        if (barrier_any(3, kSoftmax, leave)) break;
        // the tile's maximum per head, over the keys that exist (for a tile
        // after the first: of c s - m_ref)
        float x[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) x[h] = present ? (first ? v[h] * cs : v[h]) : -INFINITY;
        const float top = reduce_scatter<true>(x, lane);
        if (lane < NH) red_w[lane] = top;
        group_sync<kSoftmax>();
        if (tid < N) {
          const float mo = first ? 0.f : mref_s[tid];
          const float mt = fmaxf(fmaxf(red_s[tid], red_s[N + tid]), fmaxf(red_s[2 * N + tid], red_s[3 * N + tid]));
          // the new reference relative to the old one, which only rises
          const float up = first ? mt + kHead : fmaxf(mt + kHead, 0.f);
          fac_s[tid] = up;
          mref_s[tid] = mo + up;
        }
        group_sync<kSoftmax>();
#pragma unroll
        for (int h = 0; h < NH; ++h) v[h] = (first ? v[h] * cs : v[h]) - fac_s[hb + h];
        if (!first) {
          // O^T holds the products up to tile n - 1; scale its columns
          const bool done_o = mbar_wait_warp(&pempty[(n - 1) % kPb], ((n - 1) / kPb) & 1);
          if (!done_o && lane == 0) fail();
          tc_fence_after();
          if (done_o && quarter < kDim / 32) {
#pragma unroll 1
            for (int i = 0; i < NH; i += 8) {
              uint32_t o[8];
              tmem_load(tmem + lanes + kColO + hb + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                o[q] = __float_as_uint(__uint_as_float(o[q]) * exp2f(-fac_s[hb + i + q]));
              tmem_store8(tmem + lanes + kColO + hb + i, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
#pragma unroll
          for (int h = 0; h < NH; ++h) l[h] *= exp2f(-fac_s[hb + h]);
        }
      }
      // P^T buffer free: the product that read it last is done
      const int pb = n % kPb;
      if (!mbar_wait_warp(&pempty[pb], ((n / kPb) & 1) ^ 1) && lane == 0) fail();
      if (!__all_sync(0xffffffffu, present)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) v[h] = present ? v[h] : -INFINITY;
      }
#pragma unroll
      for (int ch = 0; ch < NH / 8; ++ch) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int h = 8 * ch + 2 * q;
          const float2 e2 = make_float2(exp2_hw(v[h]), exp2_hw(v[h + 1]));
          float2 *l2 = reinterpret_cast<float2 *>(l + h);
          *l2 = add2(*l2, e2);
          w[q] = pack_bf16x2(e2.x, e2.y);
        }
        *reinterpret_cast<uint4 *>(ps + p_offset<N>(key, pb, hb + 8 * ch)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (rec.flags & kMasked) {
        // positions past the token's own may hold anything: their V rows
        // become zeros before the product reads them (each thread its
        // share of the row)
        if (!mbar_wait_warp(&full[s], phase_of(place_v(n))) && lane == 0) fail();
        if (!present) {
          // the row in 16-byte chunks, shared by the threads that hold its key, each
          // lane in an order of its own (rows are 128 bytes apart: the same chunk
          // of all of them lies in the same banks)
          constexpr int kChunks = kDim / 8 * NH / N;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int ch = ((hb ? kChunks : 0) + i) ^ (key & 7);
            *reinterpret_cast<uint4 *>(ring + s * L::kKv + (ch >> 3) * L::kBlock + key * 128 + 16 * (ch & 7)) =
                make_uint4(0, 0, 0, 0);
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[pb]);
      if (rec.flags & kLast) {
        // sums over the keys while the last product runs (the barrier: a raise
        // in this tile still reads fac, which lies over the reduction's rows)
        const float sum_w = reduce_scatter<false>(l, lane);
        group_sync<kSoftmax>();
        if (lane < NH) red_w[lane] = sum_w;
#pragma unroll
        for (int h = 0; h < NH; ++h) l[h] = 0.f;
        group_sync<kSoftmax>();
        if (tid < N) {
          const float sum = (red_s[tid] + red_s[N + tid]) + (red_s[2 * N + tid] + red_s[3 * N + tid]);
          fac_s[tid] = sum > 0.f ? 1.f / sum : 0.f;
          if (!(rec.flags & kDirect))
            p.ml[static_cast<int64_t>(rec.slot) * N + tid] = make_float2(mref_s[tid], sum);
        }
        group_sync<kSoftmax>();
        if (!mbar_wait_warp(ofull, pieces & 1) && lane == 0) fail();
        ++pieces;
        tc_fence_after();
        if (quarter < kDim / 32) {
          const int d = 32 * quarter + lane, heads = (rec.flags >> 8) - hb;
          __nv_bfloat16 *out = p.out + (static_cast<int64_t>(rec.row) + hb) * kDim + d;
          float *part = p.part + (static_cast<int64_t>(rec.slot) * N + hb) * kDim + d;
#pragma unroll 1
          for (int i = 0; i < NH && i < heads; i += 8) {
            uint32_t o[8];
            tmem_load(tmem + lanes + kColO + hb + i, o);
            tmem_ld_wait();
            if (rec.flags & kDirect) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (i + q < heads)
                  out[(i + q) * kDim] = __float2bfloat16_rn(__uint_as_float(o[q]) * fac_s[hb + i + q]);
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (i + q < heads) part[(i + q) * kDim] = __uint_as_float(o[q]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty);
      }
    }
  }
  // The merge of kept parts also needs the kernel before this one: a CTA that
  // completes after it makes the chain transitive (one, so that the others leave
  // their SMs to the merge).
  if (p.keep && blockIdx.x == 0) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (*abort_s && tid < kSl) {
    // A wait gave up, so a copy may be on its way (else its product has waited
    // for each): the last one issued into slot tid lands before the CTA exits.
    auto issued = [&](int m) {
      return m == 0 ? issued_s[0] > 0 : (m & 1) ? (m + 1) / 2 < issued_s[0] : (m - 2) / 2 < issued_s[1];
    };
    int m = 2 * max(issued_s[0], issued_s[1]) + 2 + kSl;
    m -= (m - tid) % kSl;
    while (m >= 0 && !issued(m)) m -= kSl;
    if (m >= 0) mbar_wait(&full[tid], phase_of(m));
  }
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// Merges the parts of the unit that starts in CTA c's range and ends past it: o = sum 2^(m_i - M) o_i
// / sum 2^(m_i - M) l_i.  kSplit warps per head, each every kSplit-th part (8
// when a unit has many parts: the chain of loads is then what the merge costs).
template <int N, int kDim, int kSplit>
__global__ void __launch_bounds__(256)
merge_cut_kernel(const ListParams p) {
  __shared__ float acc_s[8][kDim + 2];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int upt = p.pv.H_kv * p.gb;
  __shared__ int2 cut_s;
  const bool known = !p.whole && gridDim.x * gridDim.y <= kFewBlocks;
  if (known) {
    // Which unit CTA c cut can be worked out while the kernel before runs: it
    // saves a load after the wait (one token over 34 pages 12.9 to 12.3 us, over
    // 20 pages of 16 12.4 to 11.6).  With many blocks the divisions take more of
    // that kernel's issue slots than the load costs (64 tokens 29.1 to 30.9):
    // those read what it wrote.
    if (threadIdx.x == 0) {
      const long long tot = static_cast<long long>(p.pv.T) * upt * p.tpu, G = min(static_cast<long long>(p.parts), tot);
      const long long x0 = tot * c / G, x1 = tot * (c + 1) / G, u = (x1 - 1) / p.tpu, end = (u + 1) * p.tpu;
      int b, pos;
      const bool is = u * p.tpu >= x0 && end > x1 &&
                      load_paged_token(p.pv, static_cast<int>(u / upt), nullptr, false, b, pos);
      cut_s = is ? make_int2(static_cast<int>(u), static_cast<int>((end * G - 1) / tot)) : make_int2(-1, 0);
    }
    __syncthreads();
  }
  pdl_wait();
  const int2 cut = known ? cut_s : p.cut[c];
  if (!cut_ok(cut.x, cut.y, static_cast<int64_t>(p.pv.T) * upt, c, p.parts)) return;  // (-1: none)
  const int t = cut.x / upt, sub = cut.x % upt;
  const int hk = sub / p.gb, h0 = hk * p.group + (sub % p.gb) * 64, heads = min(64, (hk + 1) * p.group - h0);
  const int i = blockIdx.y * (8 / kSplit) + warp / kSplit;
  if (i >= heads) return;  // (kSplit 8: the whole block)
  Merge<kDim> m;
  m.add(warp % kSplit, kSplit, cut.y - c + 1, lane, p.ml, p.part,
        [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)) * N + i; });
  if (m.template join<kSplit>(acc_s, lane)) m.store(p.out + (static_cast<int64_t>(t) * p.pv.H + h0 + i) * kDim, lane);
}

template <int N, int kDim>
cudaError_t launch_list(const sa_paged_args &pa, const void *q, ListParams &p, int grid, bool pdl,
                        cudaStream_t stream) {
  using L = ListSmem<N, kDim>;
  CUtensorMap qmap, kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(pa.n_pages) * pa.H_kv * pa.P;
  if (!encode_rows(&qmap, q, static_cast<uint64_t>(pa.T) * pa.H, kDim, N) ||
      !encode_rows(&kmap, pa.K, rows, kDim, pa.P) || !encode_rows(&vmap, pa.V, rows, kDim, pa.P))
    return cudaErrorInvalidValue;
  auto kern = page_list_kernel<N, kDim>;
  const size_t smem = L::total;
  static bool attr_done[64] = {};
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem, attr_done);
  if (e != cudaSuccess) return e;
  e = launch_ex(pdl, kern, dim3(grid), dim3(L::kThreads), smem, stream, 1, qmap, kmap, vmap, p);
  if (e != cudaSuccess || p.keep) return e;
  const int64_t units = static_cast<int64_t>(pa.T) * pa.H_kv * p.gb;
  if (!p.whole && units == grid) return cudaSuccess;  // every unit was one CTA's
  return units * 8 <= grid
             ? launch_ex(true, merge_cut_kernel<N, kDim, 8>, dim3(grid, N), dim3(256), 0, stream, 1, p)
             : launch_ex(true, merge_cut_kernel<N, kDim, 1>, dim3(grid, N / 8), dim3(256), 0, stream, 1, p);
}

template <int kDim>
cudaError_t launch_dim(const sa_paged_args &pa, const void *q, ListParams &p, int grid, bool pdl, cudaStream_t stream) {
  switch (list_cols(pa)) {
    case 16: return launch_list<16, kDim>(pa, q, p, grid, pdl, stream);
    case 32: return launch_list<32, kDim>(pa, q, p, grid, pdl, stream);
    default: return launch_list<64, kDim>(pa, q, p, grid, pdl, stream);
  }
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

bool encode_rows(CUtensorMap *m, const void *base, uint64_t rows, int dim, uint32_t box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dim), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(dim) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int list_cols(const sa_paged_args &pa) {
  const int g = pa.H / pa.H_kv;
  return g <= 16 ? 16 : g <= 32 ? 32 : 64;
}

// Most CTAs of a grid (two to an SM with up to 16 heads).
static int list_ctas(const sa_paged_args &pa) { return list_cols(pa) == 16 ? 512 : 256; }

size_t list_scratch(const sa_paged_args &pa, bool keep) {
  const int g = pa.H / pa.H_kv;
  const size_t units = static_cast<size_t>(pa.T) * pa.H_kv * ((g + 63) / 64);
  const size_t slots = keep ? units + kMaxParts : 2 * list_ctas(pa);
  return round_up(slots * list_cols(pa) * pa.D * sizeof(float)) + round_up(slots * list_cols(pa) * sizeof(float2)) +
         round_up((keep ? units : list_ctas(pa)) * sizeof(int2));
}

cudaError_t launch_page_list(const sa_paged_args &pa, const void *q, ListParams &p, void *out, void *scratch,
                             uint32_t *status, bool pdl, cudaStream_t stream) {
  p.pv = paged_view(pa);
  p.group = pa.H / pa.H_kv;
  p.gb = (p.group + 63) / 64;
  p.qk_scale = pa.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.status = status;
  const size_t units = static_cast<size_t>(pa.T) * pa.H_kv * p.gb;
  const size_t slots = p.keep ? units + kMaxParts : 2 * list_ctas(pa);
  char *w = static_cast<char *>(scratch);
  p.part = reinterpret_cast<float *>(w);
  w += round_up(slots * list_cols(pa) * pa.D * sizeof(float));
  p.ml = reinterpret_cast<float2 *>(w);
  w += round_up(slots * list_cols(pa) * sizeof(float2));
  p.info = p.cut = reinterpret_cast<int2 *>(w);
  int grid = std::min(sm_count() * (list_cols(pa) == 16 ? 2 : 1), list_ctas(pa));
  const int spt = kTile / pa.P;
  if (p.whole) {
    const int64_t tiles = (pa.max_pages - p.first_page + spt - 1) / spt;  // of a unit, at most
    grid = static_cast<int>(std::min<int64_t>(grid, std::max<int64_t>(1, static_cast<int64_t>(units) * tiles)));
  } else {
    const int64_t entries = static_cast<int64_t>(p.K) + std::min(p.local, pa.max_pages);
    p.tpu = static_cast<int>(std::max<int64_t>(1, (entries + spt - 1) / spt));
    const int64_t n = static_cast<int64_t>(units), even = (n * p.tpu + grid - 1) / grid;  // tiles of a CTA
    int64_t k = std::min<int64_t>(grid / n, p.tpu);  // whole CTAs of each unit
    if (k > 0 && p.tpu <= even + kMerge)
      k = 1;
    else if (k > 0 && (p.tpu + k - 1) / k > even + kCross)
      k = 0;
    grid = static_cast<int>(k > 0 ? n * k : std::min<int64_t>(grid, n * p.tpu));
  }
  p.parts = p.keep ? std::min(4 * sm_count(), kMaxParts) : grid;
  p.counter = p.keep ? status + kCounterWord : nullptr;
  return pa.D == 128 ? launch_dim<128>(pa, q, p, grid, pdl, stream) : launch_dim<64>(pa, q, p, grid, pdl, stream);
}

size_t block_attn_scratch(const sa_paged_args &pa, int, int) { return list_scratch(pa, false); }

cudaError_t launch_block_attn(const sa_paged_args &pa, const void *q, const int32_t *idx, int K, int local, void *out,
                              void *scratch, uint32_t *status, cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  ListParams p{};
  p.idx = idx;
  p.K = K;
  p.local = local;
  return launch_page_list(pa, q, p, out, scratch, status, false, stream);
}

}  // namespace sa
