// Attention of chunks of new tokens over a paged cache on the tensor cores:
// 16-bit or e4m3 cache, d = dv = 128, pages of a multiple of 16 positions.
//
// A block of query rows is up to 256 (token, head of the group) rows of one
// K/V head, tokens outer, so that a K/V tile serves every query head that reads
// it and a short chunk still fills the 128-row products. Two 128-row halves
// with a softmax warpgroup each alternate on the tensor core, as in the dense
// forward kernel: S = Q K^T into TMEM, one row per thread turned into P in
// place, O += P V into TMEM.
//
// K/V tiles of 128 keys come page by page: each lane of the producer warp
// looks up the page of one box of the tile and issues its copies (boxes past the
// sequence's end or in a page outside the pool take page 0, whose keys are
// masked). An e4m3 tile lands in a raw buffer, and four warps turn it into the
// 16-bit operand tiles: K's codes exactly (their scale multiplies the score
// in fp32), V's times their scales over a power of two per 32 keys, in fp16.
//
// A masked key's V row may hold anything, and 0 times an infinity is not 0.
// In tiles that some row sees only in part, or that hold such a box, the
// checker warps (e4m3: the converting ones) therefore take non-finite elements
// of V out of the operand; rows that do see such a key get them back in the
// epilogue, where the result is not finite whatever the probability was (but a
// row whose scores are all -inf stays empty). 43 us more for the blocks of one
// tile that lost some.
//
// Work split: plan_kernel lists the blocks of every sequence, deals whole items
// (block, K/V head) to the CTAs round by round, so that the CTAs walk the same
// head's tiles in step and find them in L2, and cuts the tiles of the
// remaining items into shares that even the CTAs out. A share of an item
// leaves its sums in the workspace, and chunk_join_kernel adds an item's shares
// in the CTAs' order, so the result does not depend on timing.
//
// Measured on the device, plan and joins included (32 query heads over 8): 2048
// new tokens at the end of 16384 keys, bf16 483-490 us = 1060 TFLOP/s in short
// bursts at 1965 MHz (0.64 of the measured cuBLAS rate: the two halves' softmax
// chains and the tensor pipe, 50 % busy, alternate) and 547 us under load that
// meets the power cap (1.72 GHz); e4m3 0.69-0.72 ms = 720-750 TFLOP/s (the K
// scales' loads in the softmax warps and the conversion come on top; 512 threads
// leave 128 registers, of which the softmax spills 53 words and warps 2 and 3
// use none); eight sequences of 1 to 256 new tokens over up to 4096 bf16 keys
// 119 us = 520 TFLOP/s, of which the plan and the joins are about 15.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "paged.cuh"
#include "paged_split.cuh"
#include "sm100_paged.h"
#include "sm100_softmax.cuh"

namespace attn {

using namespace sm100;

namespace {

constexpr int kPD = 128;         // head width
constexpr int kPTile = 128;      // keys per tile
constexpr int kPRows = 256;      // query rows per block, two halves
constexpr int kPStages = 2;      // K/V ring depth
constexpr int kPlanSmem = 1024;  // blocks and sequences whose lists the plan keeps in shared memory
constexpr int kPMinTiles = 2;    // tiles a CTA takes at least
constexpr uint32_t kPTileB = kPTile * kPD * 2;  // 32 KB
constexpr uint32_t kPRawB = kPTile * kPD;       // 16 KB, e4m3
constexpr uint32_t kPQ = 0;
constexpr uint32_t kPK = kPQ + 2 * kPTileB;
constexpr uint32_t kPV = kPK + kPStages * kPTileB;
constexpr uint32_t kPRaw = kPV + kPStages * kPTileB;  // e4m3: K, V

// ------------------------------------------------------------------- plan

struct PlanHead {
  int64_t total;                       // tiles of all items
  int32_t pairs, items, rounds, ranks; // (sequence, block) pairs; items = pairs x Hkv; whole rounds; shares
};
struct PlanCta {
  int64_t u, left;          // its share: `left` tiles from tile index u on
  int32_t item, at, rank, pad;  // that is tile `at` of `item`; the share's number
};
struct PlanPair {  // a block, with its sequence's view: one load names a piece
  int32_t b, blk, tiles, q0, n, L, pad[2];
};

struct PlanP {
  PlanHead* head;
  PlanCta* cta;       // [ctas]
  int64_t* starts;    // [ctas] first tile of each share
  int32_t* cta_of;    // [ctas] its CTA
  PlanPair* pair;     // [cap] longest blocks of a sequence first
  int64_t* prefix;    // [cap + 1] tiles before the pair's items
  int32_t* first;     // [batch + 1] blocks before the sequence
  JoinRec* rec;       // [ctas] by share
  float* part;        // [ctas][2] partial results
  int32_t ctas, cap;
  int32_t tokens;     // tokens per block
};

// Block blk of sequence b: its rows and the key tiles they see.
__device__ __forceinline__ Item block_item(const PagedP& p, int tokens, const SeqView& s, int b, int blk) {
  Item it;
  it.b = b;
  it.h = 0;
  it.s = s;
  const int group = p.Hq / p.c.Hkv;
  const int tok0 = blk * tokens, ntok = it.s.n - tok0 < tokens ? it.s.n - tok0 : tokens;
  it.row0 = tok0 * group;
  it.rows = ntok * group;
  it.blocks = (it.s.n + tokens - 1) / tokens;
  const int64_t p0 = it.s.L - it.s.n + tok0, p1 = p0 + ntok - 1;
  const int64_t top = (p.flags & ATTN_MASK_CAUSAL) && p1 < it.s.L - 1 ? p1 : it.s.L - 1;
  it.hi = top < 0 ? 0 : (int)(top / kPTile) + 1;
  it.lo = it.nf = 0;
  if (p.flags & ATTN_MASK_WINDOW) {
    const int64_t lo = p0 - p.window + 1;
    it.lo = lo > 0 ? (int)(lo / kPTile) : 0;
    const int64_t f = p.first < top + 1 ? p.first : top + 1;
    it.nf = f > 0 ? (int)((f + kPTile - 1) / kPTile) : 0;
  }
  const int from = it.lo > it.nf ? it.lo : it.nf;
  it.tiles = it.nf + (it.hi > from ? it.hi - from : 0);
  if (it.tiles < 1) it.tiles = 1;
  return it;
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* a, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

constexpr int kPlanThreads = 256;  // at least one per CTA

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PagedP p, const PlanP pl) {
  __shared__ SplitShared ss;
  __shared__ int32_t longest[kPlanThreads / 32];
  // The lists are read many times over: from shared memory where they fit.
  __shared__ int32_t s_first[kPlanSmem + 1], s_tiles[kPlanSmem];
  __shared__ int64_t s_prefix[kPlanSmem + 1];
  dependents_may_launch();
  const CacheP& c = p.c;
  const int tid = threadIdx.x, n = blockDim.x, B = c.batch, Hkv = c.Hkv, G = pl.ctas;
  if (tid < (int)(kStatusBytes / 4)) c.status[tid] = 0u;
  for (int i = tid; i < G; i += n) pl.rec[i].parts = 0;
  __syncthreads();
  report_ragged(c);
  int32_t* first = B <= kPlanSmem ? s_first : pl.first;
  int64_t before, carry = 0;
  for (int b0 = 0; b0 < B; b0 += n) {
    const int b = b0 + tid;
    const int64_t blocks = b < B ? (seq_view(c, b).n + pl.tokens - 1) / pl.tokens : 0;
    const int64_t sum = block_sum_scan(blocks, ss, before);
    if (b < B) first[b] = (int)(carry + before < pl.cap ? carry + before : pl.cap);
    carry += sum;
  }
  // More blocks than cap only come from overlapping cu_q ranges (reported).
  const int NB = (int)(carry < pl.cap ? carry : pl.cap);
  const bool small = NB <= kPlanSmem;
  int64_t* prefix = small ? s_prefix : pl.prefix;
  auto tiles_of = [&](int j) { return small ? s_tiles[j] : pl.pair[j].tiles; };
  __syncthreads();
  carry = 0;
  for (int j0 = 0; j0 < NB; j0 += n) {
    const int j = j0 + tid;
    int64_t units = 0;
    if (j < NB) {
      const int i = NB - 1 - j, b = last_at_most(first, B, i), blk = i - first[b];
      const SeqView sv = seq_view(c, b);
      const int tiles = block_item(p, pl.tokens, sv, b, blk).tiles;
      pl.pair[j] = PlanPair{b, blk, tiles, sv.q0, sv.n, (int)sv.L, {0, 0}};
      if (small) s_tiles[j] = tiles;
      units = (int64_t)tiles * Hkv;
    }
    const int64_t sum = block_sum_scan(units, ss, before);
    if (j < NB) prefix[j] = carry + before;
    carry += sum;
  }
  const int64_t W = carry;
  if (tid == 0) prefix[NB] = W;
  __syncthreads();
  const int NI = NB * Hkv;
  // Whole rounds, as many as leave no CTA (much) longer than the average.
  const int64_t avg = (W + G - 1) / G;
  int rounds = NI / G;
  int64_t whole = 0;
  const int most = rounds;
  for (int tries = 0; rounds > 0; ++tries) {
    whole = 0;
    if (tid < G)
      for (int r = 0; r < rounds; ++r) whole += tiles_of((tid + r * G) / Hkv);
    const int top = __reduce_max_sync(0xffffffffu, (int)(whole < 0x7fffffff ? whole : 0x7fffffff));
    __syncthreads();
    if ((tid & 31) == 0) longest[tid >> 5] = top;
    __syncthreads();
    const int64_t most_of = __reduce_max_sync(0xffffffffu, longest[tid & (kPlanThreads / 32 - 1)]);
    const bool fits = most_of * 32 <= avg * 33;
    if (fits) break;
    rounds = tries == 0 ? rounds - 1 : tries == 1 ? most * 3 / 4 : tries == 2 ? most / 2 : 0;
  }
  if (rounds == 0) whole = 0;
  const int F = rounds * G;
  const int64_t u0 = F < NI ? prefix[F / Hkv] + (int64_t)(F % Hkv) * tiles_of(F / Hkv) : W;
  const int64_t rest = W - u0;
  int64_t active = (rest + kPMinTiles - 1) / kPMinTiles;
  active = active > G ? G : active;
  const int64_t need = tid >= G ? 0 : rounds ? (avg > whole ? avg - whole : 0) : (tid < active ? 1 : 0);
  int64_t total = block_sum_scan(need, ss, before);
  if (total < 1) total = 1;
  const int64_t u = u0 + before * rest / total, end = u0 + (before + need) * rest / total;
  const bool has = tid < G && end > u;
  int64_t rank;
  const int64_t ranks = block_sum_scan(has ? 1 : 0, ss, rank);
  if (tid < G) {
    PlanCta t{u, has ? end - u : 0, 0, 0, (int)rank, 0};
    if (has) {
      const int j = last_at_most(prefix, NB, u), tiles = tiles_of(j);
      const int64_t rem = u - prefix[j];
      t.item = j * Hkv + (int)(rem / tiles);
      t.at = (int)(rem % tiles);
      pl.starts[rank] = u;
      pl.cta_of[rank] = tid;
    }
    pl.cta[tid] = t;
  }
  if (tid == 0) *pl.head = PlanHead{W, NB, NI, rounds, (int)ranks};
}

// The pieces of one CTA in order; every role of the CTA walks the same ones.
struct Pieces {
  PlanHead head;
  PlanCta mine;
  int r;
  __device__ __forceinline__ void init(const PlanP& pl) {
    head = *pl.head;
    mine = pl.cta[blockIdx.x];
    r = 0;
  }
  // The next piece: item it, tiles [k0, k1); u: index of its first tile, -1 in a whole round.
  __device__ __forceinline__ bool next(const PagedP& p, const PlanP& pl, Item& it, int& k0, int& k1, int64_t& u) {
    int item;
    if (r < head.rounds) {
      item = blockIdx.x + r * pl.ctas;
      ++r;
      u = -1;
    } else if (mine.left > 0) {
      item = mine.item;
      u = mine.u;
    } else {
      return false;
    }
    const PlanPair pr = pl.pair[item / p.c.Hkv];
    it = block_item(p, pl.tokens, SeqView{pr.q0, pr.n, pr.L}, pr.b, pr.blk);
    it.h = item % p.c.Hkv;
    if (u < 0) {
      k0 = 0;
      k1 = it.tiles;
    } else {
      k0 = mine.at;
      k1 = it.tiles - k0 < mine.left ? it.tiles : (int)(k0 + mine.left);
      mine.left -= k1 - k0;
      mine.u += k1 - k0;
      mine.item++;
      mine.at = 0;
    }
    return true;
  }
};

// What the two halves of a block see of a tile.
struct Halves {
  // Positions, lengths and windows are below 2^30 (the cache's limit), so that
  // their sums and differences fit 32 bits.
  int rows[2];
  int p0[2], p1[2];  // positions of the half's first and last token
  int L, window, first;
  bool causal, win;
  __device__ __forceinline__ void init(const PagedP& p, const Item& it) {
    const int group = p.Hq / p.c.Hkv;
    const int base = (int)it.s.L - it.s.n;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      rows[w] = it.rows - 128 * w;
      rows[w] = rows[w] < 0 ? 0 : (rows[w] > 128 ? 128 : rows[w]);
      p0[w] = base + (it.row0 + 128 * w) / group;
      p1[w] = base + (it.row0 + 128 * w + rows[w] - 1) / group;
    }
    L = (int)it.s.L;
    causal = p.flags & ATTN_MASK_CAUSAL;
    win = p.flags & ATTN_MASK_WINDOW;
    window = (int)p.window;
    first = (int)p.first;
  }
  // kEmptyH: no row of half w sees a key of tile kt; kFullH: all see all.
  __device__ __forceinline__ int cls(int w, int kt) const {
    const int c0 = kt * kPTile, c1 = c0 + kPTile - 1;
    if (rows[w] == 0 || c0 >= L || p1[w] < 0) return 0;
    if (causal && c0 > p1[w]) return 0;
    if (win && c0 >= first && c1 <= p0[w] - window) return 0;
    if (c1 >= L || p0[w] < 0 || (causal && c1 > p0[w])) return 1;
    if (win && c1 >= first && (c0 > first ? c0 : first) <= p1[w] - window) return 1;
    return 2;
  }
  // Bits 2 w, 2 w + 1: the class of half w.
  __device__ __forceinline__ uint32_t both(int kt) const { return (uint32_t)cls(0, kt) | (uint32_t)cls(1, kt) << 2; }
};

// Some half sees the tile in part.
__device__ __forceinline__ bool in_part(uint32_t cls) { return (cls & 3u) == 1u || (cls >> 2) == 1u; }

// First k in [k, k1) whose tile some half sees (k1 when none), and its classes.
__device__ __forceinline__ int next_seen(const Item& it, const Halves& hv, int k, int k1, uint32_t& cls) {
  for (; k < k1; ++k)
    if ((cls = hv.both(it.tile_at(k))) != 0u) return k;
  cls = 0;
  return k1;
}

struct PagedCtl {
  uint64_t q_full;
  uint64_t raw_full[2], raw_empty[2];  // e4m3: raw K, raw V
  uint64_t k_full[kPStages], v_full[kPStages], v_ok[kPStages], kv_empty[kPStages];
  uint64_t s_full[2], p_full[2];
  uint64_t o_final;
  uint64_t o_read;  // one arrival per softmax warp: it has passed o_final and read lost_lo, lost_hi
  uint32_t tmem_base;
  uint32_t abort_flag;
  // 1 + k of the tiles whose V lost non-finite elements, 0 none: by stage and
  // checker warp (set before v_ok), and the piece's first and last (before o_final).
  uint32_t tile_lost[kPStages][4], lost_lo, lost_hi;
  // e4m3, by 32 keys: the K scales' extremes, and the power of two (its
  // logarithm) that V's scales were divided by.
  float ks_top[kPStages][4], ks_low[kPStages][4], v_exp[kPStages][4];
  // Per stage: bits 0-3 the halves' classes, bit 4 another tile follows, bits
  // 8-15 boxes in pages outside the pool. raw_info: the same, with the raw K tile.
  uint32_t tinfo[kPStages];
  uint32_t raw_info;
};

template <bool kQ8>
struct PagedSmem {
  static constexpr uint32_t kScale = kPRaw + (kQ8 ? 2 * kPRawB : 0);  // kPStages x 128 K scales, fp32
  static constexpr uint32_t kCtl = kScale + (kQ8 ? kPStages * 512 : 0);
  static constexpr uint32_t kBytes = kCtl + 512;
  static constexpr int kThreads = kQ8 ? 512 : 384;
  static constexpr int kCheckers = kQ8 ? 4 : 2;  // warps 12-15, or 2 and 3
};
static_assert(sizeof(PagedCtl) <= 512, "control block");

// Row i's keys of tile kt as two 64-bit words.
__device__ __forceinline__ void row_bits(const Halves& hv, int pos, bool live, int kt, uint32_t bad, int box,
                                         uint64_t& w0, uint64_t& w1) {
  const int j0 = kt * kPTile;
  w0 = w1 = 0ull;
  if (!live || pos < 0) return;
  int hi = hv.L - 1;
  if (hv.causal && pos < hi) hi = pos;
  int lo = j0;
  if (hv.win && pos - hv.window + 1 > lo) lo = pos - hv.window + 1;
  w0 = range_bits64(lo - j0, hi - j0);
  w1 = range_bits64(lo - j0 - 64, hi - j0 - 64);
  if (hv.win && j0 < hv.first) {
    const int fh = hv.first - 1 < hi ? hv.first - 1 : hi;
    w0 |= range_bits64(0, fh - j0);
    w1 |= range_bits64(-64, fh - j0 - 64);
  }
  while (bad) {
    const int i = __ffs(bad) - 1;
    bad &= bad - 1;
    w0 &= ~range_bits64(i * box, i * box + box - 1);
    w1 &= ~range_bits64(i * box - 64, i * box + box - 65);
  }
}

// A masked row of a 16-bit tile, as softmax_masked_tile with its strict rules,
// but 32-key groups that no row of the warp sees are skipped and groups that
// all its rows see take no select: with a causal edge, rows of a warp (8
// tokens of 4 heads, say) differ in few columns, and one group of the four
// is mixed. 4.0 -> 1.9 us for a tile's two halves.
template <bool kH>
__device__ __forceinline__ float softmax_edge_tile(uint32_t tS, float scale_log2, uint64_t mw0, uint64_t mw1,
                                                   float& m_run, float& l_run) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t mw = (uint32_t)((q < 2 ? mw0 : mw1) >> (32 * (q & 1)));
    if (!__any_sync(0xffffffffu, mw != 0u)) continue;
    uint32_t r[32];
    tmem_ld32(tS + q * 32, r);
    tmem_wait_ld();
    if (!__all_sync(0xffffffffu, mw == ~0u)) {
      const float hide = scale_log2 >= 0.f ? -INFINITY : INFINITY;
#pragma unroll
      for (int e = 0; e < 32; ++e) r[e] = (mw >> e) & 1u ? r[e] : __float_as_uint(hide);
    }
    if (scale_log2 == 0.f) {  // 0 times the infinity that hides a key is not -inf
      if (mw) mx = max3nan(mx, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (((mw >> e) & 1u) && !isfinite(__uint_as_float(r[e]))) mx = NAN;
      continue;
    }
    float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
    if (scale_log2 > 0.f) {
#pragma unroll
      for (int e = 2; e < 32; e += 2) {
        a = max3nan(a, __uint_as_float(r[e]), a);
        b = max3nan(b, __uint_as_float(r[e + 1]), b);
      }
      a = max3nan(a, b, b);
    } else {
#pragma unroll
      for (int e = 2; e < 32; e += 2) {
        a = min3nan(a, __uint_as_float(r[e]), a);
        b = min3nan(b, __uint_as_float(r[e + 1]), b);
      }
      a = min3nan(a, b, b);
    }
    mx = max3nan(mx, a * scale_log2, mx);
  }
  const bool poison = !(mx < INFINITY);
  if (poison) mx = -INFINITY;
  const float alpha = move_max(mx, m_run);
  const float msub = m_run == -INFINITY ? 0.f : m_run;
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-msub, -msub);
  uint64_t acc0 = 0ull, acc1 = 0ull;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t mw = (uint32_t)((q < 2 ? mw0 : mw1) >> (32 * (q & 1)));
    uint32_t pk[16];
    if (!__any_sync(0xffffffffu, mw != 0u)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = 0u;
    } else {
      uint32_t r[32];
      tmem_ld32(tS + q * 32, r);
      tmem_wait_ld();
      const bool on = __all_sync(0xffffffffu, mw == ~0u);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sc2, nm2), x0, x1);
        x0 = ex2(x0);
        x1 = ex2(x1);
        if (!on) {
          x0 = (mw >> (2 * e)) & 1u ? x0 : 0.f;
          x1 = (mw >> (2 * e + 1)) & 1u ? x1 : 0.f;
        }
        if (e & 1)
          acc1 = f2_add(acc1, f2_pack(x0, x1));
        else
          acc0 = f2_add(acc0, f2_pack(x0, x1));
        pk[e] = pack16<kH>(x0, x1);
      }
    }
    tmem_st16(tS + q * 16, pk);
  }
  float a0, a1, b0, b1;
  f2_unpack(acc0, a0, a1);
  f2_unpack(acc1, b0, b1);
  l_run = poison ? NAN : l_run * alpha + ((a0 + a1) + (b0 + b1));
  return alpha;
}

// The row of an e4m3 tile: scores times the keys' scales ksc (which carry
// c log2(e)); V's scales are in its operand but for a power of two per 32
// keys, 2^vexp, which the probabilities take: the running reference m is that
// of s + vexp, P = 2^(s - m + vexp) in fp16, and the sum 2^(s - m) in fp32.
// The reference needs no exact maximum: where the largest unscaled score times
// `top` (`low`, if it is negative), the tile's extreme K scales, is above the
// largest exponent by 8 at most, so that P's largest value is 2^-8 or more and
// fp16's smallest step 2^-17 of it or less, that serves, and spares the first
// pass its 128 products and scale loads: those loads, 512 bytes of registers
// per warp and instruction, are what bounds this kernel. Elsewhere, and in
// masked tiles, the exact maximum. Strict like the 16-bit rows' functions.
template <bool kMasked>
__device__ __forceinline__ float softmax_scaled_tile(uint32_t tS, const float* ksc, const float* vexp, float top,
                                                     float low, uint64_t mw0, uint64_t mw1, float& m_run,
                                                     float& l_run) {
  float mx = -INFINITY;
  bool done = false;
  if constexpr (!kMasked) {
    float e0 = -INFINITY, e1 = e0, e2 = e0, e3 = e0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t s0[32], s1[32];
      tmem_ld32(tS + 64 * hf, s0);
      tmem_ld32(tS + 64 * hf + 32, s1);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        e0 = max3nan(e0, __uint_as_float(s0[e]), __uint_as_float(s0[e + 1]));
        e1 = max3nan(e1, __uint_as_float(s0[e + 2]), __uint_as_float(s0[e + 3]));
        e2 = max3nan(e2, __uint_as_float(s1[e]), __uint_as_float(s1[e + 1]));
        e3 = max3nan(e3, __uint_as_float(s1[e + 2]), __uint_as_float(s1[e + 3]));
      }
    }
    const float raw = max3nan(max3nan(e0, e1, e2), e3, e3);
    const float near = fmaxf(fmaxf(vexp[0], vexp[1]), fmaxf(vexp[2], vexp[3]));
    const float far = fminf(fminf(vexp[0], vexp[1]), fminf(vexp[2], vexp[3]));
    done = __all_sync(0xffffffffu, low > 0.f && fabsf(raw) * (top - low) + (near - far) <= 8.f);
    mx = raw * (raw >= 0.f ? top : low) + near;
  }
  if (!done) {
    mx = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const uint32_t mw = (uint32_t)((q < 2 ? mw0 : mw1) >> (32 * (q & 1)));
      if (kMasked && !__any_sync(0xffffffffu, mw != 0u)) continue;
      uint32_t r[32];
      tmem_ld32(tS + q * 32, r);
      tmem_wait_ld();
      float a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(ksc + q * 32 + e);
        float x0 = __uint_as_float(r[e]) * k4.x, x1 = __uint_as_float(r[e + 1]) * k4.y;
        float x2 = __uint_as_float(r[e + 2]) * k4.z, x3 = __uint_as_float(r[e + 3]) * k4.w;
        if constexpr (kMasked) {
          x0 = (mw >> e) & 1u ? x0 : -INFINITY;
          x1 = (mw >> (e + 1)) & 1u ? x1 : -INFINITY;
          x2 = (mw >> (e + 2)) & 1u ? x2 : -INFINITY;
          x3 = (mw >> (e + 3)) & 1u ? x3 : -INFINITY;
        }
        a = max3nan(a, x0, x1);
        b = max3nan(b, x2, x3);
      }
      mx = max3nan(mx, max3nan(a, b, b) + vexp[q], mx);
    }
  }
  const bool poison = !(mx < INFINITY);
  if (poison) mx = -INFINITY;
  const float alpha = move_max(mx, m_run);
  const float msub = m_run == -INFINITY ? 0.f : m_run;
  float sum = 0.f;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t mw = (uint32_t)((q < 2 ? mw0 : mw1) >> (32 * (q & 1)));
    uint32_t pk[16];
    if (kMasked && !__any_sync(0xffffffffu, mw != 0u)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = 0u;
      tmem_st16(tS + q * 16, pk);
      continue;
    }
    uint32_t r[32];
    tmem_ld32(tS + q * 32, r);
    const float off = vexp[q] - msub;
    const uint64_t nm2 = f2_pack(off, off);
    uint64_t acc0 = 0ull, acc1 = 0ull;
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(ksc + q * 32 + e);  // packed pairs
      const uint64_t x01 = f2_fma(f2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), k4.x, nm2);
      const uint64_t x23 = f2_fma(f2_pack(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), k4.y, nm2);
      float x[4];
      f2_unpack(x01, x[0], x[1]);
      f2_unpack(x23, x[2], x[3]);
      uint64_t y01, y23;
      if constexpr (kMasked) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (mw >> (e + i)) & 1u ? ex2(x[i]) : 0.f;
        y01 = f2_pack(x[0], x[1]);
        y23 = f2_pack(x[2], x[3]);
      } else {
        y01 = f2_pack(ex2(x[0]), ex2(x[1]));
        // every fourth pair on the FMA pipe, as in the 16-bit rows
        y23 = (e & 4) ? exp2_pair<true>(x[2], x[3]) : f2_pack(ex2(x[2]), ex2(x[3]));
        f2_unpack(y01, x[0], x[1]);
        f2_unpack(y23, x[2], x[3]);
      }
      acc0 = f2_add(acc0, y01);
      acc1 = f2_add(acc1, y23);
      pk[e / 2] = pack_fp16(x[0], x[1]);
      pk[e / 2 + 1] = pack_fp16(x[2], x[3]);
    }
    tmem_st16(tS + q * 16, pk);
    float a0, a1, b0, b1;
    f2_unpack(acc0, a0, a1);
    f2_unpack(acc1, b0, b1);
    sum = fmaf((a0 + a1) + (b0 + b1), __uint_as_float((uint32_t)(127 - (int)vexp[q]) << 23), sum);  // 2^-vexp
  }
  l_run = poison ? NAN : l_run * alpha + sum;
  return alpha;
}

// Columns 32 ch + e (bit e) of the calling thread's row that get a NaN, +inf or
// -inf back: the non-finite elements that the checkers took out of V, of the
// keys that the row sees. By a whole warp, which owns 32 rows of the block: of
// the tiles in [k0, k1) that lose any (seen in part, or with a box outside
// the pool) each lane looks at one key in 32, and every key that has some is
// shown to all rows. Few tiles are seen in part; with the rows' keys one after
// another, and in every tile of the piece, a chunk of a million keys would have
// taken seconds for one NaN, and the other roles' waits would have run out.
struct LostColumns {
  uint32_t nan, up, down;
};

template <bool kH, bool kQ8>
__device__ __forceinline__ LostColumns lost_columns(const PagedP& p, const Item& it, const Halves& hv, int k0, int k1,
                                                    int pos, bool valid, int box, int ch) {
  const CacheP& c = p.c;
  const int lane = threadIdx.x & 31;
  LostColumns lost{0u, 0u, 0u};
  if (!__any_sync(0xffffffffu, valid)) return lost;
  uint32_t cls;
  auto page_at = [&](int j) {  // -1: past the end or outside the pool
    if (j >= hv.L) return -1;
    const int pg = c.table[(int64_t)it.b * c.table_stride + (unsigned)j / (unsigned)c.page_size];
    return pg < c.num_pages ? pg : -1;
  };
#pragma unroll 1
  for (int k = next_seen(it, hv, k0, k1, cls); k < k1; k = next_seen(it, hv, k + 1, k1, cls)) {
    const int j0 = it.tile_at(k) * kPTile;
    if (!in_part(cls)) {
      const int j = j0 + lane * box;
      if (!__any_sync(0xffffffffu, lane * box < kPTile && j < hv.L && page_at(j) < 0)) continue;
    }
    uint64_t w0, w1;
    row_bits(hv, pos, valid, it.tile_at(k), 0u, box, w0, w1);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const uint32_t sees = (uint32_t)((q < 2 ? w0 : w1) >> (32 * (q & 1)));
      const int j = j0 + 32 * q + lane, pg = page_at(j);
      uint32_t nan = 0u, up = 0u, down = 0u;
      if (pg >= 0) {
        const int64_t off = (unsigned)j % (unsigned)c.page_size;
        const int64_t at = pg * c.sv[0] + off * c.sv[1] + (int64_t)it.h * c.sv[2] + ch * 32;
        const float vs = kQ8 ? c.vs[pg * c.svs[0] + off * c.svs[1] + (int64_t)it.h * c.svs[2]] : 1.f;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.v) + at * (kQ8 ? 1 : 2));
#pragma unroll 4
        for (int i = 0; i < (kQ8 ? 8 : 16); ++i) {
          const uint32_t v = row[i];
          float x[4];
          if constexpr (kQ8) {
            const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3);
            const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v >> 16), __NV_E4M3);
            const float2 f0 = __half22float2(__half2(a)), f1 = __half22float2(__half2(b));
            x[0] = f0.x * vs, x[1] = f0.y * vs, x[2] = f1.x * vs, x[3] = f1.y * vs;
          } else {
            const float2 f = unpack16<kH>(v);
            x[0] = f.x, x[1] = f.y;
          }
#pragma unroll
          for (int e = 0; e < (kQ8 ? 4 : 2); ++e) {
            const uint32_t bit = 1u << ((kQ8 ? 4 : 2) * i + e);
            if (x[e] != x[e]) nan |= bit;
            if (x[e] == INFINITY) up |= bit;
            if (x[e] == -INFINITY) down |= bit;
          }
        }
      }
      uint32_t keys = __ballot_sync(0xffffffffu, (nan | up | down) != 0u);
      while (keys) {
        const int src = __ffs(keys) - 1;
        keys &= keys - 1;
        const uint32_t a = __shfl_sync(0xffffffffu, nan, src), b = __shfl_sync(0xffffffffu, up, src),
                       d = __shfl_sync(0xffffffffu, down, src);
        if ((sees >> src) & 1u) {
          lost.nan |= a;
          lost.up |= b;
          lost.down |= d;
        }
      }
    }
  }
  return lost;
}

template <bool v>
struct Tag {
  static constexpr bool value = v;
};

template <bool kH, bool kQ8>
__global__ void __launch_bounds__(PagedSmem<kQ8>::kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedP p,
                   const __grid_constant__ PlanP pl, int box, int q_boxes) {
  using M = PagedSmem<kQ8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  PagedCtl* ctl = reinterpret_cast<PagedCtl*>(smem + M::kCtl);
  volatile uint32_t* abort_flag = &ctl->abort_flag;
  const CacheP& c = p.c;
  uint32_t* status = c.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kHP = kH || kQ8;  // P and V in fp16, else bf16

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&ctl->q_full), q_boxes ? 1 : 8);
    for (int s = 0; s < kPStages; ++s) {
      mbar_init(smem_u32(&ctl->raw_full[s]), 1);
      mbar_init(smem_u32(&ctl->raw_empty[s]), M::kCheckers);
      mbar_init(smem_u32(&ctl->k_full[s]), kQ8 ? M::kCheckers : 1);
      mbar_init(smem_u32(&ctl->v_full[s]), 1);
      mbar_init(smem_u32(&ctl->v_ok[s]), M::kCheckers);
      mbar_init(smem_u32(&ctl->kv_empty[s]), 1);
      mbar_init(smem_u32(&ctl->s_full[s]), 1);
      mbar_init(smem_u32(&ctl->p_full[s]), 4);
    }
    mbar_init(smem_u32(&ctl->o_final), 2);  // the products' completion, and the word in front of it
    mbar_init(smem_u32(&ctl->o_read), 8);
    ctl->abort_flag = 0;
    ctl->lost_lo = ctl->lost_hi = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  // TMEM columns: S/P of half w at 128 w, O of half w at 256 + 128 w.
  wait_for_previous();
  Pieces pieces;
  pieces.init(pl);
  Item it;
  Halves hv;
  int k0, k1;
  int64_t u;

  if (warp == 0) {
    // ---------------- producer: lane i < 128 / box takes box i of every tile
    if (lane == 0) {
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    const int boxes = kPTile / box;
    int n = 0;
    [[maybe_unused]] int nk8 = 0;  // e4m3: raw K tiles under way or landed (n: K and V)
    bool ok = true;
    while (ok && pieces.next(p, pl, it, k0, k1, u)) {
      hv.init(p, it);
      uint32_t cls;
      int k = next_seen(it, hv, k0, k1, cls);
      auto page_at = [&](int kk) {  // -2: past the end, -1: outside the pool
          const int j = it.tile_at(kk) * kPTile + lane * box;
          if (lane >= boxes || j >= hv.L) return -2;
          const int pg = c.table[(int64_t)it.b * c.table_stride + (unsigned)j / (unsigned)c.page_size];
          if (pg >= 0 && pg < c.num_pages) return pg;
          set_status(status, ATTN_DEVERR_PAGE);
          return -1;
      };
      int pg = k < k1 ? page_at(k) : -2;
      while (k < k1) {
        uint32_t ncls;
        const int nk = next_seen(it, hv, k + 1, k1, ncls);
        const int npg = nk < k1 ? page_at(nk) : -2;
        const int s = n % kPStages;
        const uint32_t info = cls | (nk < k1 ? 16u : 0u) | __ballot_sync(0xffffffffu, pg == -1) << 8;
        const int off = (int)((unsigned)(it.tile_at(k) * kPTile + lane * box) % (unsigned)c.page_size);
        const int page = pg < 0 ? 0 : pg;  // whatever is there: masked, and made finite by the checkers
        if constexpr (!kQ8) {
          ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl->kv_empty[s]), ((n / kPStages) & 1) ^ 1, abort_flag, status));
          if (!ok) break;
          const uint32_t kf = smem_u32(&ctl->k_full[s]), vf = smem_u32(&ctl->v_full[s]);
          if (lane == 0) {
            ctl->tinfo[s] = info;  // published by the arrive below
            mbar_expect_tx(kf, kPTileB);
            mbar_expect_tx(vf, kPTileB);
          }
          __syncwarp();
          if (lane < boxes) {
            const uint32_t kd = sbase + kPK + s * kPTileB + lane * box * 128;
            const uint32_t vd = sbase + kPV + s * kPTileB + lane * box * 128;
            tma_load_4d(kd, &tk, kf, 0, off, it.h, page);
            tma_load_4d(kd + kPTileB / 2, &tk, kf, 64, off, it.h, page);
            tma_load_4d(vd, &tv, vf, 0, off, it.h, page);
            tma_load_4d(vd + kPTileB / 2, &tv, vf, 64, off, it.h, page);
          }
        } else {
          const uint32_t kf = smem_u32(&ctl->raw_full[0]), vf = smem_u32(&ctl->raw_full[1]);
          ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl->raw_empty[0]), (n & 1) ^ 1, abort_flag, status));
          if (!ok) break;
          if (lane == 0) {
            ctl->raw_info = info;
            mbar_expect_tx(kf, kPRawB);
          }
          __syncwarp();
          if (lane < boxes) tma_load_4d(sbase + kPRaw + lane * box * 128, &tk, kf, 0, off, it.h, page);
          ++nk8;
          ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl->raw_empty[1]), (n & 1) ^ 1, abort_flag, status));
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(vf, kPRawB);
          __syncwarp();
          if (lane < boxes) tma_load_4d(sbase + kPRaw + kPRawB + lane * box * 128, &tv, vf, 0, off, it.h, page);
        }
        __syncwarp();
        ++n;
        k = nk;
        cls = ncls;
        pg = npg;
      }
    }
    // Every copy lands before the CTA's shared memory goes, aborted or not.
    uint32_t calm = 0;  // stands in for the abort flag, which would end these waits at once
    if constexpr (!kQ8) {
      for (int r = (n > kPStages ? n - kPStages : 0); r < n; ++r) {
        wait_bar(smem_u32(&ctl->k_full[r % kPStages]), (r / kPStages) & 1, &calm, nullptr);
        wait_bar(smem_u32(&ctl->v_full[r % kPStages]), (r / kPStages) & 1, &calm, nullptr);
      }
    } else {
      // (an abort between the two leaves a tile's K under way without its V)
      if (nk8 > 0) wait_bar(smem_u32(&ctl->raw_full[0]), (nk8 - 1) & 1, &calm, nullptr);
      if (n > 0) wait_bar(smem_u32(&ctl->raw_full[1]), (n - 1) & 1, &calm, nullptr);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (whole warp; one elected lane issues)
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc16<kH>(128, 128, 0, 0);
    constexpr uint32_t idPV = idesc16<kHP>(128, 128, 0, 1);
    const uint64_t dQ0 = smem_desc_sw128(sbase + kPQ, 16, 1024), dK0 = smem_desc_sw128(sbase + kPK, 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(sbase + kPV, kPTileB / 2, 1024);
    constexpr uint64_t kTileStep = kPTileB >> 4;
    auto wait_all = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, wait_bar(smem_u32(bar), par, abort_flag, status));
    };
    auto issue_s = [&](int w, int stage) {
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * (kPTileB / 2) + (kk & 3) * 32) >> 4;
          mma_ss(tmem + w * 128, dQ0 + (uint64_t)w * kTileStep + off, dK0 + (uint64_t)stage * kTileStep + off, idS, kk > 0);
        }
        mma_commit(smem_u32(&ctl->s_full[w]));
      }
      __syncwarp();
    };
    int n = 0, piece = 0;
    int done[2] = {0, 0};  // P tiles taken of each half, over all pieces
    bool ok = true;
    while (ok && pieces.next(p, pl, it, k0, k1, u)) {
      hv.init(p, it);
      uint32_t cls;
      const bool any = next_seen(it, hv, k0, k1, cls) < k1;
      // A piece begins once every softmax warp has passed the previous one's
      // o_final, whether the piece has tiles (or its half has) or not: o_final is
      // waited for by its parity, so nobody may be two of its phases behind.
      if (piece > 0 && !(ok = wait_all(&ctl->o_read, (piece - 1) & 1))) break;
      if (q_boxes) {
        // Q (the previous piece's products have read the last one: o_final): two
        // boxes of (64 columns, the group's heads, 128 / group tokens) a half.
        // Rows past the block's belong to other tokens; their results go
        // nowhere. The softmax warps may still be writing the previous piece:
        // its O and this piece's S are different columns.
        if (leader) {
          const uint32_t qf = smem_u32(&ctl->q_full);
          const int group = p.Hq / c.Hkv, halves = it.rows > 128 ? 2 : 1;
          mbar_expect_tx(qf, halves * kPTileB);
          for (int w = 0; w < halves; ++w) {
            const int tok = it.s.q0 + it.row0 / group + w * (128 / group);
            tma_load_3d(sbase + kPQ + w * kPTileB, &tq, qf, 0, it.h * group, tok);
            tma_load_3d(sbase + kPQ + w * kPTileB + kPTileB / 2, &tq, qf, 64, it.h * group, tok);
          }
        }
        __syncwarp();
      }
      if (!(ok = wait_all(&ctl->q_full, piece & 1))) {
        uint32_t calm = 0;  // Q's copies land before the CTA's shared memory goes
        if (q_boxes) wait_bar(smem_u32(&ctl->q_full), piece & 1, &calm, nullptr);
        break;
      }
      tc_fence_after();
      uint32_t info = 0, lost_lo = 0, lost_hi = 0;
      int npv[2] = {0, 0};
      if (any) {
        const int s = n % kPStages;
        if (!(ok = wait_all(&ctl->k_full[s], (n / kPStages) & 1))) break;
        tc_fence_after();
        info = ctl->tinfo[s];
        for (int w = 0; w < 2; ++w)
          if ((info >> (2 * w)) & 3u) issue_s(w, s);
      }
      while (any) {
        const int s = n % kPStages, s1 = (n + 1) % kPStages;
        const bool more = info & 16u;
        uint32_t ninfo = 0;
        for (int w = 0; w < 2 && ok; ++w) {
          if ((info >> (2 * w)) & 3u) {
            if (!(ok = wait_all(&ctl->p_full[w], done[w] & 1))) break;
            if (!(ok = wait_all(&ctl->v_ok[s], (n / kPStages) & 1))) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ts(tmem + 256 + w * 128, tmem + w * 128 + kk * 8,
                       dV0 + (uint64_t)s * kTileStep + (uint64_t)(kk * (2048 >> 4)), idPV,
                       (npv[w] > 0 || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
            ++npv[w];
            ++done[w];
          }
          if (more) {
            if (w == 0) {
              if (!(ok = wait_all(&ctl->k_full[s1], ((n + 1) / kPStages) & 1))) break;
              tc_fence_after();
              ninfo = ctl->tinfo[s1];
            }
            if ((ninfo >> (2 * w)) & 3u) issue_s(w, s1);
          }
        }
        if (!ok) break;
        const uint32_t lost = __reduce_max_sync(0xffffffffu, lane < M::kCheckers ? ctl->tile_lost[s][lane] : 0u);
        if (lost) {
          if (!lost_lo) lost_lo = lost;
          lost_hi = lost;
        }
        if (leader) mma_commit(smem_u32(&ctl->kv_empty[s]));
        __syncwarp();
        ++n;
        if (!more) break;
        info = ninfo;
      }
      if (!ok) break;
      if (leader) {
        ctl->lost_lo = lost_lo;  // (the softmax warps have read the previous piece's: o_read)
        ctl->lost_hi = lost_hi;
        mbar_arrive(smem_u32(&ctl->o_final));
        mma_commit(smem_u32(&ctl->o_final));
      }
      __syncwarp();
      ++piece;
    }
  } else if (kQ8 ? warp >= 12 : warp < 4) {
    // ---------------- checkers (e4m3: converters): V's non-finite elements, and
    // an e4m3 tile's 16-bit form
    const int ci = kQ8 ? warp - 12 : warp - 2;
    int n = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, wait_bar(smem_u32(bar), par, abort_flag, status));
    };
    while (ok && pieces.next(p, pl, it, k0, k1, u)) {
      hv.init(p, it);
      uint32_t cls, ncls;
      // e4m3: the thread's row of the tile. Its scales are loaded one tile
      // ahead and the page that holds them two, so that neither is waited for.
      const int row = ci * 32 + lane;
      float ks_next = 0.f, vs_next = 0.f;
      int page_next = -1;
      auto page_at = [&](int kk) {
        const unsigned j = (unsigned)(it.tile_at(kk) * kPTile + row);
        if (kk >= k1 || j >= (unsigned)hv.L) return -1;
        return (int)c.table[(int64_t)it.b * c.table_stride + j / (unsigned)c.page_size];
      };
      auto scales = [&](int kk, int pg) {
        ks_next = vs_next = 0.f;
        if (pg < 0 || pg >= c.num_pages) return;
        const unsigned o = (unsigned)(it.tile_at(kk) * kPTile + row) % (unsigned)c.page_size;
        ks_next = c.ks[pg * c.sks[0] + o * c.sks[1] + (int64_t)it.h * c.sks[2]];
        vs_next = c.vs[pg * c.svs[0] + o * c.svs[1] + (int64_t)it.h * c.svs[2]];
      };
      int k = next_seen(it, hv, k0, k1, cls);
      int nk = next_seen(it, hv, k + 1, k1, ncls);
      if constexpr (kQ8) {
        if (k < k1) scales(k, page_at(k));
        page_next = page_at(nk);
      }
      while (k < k1) {
        const int s = n % kPStages;
        const uint32_t par = (n / kPStages) & 1;
        const int live = hv.L - it.tile_at(k) * kPTile;  // rows of the tile inside the sequence
        bool part = in_part(cls);
        uint32_t nncls;
        const int nnk = next_seen(it, hv, nk + 1, k1, nncls);
        bool odd = false;
        if constexpr (!kQ8) {
          if (!(ok = wait_all(&ctl->v_full[s], par))) break;
          part = part || ctl->tinfo[s] >> 8 != 0u;
          if (part) {
            const uint32_t expo = kHP ? 0x7c00u : 0x7f80u;
            const uint32_t base = kPV + s * kPTileB + ci * (kPTileB / 2);  // one 64-column half a warp
#pragma unroll 4
            for (int i = 0; i < (int)(kPTileB / 2 / 512); ++i) {
              uint4* at = reinterpret_cast<uint4*>(smem + base + i * 512 + lane * 16);
              uint4 v = *at;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & expo) == expo) {
                  w[e] &= 0xffff0000u;
                  hit = true;
                }
                if (((w[e] >> 16) & expo) == expo) {
                  w[e] &= 0x0000ffffu;
                  hit = true;
                }
              }
              if (hit) {
                *at = make_uint4(w[0], w[1], w[2], w[3]);
                odd = odd || i * 4 + (lane >> 3) < live;
              }
            }
            fence_proxy_async_smem();
          }
        } else {
          const float ks = ks_next * (p.scale * kLog2e), vs = vs_next;
          scales(nk, page_next);
          page_next = page_at(nnk);
          // K: wait for the raw tile and for the operand stage
          if (!(ok = wait_all(&ctl->raw_full[0], n & 1))) break;
          if (!(ok = wait_all(&ctl->kv_empty[s], par ^ 1))) break;
          const uint32_t info = ctl->raw_info;
          if (ci == 0 && lane == 0) ctl->tinfo[s] = info;
          part = part || info >> 8 != 0u;
          float* sc = reinterpret_cast<float*>(smem + M::kScale + s * 512);
          sc[row] = ks;
          float hi = ks, lo = ks, ve = isfinite(vs) ? fabsf(vs) : 0.f;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            hi = max3nan(hi, __shfl_xor_sync(0xffffffffu, hi, o), hi);
            lo = min3nan(lo, __shfl_xor_sync(0xffffffffu, lo, o), lo);
            ve = fmaxf(ve, __shfl_xor_sync(0xffffffffu, ve, o));
          }
          // V's operand is code (s / 2^e) in fp16, with 2^e the power of two at
          // or below the 32 rows' largest scale (so below 896), and 2^e goes
          // to the probabilities' exponents. Rows whose scale is far below the
          // largest lose bits only where they are below 2^-25 of its rows.
          const int e2 = min(max((int)(__float_as_uint(ve) >> 23) - 127, -100), 120);
          if (lane == 0) {
            ctl->ks_top[s][ci] = hi;
            ctl->ks_low[s][ci] = lo;
            ctl->v_exp[s][ci] = (float)e2;
          }
          // vs / 2^e in two steps that stay in range
          const float vq = vs * __uint_as_float((uint32_t)(127 - e2 / 2) << 23) *
                           __uint_as_float((uint32_t)(127 - (e2 - e2 / 2)) << 23);
          const __half2 vh = __float2half2_rn(vq);
          const uint32_t vscale = *reinterpret_cast<const uint32_t*>(&vh);
          // kV: V rows (scaled, in fp16); else K rows in the type of Q.
          auto turn = [&](auto value_rows, uint32_t raw, uint32_t dst) {
            constexpr bool kV = decltype(value_rows)::value, kOutH = kV || kH;
#pragma unroll 4
            for (int ch = 0; ch < 8; ++ch) {  // 16 codes -> two 16-byte chunks
              const uint4 v = *reinterpret_cast<const uint4*>(smem + raw + sw128_offset(row, ch * 16));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t h0, h1;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                    : "=r"(h0), "=r"(h1)
                    : "r"(w[e]));
                if constexpr (kV) {
                  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h0) : "r"(vscale));
                  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h1) : "r"(vscale));
                }
                if constexpr (kOutH) {
                  o[2 * e] = h0;
                  o[2 * e + 1] = h1;
                } else {
                  const float2 f0 = unpack16<true>(h0), f1 = unpack16<true>(h1);
                  o[2 * e] = pack_bf16(f0.x, f0.y);
                  o[2 * e + 1] = pack_bf16(f1.x, f1.y);
                }
              }
              const uint32_t half = dst + (ch >> 2) * (kPTileB / 2);
              *reinterpret_cast<uint4*>(smem + half + sw128_offset(row, (ch & 3) * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(smem + half + sw128_offset(row, (ch & 3) * 32 + 16)) =
                  make_uint4(o[4], o[5], o[6], o[7]);
            }
          };
          turn(Tag<false>(), kPRaw, kPK + s * kPTileB);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&ctl->k_full[s]));
            mbar_arrive(smem_u32(&ctl->raw_empty[0]));
          }
          if (!(ok = wait_all(&ctl->raw_full[1], n & 1))) break;
          turn(Tag<true>(), kPRaw + kPRawB, kPV + s * kPTileB);
          if (part) {  // the thread's own row again: non-finite elements to 0
#pragma unroll 1
            for (int ch = 0; ch < 16; ++ch) {
              uint32_t* at = reinterpret_cast<uint32_t*>(smem + kPV + s * kPTileB + (ch >> 3) * (kPTileB / 2) +
                                                         sw128_offset(row, (ch & 7) * 16));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t h = at[e], f = h & 0x7c007c00u;
                uint32_t keep = 0xffffffffu;
                if ((f & 0x7c00u) == 0x7c00u) keep &= 0xffff0000u;
                if ((f >> 16) == 0x7c00u) keep &= 0x0000ffffu;
                if (keep != 0xffffffffu) {
                  at[e] = h & keep;
                  odd = odd || row < live;
                }
              }
            }
          }
          fence_proxy_async_smem();
        }
        // The mark goes with the tile: this warp may be pieces ahead of the
        // products, so the issuing warp gathers the marks of a piece's tiles.
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) {
          ctl->tile_lost[s][ci] = odd ? (uint32_t)k + 1u : 0u;
          mbar_arrive(smem_u32(&ctl->v_ok[s]));
          if constexpr (kQ8) mbar_arrive(smem_u32(&ctl->raw_empty[1]));
        }
        ++n;
        k = nk;
        cls = ncls;
        nk = nnk;
        ncls = nncls;
      }
    }
  } else if (warp >= 4) {
    // ---------------- softmax warpgroups: warps 4-7 and 8-11, thread t of
    // warpgroup w owns row 128 w + t of the block (TMEM lane t).
    const int w = (warp - 4) >> 2;
    const int t = ((warp & 3) << 5) | lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + w * 128, tO = tmem + lane_off + 256 + w * 128;
    const int group = p.Hq / c.Hkv;
    int n = 0, mine = 0, piece = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, wait_bar(smem_u32(bar), par, abort_flag, status));
    };
    bool have = pieces.next(p, pl, it, k0, k1, u);
    while (ok && have) {
      hv.init(p, it);
      // ---- Q, where the heads of a group do not divide a half into whole tokens:
      // a half-warp a row, 16 bytes a lane; rows past the block's are zero. Every
      // product of the previous piece has completed (o_final).
      if (!q_boxes) {
        uint4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rr = 128 * w + (warp & 3) * 32 + 2 * i + (lane >> 4);
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (rr < it.rows) {
            int64_t tok;
            int h;
            row_place(p, it, rr, tok, h);
            v[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + tok * p.sq[0] + h * p.sq[1] +
                                                   (lane & 15) * 8);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = (warp & 3) * 32 + 2 * i + (lane >> 4);
          const uint32_t dst = kPQ + w * kPTileB + ((lane >> 3) & 1) * (kPTileB / 2) + sw128_offset(r, (lane & 7) * 16);
          *reinterpret_cast<uint4*>(smem + dst) = v[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full));
      }

      const int rr = 128 * w + t;
      const bool valid = rr < it.rows;
      const int pos = hv.L - it.s.n + (it.row0 + rr) / group;
      float m_run = -INFINITY, l_run = 0.f;
      int got = 0;
      uint32_t cls;
      for (int k = next_seen(it, hv, k0, k1, cls); k < k1; k = next_seen(it, hv, k + 1, k1, cls), ++n) {
        const uint32_t cl = (cls >> (2 * w)) & 3u;
        if (cl == 0u) continue;
        const int kt = it.tile_at(k), s = n % kPStages;
        if (!(ok = wait_all(&ctl->s_full[w], mine & 1))) break;
        tc_fence_after();
        const uint32_t bad = (ctl->tinfo[s] >> 8) & 0xffu;
        uint64_t w0 = ~0ull, w1 = ~0ull;
        const bool full = cl == 2u && bad == 0u;
        if (!full) row_bits(hv, pos, valid, kt, bad, box, w0, w1);
        float alpha;
        if constexpr (!kQ8) {
          const float sl2 = p.scale * kLog2e;
          alpha = full ? softmax_full_tile<kH, false, true>(tS, sl2, m_run, l_run, ~0ull, ~0ull)
                       : softmax_edge_tile<kH>(tS, sl2, w0, w1, m_run, l_run);
        } else {
          const float* sc = reinterpret_cast<const float*>(smem + M::kScale + s * 512);
          const float* t4 = ctl->ks_top[s];
          const float* l4 = ctl->ks_low[s];
          const float top = max3nan(max3nan(t4[0], t4[1], t4[2]), t4[3], t4[3]);
          const float low = min3nan(min3nan(l4[0], l4[1], l4[2]), l4[3], l4[3]);
          alpha = full ? softmax_scaled_tile<false>(tS, sc, ctl->v_exp[s], top, low, w0, w1, m_run, l_run)
                       : softmax_scaled_tile<true>(tS, sc, ctl->v_exp[s], top, low, w0, w1, m_run, l_run);
        }
        if (got > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            tmem_ld32(tO + ch * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + ch * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[w]));
        ++got;
        ++mine;
      }
      if (!ok) break;
      // The next piece, and its rows' Q into L2, while the last products run.
      Item nit;
      int nk0 = 0, nk1 = 0;
      int64_t nu = 0;
      have = pieces.next(p, pl, nit, nk0, nk1, nu);
      if (!q_boxes && have && 128 * w + t < nit.rows) {
        int64_t tok;
        int h;
        row_place(p, nit, 128 * w + t, tok, h);
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + tok * p.sq[0] + h * p.sq[1];
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
      }
      if (!(ok = wait_all(&ctl->o_final, piece & 1))) break;
      tc_fence_after();
      // ---- epilogue: the rows, or this piece's part of them
      const bool whole = k0 == 0 && k1 == it.tiles;
      const int lost0 = (int)*reinterpret_cast<volatile uint32_t*>(&ctl->lost_lo) - 1;  // -1: none
      const int lost1 = (int)*reinterpret_cast<volatile uint32_t*>(&ctl->lost_hi);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->o_read));
      int64_t tok;
      int h;
      row_place(p, it, valid ? rr : 0, tok, h);
      float lse = 0.f, osc = 1.f;
      if (whole) osc = finish_scale(p, h, m_run, l_run, lse);
      uint16_t* orow = static_cast<uint16_t*>(p.o) + tok * p.so[0] + h * p.so[1];
      float* slot = split_slot<kPRows, kPD>(SplitP{0, 0, nullptr, pl.part}, blockIdx.x, k0 == 0 ? 1 : 0);
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        LostColumns lost{0u, 0u, 0u};
        if (lost0 >= 0) lost = lost_columns<kH, kQ8>(p, it, hv, lost0, lost1, pos, valid, box, ch);
        if (whole && l_run == 0.f) lost = LostColumns{0u, 0u, 0u};  // an empty row (a part's: the join knows)
        uint32_t o[32];
        if (got > 0) {
          tmem_ld32(tO + ch * 32, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (got == 0 || l_run == 0.f) o[e] = 0u;
        if (lost.nan | lost.up | lost.down) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(o[e]);
            if ((lost.up >> e) & 1u) v += INFINITY;
            if ((lost.down >> e) & 1u) v -= INFINITY;
            o[e] = (lost.nan >> e) & 1u ? 0x7fffffffu : __float_as_uint(v);
          }
        }
        if (valid && whole) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pk[e] = pack16<kH>(__uint_as_float(o[c8 * 8 + 2 * e]) * osc, __uint_as_float(o[c8 * 8 + 2 * e + 1]) * osc);
            *reinterpret_cast<uint4*>(orow + ch * 32 + c8 * 8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else if (valid) {
#pragma unroll
          for (int c4 = 0; c4 < 8; ++c4)
            reinterpret_cast<uint4*>(slot)[(ch * 8 + c4) * kPRows + rr] =
                make_uint4(o[4 * c4], o[4 * c4 + 1], o[4 * c4 + 2], o[4 * c4 + 3]);
        }
      }
      if (valid && whole) p.lse[tok * p.sl[0] + h * p.sl[1]] = lse;
      if (!whole) {
        if (valid) {
          slot[kPRows * kPD + rr] = m_run;
          slot[kPRows * kPD + kPRows + rr] = l_run;
        }
        if (k0 == 0 && w == 0 && t == 0) {
          const int last = last_at_most(pl.starts, pieces.head.ranks, u + it.tiles - 1);
          const JoinRec rec{last - pieces.mine.rank + 1, it.s.q0, it.row0, it.rows, it.h, 0u, {0, 0}};
          pl.rec[pieces.mine.rank] = rec;
        }
      }
      tc_fence_before();
      ++piece;
      it = nit;
      k0 = nk0;
      k1 = nk1;
      u = nu;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The joins that the records ask for. A piece's rows lie four columns at a time
// ([32][256 rows] float4), as the row-per-thread epilogue writes them in whole
// lines; a warp joins 8 rows x 32 columns (lane: row lane % 8, columns
// 4 (lane / 8) and so on), and block (share, y) the rows 32 y .. of its record.
constexpr int kJoinBlockRows = 32;

template <bool kH>
__global__ void __launch_bounds__(512) chunk_join_kernel(const PagedP p, const PlanP pl) {
  wait_for_previous();
  const JoinRec rec = pl.rec[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * kJoinBlockRows + (warp >> 2) * 8 + (lane & 7);
  if (rec.parts == 0 || r - (lane & 7) >= rec.rows) return;
  const bool live = r < rec.rows;
  const int c4 = (warp & 3) * 8 + (lane >> 3);  // and c4 + 4
  auto at = [&](int i) {
    return split_slot<kPRows, kPD>(SplitP{0, 0, nullptr, pl.part}, pl.cta_of[blockIdx.x + i], i == 0 ? 1 : 0);
  };
  float M = -INFINITY, L = 0.f;
  float4 v[2];
  v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  // A running maximum over the pieces, four of them in flight.
  for (int i0 = 0; i0 < rec.parts; i0 += 4) {
    float m[4], l[4];
    float4 x[4][2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
      x[e][0] = x[e][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + e < rec.parts && live) {
        const float* s = at(i0 + e);
        m[e] = s[kPRows * kPD + r];
        l[e] = s[kPRows * kPD + kPRows + r];
        x[e][0] = reinterpret_cast<const float4*>(s)[c4 * kPRows + r];
        x[e][1] = reinterpret_cast<const float4*>(s)[(c4 + 4) * kPRows + r];
      }
    }
    const float top = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
    const float old = part_factor(M, top);
    L *= old;
#pragma unroll
    for (int a = 0; a < 2; ++a) v[a] = make_float4(v[a].x * old, v[a].y * old, v[a].z * old, v[a].w * old);
    M = top;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i0 + e >= rec.parts) break;
      const float f = part_factor(m[e], M);
      L += l[e] * f;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        v[a].x = fmaf(x[e][a].x, f, v[a].x);
        v[a].y = fmaf(x[e][a].y, f, v[a].y);
        v[a].z = fmaf(x[e][a].z, f, v[a].z);
        v[a].w = fmaf(x[e][a].w, f, v[a].w);
      }
    }
  }
  if (!live) return;
  Item it;
  it.s.q0 = rec.q0;
  it.row0 = rec.row0;
  it.h = rec.h;
  finish_four<kH>(p, it, r, c4, M, L, v[0]);
  finish_four<kH>(p, it, r, c4 + 4, M, L, v[1]);
}

// ----------------------------------------------------------- host helpers

PFN_cuTensorMapEncodeTiled_v12000 paged_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

// 4-D map over (d, position in page, head, page) with a (64 or 128, box, 1, 1)
// box of 128-byte rows, 128-byte swizzle.
bool pool_map(CUtensorMap* map, const void* base, const CacheP& c, const int64_t s[3], int box) {
  auto fn = paged_encode_fn();
  if (!fn) return false;
  const bool q8 = c.dtype == ATTN_E4M3;
  const cuuint64_t el = q8 ? 1 : 2;
  cuuint64_t dims[4] = {(cuuint64_t)kPD, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)s[1] * el, (cuuint64_t)s[2] * el, (cuuint64_t)s[0] * el};
  cuuint32_t bx[4] = {q8 ? 128u : 64u, (cuuint32_t)box, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  const auto type = q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                       : c.dtype == ATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, type, 4, const_cast<void*>(base), dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// 3-D map of Q over (d, head, token) with a (64, group, 128 / group) box.
bool q_map(CUtensorMap* map, const PagedP& p, int group) {
  auto fn = paged_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kPD, (cuuint64_t)p.Hq, (cuuint64_t)p.c.rows};
  cuuint64_t strides[2] = {(cuuint64_t)p.sq[1] * 2, (cuuint64_t)p.sq[0] * 2};
  cuuint32_t bx[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(map, p.dtype == ATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(p.q), dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys per copy box: the largest power of two up to 128 that divides the page.
int box_of(int page_size) {
  int b = 16;
  while (b < kPTile && page_size % (2 * b) == 0) b *= 2;
  return b;
}

struct PlanSizes {
  size_t head, cta, starts, cta_of, pair, prefix, first, rec, part, total;
  int cap;
};

PlanSizes plan_sizes(int64_t rows, int batch, int group) {
  PlanSizes z;
  const int tokens = kPRows / group, G = sm_count();
  z.cap = (int)(rows / tokens + batch);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 256);
    return a;
  };
  z.head = take(sizeof(PlanHead));
  z.cta = take(sizeof(PlanCta) * G);
  z.starts = take(sizeof(int64_t) * (G + 1));
  z.cta_of = take(sizeof(int32_t) * G);
  z.pair = take(sizeof(PlanPair) * z.cap);
  z.prefix = take(sizeof(int64_t) * (z.cap + 1));
  z.first = take(sizeof(int32_t) * (batch + 1));
  z.rec = take(sizeof(JoinRec) * G);
  z.part = take(sizeof(float) * split_part_floats<kPRows, kPD>() * 2 * G);
  z.total = at;
  return z;
}

template <bool kH, bool kQ8>
cudaError_t launch_chunk(const PagedP& p, const PlanP& pl, const CUtensorMap& mq, const CUtensorMap& mk,
                         const CUtensorMap& mv, int box, int q_boxes, cudaStream_t st) {
  using M = PagedSmem<kQ8>;
  auto kern = paged_chunk_kernel<kH, kQ8>;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)M::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  plan_kernel<<<1, kPlanThreads, 0, st>>>(p, pl);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // The chunk kernel's set-up runs under the plan; it waits for the plan's end
  // before it reads anything.
  if ((e = launch_after(kern, dim3(pl.ctas), M::kThreads, M::kBytes, st, mq, mk, mv, p, pl, box,
                        q_boxes)) != cudaSuccess) return e;
  return launch_after(chunk_join_kernel<kH>, dim3(pl.ctas, kPRows / kJoinBlockRows), 512, 0, st, p, pl);
}

}  // namespace

bool paged_chunk_supported(const PagedP& p) {
  if (!paged_pieces_ok(p) || p.Hq / p.c.Hkv > kPRows || sm_count() > kPlanThreads || !paged_encode_fn()) return false;
  const CacheP& c = p.c;
  // What a tensor map can describe: positive strides below 2^40 bytes.
  for (int i = 0; i < 3; ++i)
    if (c.sk[i] < 1 || c.sv[i] < 1 || c.sk[i] >= (1LL << 38) || c.sv[i] >= (1LL << 38)) return false;
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  return major == 10 && minor == 0;
}

size_t paged_chunk_workspace_bytes(int64_t rows, int batch, int group) {
  return group > kPRows ? 0 : plan_sizes(rows, batch, group).total;
}

cudaError_t launch_paged_chunk(const PagedP& p, void* ws, cudaStream_t st) {
  const CacheP& c = p.c;
  const PlanSizes z = plan_sizes(c.rows, c.batch, p.Hq / c.Hkv);
  char* w = static_cast<char*>(ws);
  PlanP pl;
  pl.head = reinterpret_cast<PlanHead*>(w + z.head);
  pl.cta = reinterpret_cast<PlanCta*>(w + z.cta);
  pl.starts = reinterpret_cast<int64_t*>(w + z.starts);
  pl.cta_of = reinterpret_cast<int32_t*>(w + z.cta_of);
  pl.pair = reinterpret_cast<PlanPair*>(w + z.pair);
  pl.prefix = reinterpret_cast<int64_t*>(w + z.prefix);
  pl.first = reinterpret_cast<int32_t*>(w + z.first);
  pl.rec = reinterpret_cast<JoinRec*>(w + z.rec);
  pl.part = reinterpret_cast<float*>(w + z.part);
  pl.ctas = sm_count();
  pl.cap = z.cap;
  pl.tokens = kPRows / (p.Hq / c.Hkv);
  const int box = box_of(c.page_size);
  // A copy box holds whole tokens of a group where the group divides a half.
  const int group = p.Hq / c.Hkv;
  const int q_boxes = 128 % group == 0 && p.sq[0] > 0 && p.sq[1] > 0 && p.sq[0] < (1LL << 38) && p.sq[1] < (1LL << 38);
  CUtensorMap mq = {}, mk, mv;
  if (q_boxes && !q_map(&mq, p, group)) return cudaErrorInvalidValue;
  if (!pool_map(&mk, c.k, c, c.sk, box) || !pool_map(&mv, c.v, c, c.sv, box)) return cudaErrorInvalidValue;
  const bool h = p.dtype == ATTN_F16;
  if (c.dtype == ATTN_E4M3)
    return h ? launch_chunk<true, true>(p, pl, mq, mk, mv, box, q_boxes, st)
             : launch_chunk<false, true>(p, pl, mq, mk, mv, box, q_boxes, st);
  return h ? launch_chunk<true, false>(p, pl, mq, mk, mv, box, q_boxes, st)
           : launch_chunk<false, false>(p, pl, mq, mk, mv, box, q_boxes, st);
}

}  // namespace attn
