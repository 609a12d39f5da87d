// How the paged kernels share their work: an item is (sequence, K/V head,
// block of query rows), its cost the number of key tiles it walks, and the
// tiles of all items, in order, are dealt to the CTAs of one wave in equal
// consecutive shares. Lengths are read on the device, so a captured call
// serves whatever lengths it meets, and every SM gets the same number of tiles
// whether the batch holds one long sequence or many ragged ones. An item
// whose tiles fall to several CTAs leaves one partial result (running maximum,
// sum and unnormalised rows, fp32) per CTA in the workspace; the CTA that
// finishes last joins them in the CTAs' order, so the result is the same
// every time. No CTA waits for another.
#pragma once

#include <math.h>

#include "paged.cuh"

namespace attn {

struct SplitP {
  int32_t ctas;        // grid size
  int32_t min_tiles;   // least tiles a CTA takes before another one is given work
  uint32_t* counters;  // [ctas], zeroed before the launch
  float* part;         // [ctas][2]: slot 0 a piece that begins inside an item, slot 1 one that begins it
};

template <int kRows, int kD>
__host__ __device__ constexpr size_t split_part_floats() {
  return (size_t)kRows * kD + 2 * kRows;  // rows, then m, then l
}

struct SplitShared {
  int64_t sums[32];
  int64_t rem;
  int b;
  int last;
};

// A CTA's share: `left` tiles from tile `at` of item `sub` of sequence b on.
struct Share {
  int64_t left, at, u;  // u: index of the current tile among all of them
  int64_t total;
  int b, sub, ctas;
};

struct Item {
  SeqView s;
  int b, h, row0, rows;   // rows row0 .. row0 + rows - 1 of the sequence's n * group
  int nf, lo, hi;         // key tiles [0, nf) and [max(lo, nf), hi)
  int tiles, blocks;
  // The item's k-th key tile.
  __device__ __forceinline__ int tile_at(int k) const { return k < nf ? k : k - nf + (lo > nf ? lo : nf); }
};

// The key tiles that some new token of sequence b sees, and its row blocks.
// One tile at least, so that a sequence without keys still gets its rows
// written.
template <int kTile, int kRows>
__device__ __forceinline__ Item seq_tiles(const PagedP& p, int b) {
  Item it;
  it.b = b;
  it.s = seq_view(p.c, b);
  const int64_t L = it.s.L;
  it.hi = (int)((L + kTile - 1) / kTile);
  it.lo = it.nf = 0;
  if (p.flags & ATTN_MASK_WINDOW) {
    const int64_t lo = L - it.s.n - p.window + 1;
    it.lo = lo > 0 ? (int)(lo / kTile) : 0;
    const int64_t f = p.first < L ? p.first : L;
    it.nf = (int)((f + kTile - 1) / kTile);
  }
  const int from = it.lo > it.nf ? it.lo : it.nf;
  it.tiles = it.nf + (it.hi > from ? it.hi - from : 0);
  if (it.tiles < 1) it.tiles = 1;
  it.blocks = (int)(((int64_t)it.s.n * (p.Hq / p.c.Hkv) + kRows - 1) / kRows);
  return it;
}

__device__ __forceinline__ int64_t block_sum_scan(int64_t x, SplitShared& ss, int64_t& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) ss.sums[warp] = incl;
  __syncthreads();
  int64_t total = 0, base = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) base = total;
    total += ss.sums[w];
  }
  before = base + incl - x;
  return total;
}

// The calling CTA's share (all threads of the block).
template <int kTile, int kRows>
__device__ __forceinline__ Share split_share(const PagedP& p, const SplitP& sp, SplitShared& ss) {
  const int B = p.c.batch;
  auto units = [&](int b) {
    if (b >= B) return (int64_t)0;
    const Item it = seq_tiles<kTile, kRows>(p, b);
    return (int64_t)it.tiles * it.blocks * p.c.Hkv;
  };
  int64_t before, total = 0, mine = 0;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    mine = units(b0 + threadIdx.x);
    total += block_sum_scan(mine, ss, before);
  }
  Share sh;
  sh.total = total;
  int64_t ctas = (total + sp.min_tiles - 1) / sp.min_tiles;
  ctas = ctas < 1 ? 1 : (ctas > sp.ctas ? sp.ctas : ctas);
  sh.ctas = (int)ctas;
  const int me = blockIdx.x;
  if (me >= ctas || !total) {
    sh.left = sh.at = sh.u = 0;
    sh.b = sh.sub = 0;
    return sh;
  }
  sh.u = me * total / ctas;
  sh.left = (me + 1) * total / ctas - sh.u;
  int64_t base = 0;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    if (B > blockDim.x) {
      mine = units(b0 + threadIdx.x);
      const int64_t sum = block_sum_scan(mine, ss, before);
      before += base;
      base += sum;
    }
    if (before <= sh.u && sh.u < before + mine) {
      ss.b = b0 + threadIdx.x;
      ss.rem = sh.u - before;
    }
  }
  __syncthreads();
  sh.b = ss.b;
  const int tiles = seq_tiles<kTile, kRows>(p, sh.b).tiles;
  sh.sub = (int)(ss.rem / tiles);
  sh.at = ss.rem % tiles;
  return sh;
}

template <int kTile, int kRows>
__device__ __forceinline__ Item split_item(const PagedP& p, const Share& sh) {
  Item it = seq_tiles<kTile, kRows>(p, sh.b);
  it.h = sh.sub / it.blocks;  // the row blocks of a head follow one another: its keys are in L2 by then
  it.row0 = (sh.sub % it.blocks) * kRows;
  const int all = it.s.n * (p.Hq / p.c.Hkv);
  it.rows = all - it.row0 < kRows ? all - it.row0 : kRows;
  return it;
}

template <int kTile, int kRows>
__device__ __forceinline__ void split_advance(const PagedP& p, Share& sh, const Item& it, int done) {
  sh.left -= done;
  sh.u += done;
  sh.at += done;
  if (sh.at < it.tiles) return;
  sh.at = 0;
  if (++sh.sub < it.blocks * p.c.Hkv) return;
  sh.sub = 0;
  if (sh.left > 0) {  // then a later sequence has rows
    do ++sh.b;
    while (seq_view(p.c, sh.b).n == 0);
  }
}

__device__ __forceinline__ int split_owner(const Share& sh, int64_t u) {
  return (int)(((u + 1) * sh.ctas - 1) / sh.total);
}

// One row's finish: the factor that turns the unnormalised row into the
// output, and the LSE to store. m in base 2; l is 0 exactly when no key had a
// share (a NaN score makes it NaN, and the row with it).
__device__ __forceinline__ float finish_scale(const PagedP& p, int h, float m, float l, float& lse) {
  const bool has_sink = p.sink != nullptr;
  const float z2 = has_sink ? p.sink[h] * 1.4426950408889634f : -INFINITY;
  float osc, lse2;
  if (l == 0.f) {
    lse2 = z2;
    osc = 0.f;
    m = -INFINITY;
  } else {
    if (m == -INFINITY) m = 0.f;  // only with l NaN
    const float M = fmaxf(m, z2);
    const float up = exp2f(m - M);
    const float tot = l * up + (has_sink ? exp2f(z2 - M) : 0.f);
    osc = up / tot;
    lse2 = M + log2f(tot);
  }
  lse = stored_lse_log2(p.lse_fmt, lse2, m, l);
  return osc;
}

// Where row r of the item goes: its token's row and its query head.
__device__ __forceinline__ void row_place(const PagedP& p, const Item& it, int r, int64_t& t, int& h) {
  const int group = p.Hq / p.c.Hkv, rr = it.row0 + r;
  t = it.s.q0 + rr / group;
  h = it.h * group + rr % group;
}

// Four consecutive output elements of row r (and, with the first ones, the LSE).
template <bool kHalf>
__device__ __forceinline__ void finish_four(const PagedP& p, const Item& it, int r, int c4, float m, float l,
                                            const float4& v) {
  int64_t t;
  int h;
  row_place(p, it, r, t, h);
  float lse;
  const float f = finish_scale(p, h, m, l, lse);
  uint2 w = make_uint2(0u, 0u);
  if (f != 0.f) {
    if constexpr (kHalf) {
      const __half2 a = __floats2half2_rn(v.x * f, v.y * f), b = __floats2half2_rn(v.z * f, v.w * f);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f), b = __floats2bfloat162_rn(v.z * f, v.w * f);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + t * p.so[0] + h * p.so[1] + 4 * c4) = w;
  if (c4 == 0) p.lse[t * p.sl[0] + h * p.sl[1]] = lse;
}

// The factor of a part with maximum m in a sum whose maximum is M.
__device__ __forceinline__ float part_factor(float m, float M) { return m == M ? 1.f : exp2f(m - M); }

// Joins `parts` results: part(i, r, m, l) and vec(i, r, c4) give the i-th one's
// summary and four elements; put(r, c4, M, l, v) takes the sum. By `threads`
// threads, of which the caller is number tid.
template <int kD, class Part, class Vec, class Put>
__device__ __forceinline__ void join_parts(int tid, int threads, int rows, int parts, Part part, Vec vec, Put put) {
  for (int e = tid; e < rows * (kD / 4); e += threads) {
    const int r = e / (kD / 4), c4 = e % (kD / 4);
    float M = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      float m, l;
      part(i, r, m, l);
      M = fmaxf(M, m);
    }
    float L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      float m, l;
      part(i, r, m, l);
      const float f = part_factor(m, M);
      const float4 x = vec(i, r, c4);
      L += l * f;
      v.x = fmaf(x.x, f, v.x);
      v.y = fmaf(x.y, f, v.y);
      v.z = fmaf(x.z, f, v.z);
      v.w = fmaf(x.w, f, v.w);
    }
    put(r, c4, M, L, v);
  }
}

template <int kRows, int kD>
__device__ __forceinline__ float* split_slot(const SplitP& sp, int cta, int slot) {
  return sp.part + ((size_t)cta * 2 + slot) * split_part_floats<kRows, kD>();
}

// After this CTA's piece of an item that it does not cover alone lies in its
// slot (slot 1 when the piece begins the item, else 0): counts it, and, as the
// last, joins all pieces and writes the rows. All threads.
template <int kRows, int kD, bool kHalf>
__device__ __forceinline__ void split_join(const PagedP& p, const SplitP& sp, SplitShared& ss, const Share& sh,
                                           const Item& it, int k0) {
  const int64_t first = sh.u - k0;  // the item's first tile
  const int c0 = split_owner(sh, first), c1 = split_owner(sh, first + it.tiles - 1);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) ss.last = atomicAdd(sp.counters + c0, 1u) == (uint32_t)(c1 - c0);
  __syncthreads();
  if (!ss.last) return;
  __threadfence();
  auto at = [&](int i) { return split_slot<kRows, kD>(sp, c0 + i, i == 0 ? 1 : 0); };
  join_parts<kD>(
      threadIdx.x, blockDim.x, it.rows, c1 - c0 + 1,
      [&](int i, int r, float& m, float& l) {
        const float* x = at(i) + kRows * kD;
        m = __ldcg(x + r);
        l = __ldcg(x + kRows + r);
      },
      [&](int i, int r, int c4) { return __ldcg(reinterpret_cast<const float4*>(at(i)) + r * (kD / 4) + c4); },
      [&](int r, int c4, float M, float l, const float4& v) { finish_four<kHalf>(p, it, r, c4, M, l, v); });
}

// Joins a CTA's own partial results for tiles [k0, k1) of the item and writes
// the rows, or its piece of them. All threads.
template <int kRows, int kD, bool kHalf, class Part, class Vec>
__device__ __forceinline__ void split_finish(const PagedP& p, const SplitP& sp, SplitShared& ss, const Share& sh,
                                             const Item& it, int k0, int k1, int parts, Part part, Vec vec) {
  if (k0 == 0 && k1 == it.tiles) {
    join_parts<kD>(threadIdx.x, blockDim.x, it.rows, parts, part, vec, [&](int r, int c4, float M, float l, const float4& v) {
      finish_four<kHalf>(p, it, r, c4, M, l, v);
    });
    return;
  }
  float* slot = split_slot<kRows, kD>(sp, blockIdx.x, k0 == 0 ? 1 : 0);
  join_parts<kD>(threadIdx.x, blockDim.x, it.rows, parts, part, vec, [&](int r, int c4, float M, float l, const float4& v) {
    __stcg(reinterpret_cast<float4*>(slot) + r * (kD / 4) + c4, v);
    if (c4 == 0) {
      slot[kRows * kD + r] = M;
      slot[kRows * kD + kRows + r] = l;
    }
  });
  split_join<kRows, kD, kHalf>(p, sp, ss, sh, it, k0);
}

}  // namespace attn
