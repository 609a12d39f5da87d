// How the paged kernels share their work: an item is (sequence, K/V head,
// block of query rows), its cost the number of key tiles it walks, and the
// tiles of all items, in order, are dealt to the CTAs of one wave in equal
// consecutive shares. Lengths are read on the device, so a captured call
// serves whatever lengths it meets, and every SM gets the same number of tiles
// whether the batch holds one long sequence or many ragged ones. (The lengths
// must not change meanwhile; if they do, the readings disagree and the results
// mean nothing, but every index stays within its range.) An item
// whose tiles fall to several CTAs leaves one partial result (running maximum,
// sum and unnormalised rows, fp32) per CTA in the workspace, and the CTA that
// begins it a record of what is to be joined; a second, small kernel joins
// them in the CTAs' order, so the result is the same every time, and no CTA
// waits for another. (Joined by the last CTA to finish, in the same kernel,
// the join's registers cost the main loops more than the second launch does:
// 223 against 178 us for 64 e4m3 sequences of up to 8192 keys.)
#pragma once

#include <math.h>

#include "paged.cuh"

namespace attn {

// What a CTA leaves for the join: the item that it begins and others finish
// (parts 0: none), and its error bits.
struct JoinRec {
  int32_t parts, q0, row0, rows, h;
  uint32_t errors;
  int32_t pad[2];
};

struct SplitP {
  int32_t ctas;        // grid size
  int32_t min_tiles;   // least tiles a CTA takes before another one is given work
  JoinRec* rec;        // [ctas]
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
  uint32_t errors;
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

// The key tiles that some new token of sequence b (whose view s is) sees, and
// its row blocks. One tile at least, so that a sequence without keys still gets
// its rows written.
template <int kTile, int kRows>
__device__ __forceinline__ Item seq_tiles(const PagedP& p, int b, const SeqView& s) {
  Item it;
  it.b = b;
  it.s = s;
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
    const Item it = seq_tiles<kTile, kRows>(p, b, seq_view(p.c, b));
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
  if (threadIdx.x == 0) {
    ss.b = 0;
    ss.rem = 0;
  }
  __syncthreads();
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
  const int tiles = seq_tiles<kTile, kRows>(p, sh.b, warp_seq_view(p.c, sh.b)).tiles;
  sh.sub = (int)(ss.rem / tiles);
  sh.at = ss.rem % tiles;
  return sh;
}

template <int kTile, int kRows>
__device__ __forceinline__ Item split_item(const PagedP& p, Share& sh) {
  Item it = seq_tiles<kTile, kRows>(p, sh.b, warp_seq_view(p.c, sh.b));
  if (it.blocks < 1) it.blocks = 1;  // (only with lengths that change)
  if (sh.at >= it.tiles) sh.at = it.tiles - 1;
  it.h = sh.sub / it.blocks;  // the row blocks of a head follow one another: its keys are in L2 by then
  if (it.h >= p.c.Hkv) it.h = p.c.Hkv - 1;
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
    while (sh.b < p.c.batch && warp_seq_view(p.c, sh.b).n == 0);
    if (sh.b >= p.c.batch) sh.left = 0;
  }
}

__device__ __forceinline__ int split_owner(const Share& sh, int64_t u) {
  const int64_t o = ((u + 1) * sh.ctas - 1) / sh.total;
  return o < sh.ctas ? (int)o : sh.ctas - 1;
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

// Joins a CTA's own partial results for tiles [k0, k1) of the item and writes
// the rows, or its piece of them. All threads.
template <int kRows, int kD, bool kHalf, class Part, class Vec>
__device__ __forceinline__ void split_finish(const PagedP& p, const SplitP& sp, const Share& sh, const Item& it, int k0,
                                             int k1, int parts, Part part, Vec vec) {
  if (k0 == 0 && k1 == it.tiles) {
    join_parts<kD>(threadIdx.x, blockDim.x, it.rows, parts, part, vec,
                   [&](int r, int c4, float M, float l, const float4& v) { finish_four<kHalf>(p, it, r, c4, M, l, v); });
    return;
  }
  float* slot = split_slot<kRows, kD>(sp, blockIdx.x, k0 == 0 ? 1 : 0);
  join_parts<kD>(threadIdx.x, blockDim.x, it.rows, parts, part, vec,
                 [&](int r, int c4, float M, float l, const float4& v) {
                   reinterpret_cast<float4*>(slot)[r * (kD / 4) + c4] = v;
                   if (c4 == 0) {
                     slot[kRows * kD + r] = M;
                     slot[kRows * kD + kRows + r] = l;
                   }
                 });
  if (k0 == 0 && threadIdx.x == 0) {
    JoinRec rec{split_owner(sh, sh.u + it.tiles - 1) - (int)blockIdx.x + 1, it.s.q0, it.row0, it.rows, it.h, 0u, {0, 0}};
    sp.rec[blockIdx.x] = rec;
  }
}

// A kernel that the next one may follow into the machine early, and that one's
// wait for its end (programmatic dependent launch).
__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The joins that the records ask for: block (i, y) takes rows y kJoinRows ..
// of CTA i's record, a warp a row: a lane per piece for the summaries, then a
// lane per four columns with eight pieces' loads in flight. slot(i, e): the e-th
// piece of CTA i's item. Block (0, 0) also gathers the CTAs' error bits.
constexpr int kJoinRows = 8;

template <int kRows, int kD, bool kHalf, class Slot>
__device__ __forceinline__ void join_record(const PagedP& p, const JoinRec* recs, int ctas, bool gather, Slot slot) {
  static_assert(kD == 128, "a lane per four columns");
  const int lane = threadIdx.x & 31;
  if (gather && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
    uint32_t bits = 0;
    for (int i = lane; i < ctas; i += 32) bits |= recs[i].errors;
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) *p.c.status = bits;
  }
  const JoinRec rec = recs[blockIdx.x];
  const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5), parts = rec.parts;
  if (parts == 0 || r >= rec.rows) return;
  Item it;
  it.s.q0 = rec.q0;
  it.row0 = rec.row0;
  it.h = rec.h;
  float M = -INFINITY, L = 0.f;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, slot(blockIdx.x, i)[kRows * kD + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float f = 0.f;
    if (i0 + lane < parts) {
      const float* x = slot(blockIdx.x, i0 + lane) + kRows * kD + r;
      f = part_factor(x[0], M);
      L += x[kRows] * f;
    }
    const int n = parts - i0 < 32 ? parts - i0 : 32;
    for (int i = 0; i < n; i += 8) {
      float4 x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) x[e] = reinterpret_cast<const float4*>(slot(blockIdx.x, i0 + i + e) + r * kD)[lane];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = __shfl_sync(0xffffffffu, f, (i + e) & 31);
        if (i + e < n) {
          v.x = fmaf(x[e].x, g, v.x);
          v.y = fmaf(x[e].y, g, v.y);
          v.z = fmaf(x[e].z, g, v.z);
          v.w = fmaf(x[e].w, g, v.w);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  finish_four<kHalf>(p, it, r, lane, M, L, v);
}

// Launches `kern` so that it may enter the machine while the kernel before it
// in the stream still runs; it must wait_for_previous before it reads.
template <class Kern, class... Args>
cudaError_t launch_after(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace attn
