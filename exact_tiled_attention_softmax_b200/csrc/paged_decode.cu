// Attention over a paged cache for few new tokens per sequence (at most 16
// (token, head of the group) rows per K/V head): 16-bit or e4m3 cache, d = dv =
// 128, pages of a multiple of 16 positions.
//
// The arithmetic is 4 flops per cached element and row, so with up to 16 rows
// the cache's bytes bound it, and what matters is to keep enough of them in
// flight. Every warp streams 16-key pieces of its own through a private ring
// of asynchronous copies (no barrier between warps until an item ends) and
// multiplies them with m16n8k16 matrix instructions: S = Q K^T with the rows
// as the 16-row operand, the running maximum and sum in registers, O += P V
// with P straight from the score fragments.
//
// Work split: an item is (sequence, 16-row block, K/V head); its keys are cut
// into 64-key tiles (one 16-key piece per warp) and all tiles of all items,
// in order, are dealt to the CTAs in equal consecutive shares, so the load is
// even whatever the lengths are and the grid needs no length from the host. An
// item that several CTAs share is joined by the last of them to finish, in
// the CTAs' order, so the result does not depend on timing.
#include <math.h>

#include "paged.cuh"
#include "paged_split.cuh"
#include "sm100_paged.h"
#include "sm100_ptx.cuh"

namespace attn {

using namespace sm100;

namespace {

constexpr int kDD = 128;          // head width
constexpr int kRows = 16;         // query rows per item
constexpr int kDWarps = 4;
constexpr int kDThreads = kDWarps * 32;
constexpr int kPiece = 16;        // keys per warp and tile
constexpr int kDTile = kDWarps * kPiece;
constexpr float kLog2eD = 1.4426950408889634f;
constexpr int kMinTiles = 2;      // key tiles a CTA takes at least
constexpr float kRescaleD = 8.f;  // move the running maximum only past 2^8

enum { kBf16 = 0, kF16 = 1, kE4m3Bf16 = 2, kE4m3F16 = 3 };  // cache type (and query type)

template <int kMode>
struct Ring {
  static constexpr bool kQ8 = kMode >= kE4m3Bf16;
  static constexpr int kRowBytes = kQ8 ? kDD : 2 * kDD;
  static constexpr int kTileB = kPiece * kRowBytes;            // one of K, V
  static constexpr int kStageB = 2 * kTileB + (kQ8 ? 128 : 0); // + 16 K scales, 16 V scales
  static constexpr int kStages = kQ8 ? 6 : 3;
  static constexpr int kWarpB = kStages * kStageB;
  static constexpr int kSmem = kDWarps * kWarpB;
  static_assert(kWarpB >= kRows * kDD * 4 + 2 * kRows * 4, "the ring also carries a warp's result to the join");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Copies of 16 (4) bytes, or that many zeros when !live (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}

// Two e4m3 codes (the low 16 bits) as packed fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
// The same as packed bf16, exact too (fp16 holds every e4m3 value, bf16 as well).
__device__ __forceinline__ uint32_t e4m3x2_bf16(uint32_t v) {
  const float2 f = unpack16<true>(e4m3x2_f16(v));
  return pack_bf16(f.x, f.y);
}

// Does a word of stored values (two of 16 bits with the exponent mask expo, or
// four e4m3 codes) hold an infinity or a NaN?
__device__ __forceinline__ bool nonfinite16(uint32_t v, uint32_t expo) {
  return (v & expo) == expo || ((v >> 16) & expo) == expo;
}
__device__ __forceinline__ bool nan_e4m3(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// The running summary of the calling thread's two rows (lane / 4 and + 8).
struct Rows2 {
  float m[2], l[2];
};

template <int kMode>
__global__ void __launch_bounds__(kDThreads, 2) paged_decode_kernel(const PagedP p, const SplitP sp) {
  using R = Ring<kMode>;
  constexpr bool kQ8 = R::kQ8;
  constexpr bool kHalfS = kMode != kBf16;   // Q K^T in fp16 (an e4m3 K is exact in it)
  constexpr bool kHalfP = kMode == kF16;    // P V in fp16, else bf16
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SplitShared ss;
  const CacheP& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3, g8 = lane >> 2;
  const uint32_t ring = smem_u32(smem) + warp * R::kWarpB;
  if (blockIdx.x == 0) report_ragged(c);
  const int group = p.Hq / c.Hkv;

  Share share = split_share<kDTile, kRows>(p, sp, ss);
  while (share.left > 0) {
    const Item it = split_item<kDTile, kRows>(p, share);
    const int k0 = (int)share.at, k1 = (int)(it.tiles - k0 < share.left ? it.tiles : k0 + share.left);
    const int rows = it.rows;
    const int64_t row_pos0 = it.s.L - it.s.n;  // key position of the sequence's first new token
    const bool causal = p.flags & ATTN_MASK_CAUSAL, window = p.flags & ATTN_MASK_WINDOW;

    // ---- the loads of one 16-key piece (tile k of the item) into stage s
    int pg_base = k0 - 32;  // lane l holds the page of tile pg_base + l
    int pg_mine = -1;
    const int tok_lo = it.row0 / group, tok_hi = (it.row0 + rows - 1) / group;
    const int64_t p_lo = row_pos0 + tok_lo, p_hi = row_pos0 + tok_hi;  // positions of the block's first and last token
    const uint8_t* kb = static_cast<const uint8_t*>(c.k);
    const uint8_t* vb = static_cast<const uint8_t*>(c.v);
    constexpr int kChunks = R::kRowBytes / 16;      // 16-byte chunks of a row
    constexpr int kRowsAt = 32 / kChunks;           // rows a warp covers per copy instruction
    const int cr = lane / kChunks, cc = lane % kChunks;
    constexpr int kEl = kQ8 ? 1 : 2;
    const int64_t ko = ((int64_t)it.h * c.sk[2] + cr * c.sk[1]) * kEl + cc * 16;
    const int64_t vo = ((int64_t)it.h * c.sv[2] + cr * c.sv[1]) * kEl + cc * 16;
    auto seen_by_any = [&](int64_t j) {
      if (j >= it.s.L || (causal && j > p_hi)) return false;
      return !window || j < p.first || j > p_lo - p.window;
    };
    uint32_t dead = 0;  // bit s: stage s holds a piece that no row sees, or whose page is bad
    auto fetch = [&](int k) {
      if (k < k1) {
        if (k - pg_base >= 32) {
          pg_base = k;
          const int64_t j = (int64_t)it.tile_at(k + lane) * kDTile + warp * kPiece;
          pg_mine = -1;
          if (k + lane < k1 && j < it.s.L) pg_mine = (int)page_of(c, it.b, j);
        }
        const int pg = __shfl_sync(0xffffffffu, pg_mine, k - pg_base);
        const int64_t j0 = (int64_t)it.tile_at(k) * kDTile + warp * kPiece;
        const int stage = (k - k0) % R::kStages;
        const bool live = pg >= 0 && (!causal || j0 <= p_hi) &&
                          (!window || j0 < p.first || j0 + kPiece - 1 > p_lo - p.window);
        dead = live ? dead & ~(1u << stage) : dead | 1u << stage;
        if (live) {
          const uint32_t st = ring + stage * R::kStageB;
          const int64_t off = j0 % c.page_size;
          const uint8_t* ks = kb + (pg * c.sk[0] + off * c.sk[1]) * kEl + ko;
          const uint8_t* vs = vb + (pg * c.sv[0] + off * c.sv[1]) * kEl + vo;
#pragma unroll
          for (int i = 0; i < kPiece / kRowsAt; ++i) {
            const int r = cr + i * kRowsAt;
            const bool take = seen_by_any(j0 + r);
            // 16-bit rows: the 16-byte chunk index is permuted by the row so
            // that ldmatrix reads eight rows without bank conflicts; e4m3
            // rows: odd rows swap the halves of their eight chunks (each
            // thread reads whole chunks of one row there).
            const int pc = kQ8 ? cc ^ ((r & 1) << 2) : cc ^ (r & 7);
            cp16(st + r * R::kRowBytes + pc * 16, ks + (int64_t)i * kRowsAt * c.sk[1] * kEl, take);
            cp16(st + R::kTileB + r * R::kRowBytes + pc * 16, vs + (int64_t)i * kRowsAt * c.sv[1] * kEl, take);
          }
          if constexpr (kQ8) {
            const int r = lane & 15;
            const float* sc = lane < 16 ? c.ks + pg * c.sks[0] + (off + r) * c.sks[1] + (int64_t)it.h * c.sks[2]
                                        : c.vs + pg * c.svs[0] + (off + r) * c.svs[1] + (int64_t)it.h * c.svs[2];
            cp4(st + 2 * R::kTileB + lane * 4, sc, seen_by_any(j0 + r));
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int k = k0; k < k0 + R::kStages - 1; ++k) fetch(k);

    // ---- Q as A fragments (rows past the block's are zero)
    uint32_t qa[8][4];
    float xs[2];  // score factor of the thread's two rows: c log2(e), over the row's power of two
    {
      const uint16_t* qb = static_cast<const uint16_t*>(p.q);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g8 + 8 * e, rr = it.row0 + r;
        const bool live = r < rows;
        const uint16_t* qr = qb + (it.s.q0 + rr / group) * p.sq[0] + (int64_t)(it.h * group + rr % group) * p.sq[1];
        xs[e] = p.scale * kLog2eD;
        if constexpr (!kQ8) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            qa[ks][e] = live ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t4) : 0u;
            qa[ks][e + 2] = live ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8 + 2 * t4) : 0u;
          }
        } else {
          // The sum over d may take d in any order: step ks, thread t4 takes the
          // four elements from 16 (t4 + 4 (ks / 4)) + 4 (ks % 4), for which an
          // e4m3 row's thread reads whole 16-byte chunks.
          float top = 0.f;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint2 u = live ? *reinterpret_cast<const uint2*>(qr + 16 * (t4 + 4 * (ks >> 2)) + 4 * (ks & 3))
                                 : make_uint2(0u, 0u);
            qa[ks][e] = u.x;
            qa[ks][e + 2] = u.y;
            if constexpr (kMode == kE4m3Bf16) {
              const float2 a = unpack16<false>(u.x), b = unpack16<false>(u.y);
              top = fmaxf(fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
            }
          }
          if constexpr (kMode == kE4m3Bf16) {
            // A bf16 row goes to fp16 times the power of two that puts its
            // largest element in [2^13, 2^14): exact but for elements more than
            // 2^27 below the largest, whose absolute error is at most 2^-25
            // of fp16's unit, 2^-38 of the largest.
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = (int)((__float_as_uint(top) >> 23) & 0xffu) - 127;
            ex = top == 0.f || ex == 128 ? 13 : (ex < -100 ? -100 : ex);
            const float up = __uint_as_float((uint32_t)(13 - ex + 127) << 23);    // 2^(13 - ex), ex in [-100, 127]
            xs[e] *= __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const float2 a = unpack16<false>(qa[ks][e + i]);
                qa[ks][e + i] = pack_fp16(a.x * up, a.y * up);
              }
          }
        }
      }
    }
    int64_t pos[2];  // key positions of the thread's rows
#pragma unroll
    for (int e = 0; e < 2; ++e) pos[e] = row_pos0 + (it.row0 + g8 + 8 * e) / group;

    float acc[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    Rows2 rs{{-INFINITY, -INFINITY}, {0.f, 0.f}};

#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      cp_async_wait<R::kStages - 2>();
      __syncwarp();
      const int64_t j0 = (int64_t)it.tile_at(k) * kDTile + warp * kPiece;
      const uint32_t st = ring + (k - k0) % R::kStages * R::kStageB;
      if (!((dead >> (k - k0) % R::kStages) & 1u)) {
        // ---- S = Q K^T: two 8-key tiles, even and odd steps summed apart
        float s[2][4], s2[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
        if constexpr (!kQ8) {
          const int r = (lane & 7) + ((lane >> 4) << 3), hc = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t b[4];
            ldsm4(st + r * R::kRowBytes + (((2 * ks + hc) ^ (r & 7)) << 4), b);
            mma16816<kHalfS>(ks & 1 ? s2[0] : s[0], qa[ks], b[0], b[1]);
            mma16816<kHalfS>(ks & 1 ? s2[1] : s[1], qa[ks], b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = g8 + 8 * n;
              const uint4 u = lds128(st + r * R::kRowBytes + (((t4 + 4 * i) ^ ((r & 1) << 2)) << 4));
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mma16816<kHalfS>(q & 1 ? s2[n] : s[n], qa[4 * i + q], e4m3x2_f16(w[q]), e4m3x2_f16(w[q] >> 16));
            }
        }
        // ---- scale, mask, running summary. Fragment element e of n-tile n:
        // row g8 + 8 (e >> 1), key j0 + 8 n + 2 t4 + (e & 1).
        float vsc[2][2];
        uint32_t out = 0;  // bit 4 n + e: masked
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kc = 8 * n + 2 * t4 + (e & 1);
            float x = (s[n][e] + s2[n][e]) * xs[e >> 1];
            if constexpr (kQ8) {
              x *= lds32(st + 2 * R::kTileB + kc * 4);
              if (e < 2) vsc[n][e] = lds32(st + 2 * R::kTileB + 64 + kc * 4);
            }
            const int64_t j = j0 + kc;
            bool ok = j < it.s.L && g8 + 8 * (e >> 1) < rows && pos[e >> 1] >= 0;
            if (causal) ok = ok && j <= pos[e >> 1];
            if (window) ok = ok && (j > pos[e >> 1] - p.window || j < p.first);
            s[n][e] = ok ? x : -INFINITY;
            out |= (ok ? 0u : 1u) << (4 * n + e);
          }
        float mx[2], al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          float mn = rs.m[e];
          if (mx[e] > -INFINITY && (mn == -INFINITY || mx[e] > mn + kRescaleD)) mn = mx[e];
          al[e] = mn == rs.m[e] ? 1.f : ex2(rs.m[e] - mn);
          rs.m[e] = mn;
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] *= al[e >> 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) rs.l[e] *= al[e];
        }
        float pr[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = rs.m[e >> 1] == -INFINITY ? 0.f : rs.m[e >> 1];
            const float w = (out >> (4 * n + e)) & 1u ? 0.f : ex2(s[n][e] - m);
            rs.l[e >> 1] += w;
            pr[n][e] = w;
            if constexpr (kQ8) pr[n][e] = (out >> (4 * n + e)) & 1u ? 0.f : w * vsc[n][e & 1];
          }
        // ---- O += P V
        // A key that some rows see and others do not may hold anything in its
        // V row, and 0 times an infinity is not 0: such a piece, if its V rows
        // are not all finite, is added key by key.
        bool plain = true;
        if (__any_sync(0xffffffffu, out != 0u)) {
          bool bad = false;
#pragma unroll
          for (int i = 0; i < R::kTileB / 512; ++i) {
            const uint4 u = lds128(st + R::kTileB + i * 512 + lane * 16);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) bad = bad || (kQ8 ? nan_e4m3(w[q]) : nonfinite16(w[q], kHalfP ? 0x7c00u : 0x7f80u));
          }
          plain = !__any_sync(0xffffffffu, bad);
        }
        if (plain) {
          uint32_t pa[4];
          pa[0] = pack16<kHalfP>(pr[0][0], pr[0][1]);
          pa[1] = pack16<kHalfP>(pr[0][2], pr[0][3]);
          pa[2] = pack16<kHalfP>(pr[1][0], pr[1][1]);
          pa[3] = pack16<kHalfP>(pr[1][2], pr[1][3]);
          const uint32_t vt = st + R::kTileB;
          if constexpr (!kQ8) {
            const int r = lane & 15, hc = lane >> 4;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              uint32_t b[4];
              ldsm4t(vt + r * R::kRowBytes + (((2 * n + hc) ^ (r & 7)) << 4), b);
              mma16816<kHalfP>(acc[2 * n], pa, b[0], b[1]);
              mma16816<kHalfP>(acc[2 * n + 1], pa, b[2], b[3]);
            }
          } else {
            // Column g8 of n-tile j stands for d = 16 g8 + j: a thread reads
            // whole 16-byte chunks of its four keys and pairs their bytes.
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 2 * t4 + (i & 1) + 8 * (i >> 1);
              u[i] = lds128(vt + r * R::kRowBytes + ((g8 ^ ((r & 1) << 2)) << 4));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t w[4] = {(&u[0].x)[q], (&u[1].x)[q], (&u[2].x)[q], (&u[3].x)[q]};
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                // bytes (w0[2y], w1[2y], w0[2y + 1], w1[2y + 1]): columns 2y and 2y + 1 of two keys
                const uint32_t sel = y ? 0x7362u : 0x5140u;
                const uint32_t lo = __byte_perm(w[0], w[1], sel), hi = __byte_perm(w[2], w[3], sel);
                mma16816<false>(acc[4 * q + 2 * y], pa, e4m3x2_bf16(lo), e4m3x2_bf16(hi));
                mma16816<false>(acc[4 * q + 2 * y + 1], pa, e4m3x2_bf16(lo >> 16), e4m3x2_bf16(hi >> 16));
              }
            }
          }
        } else {
#pragma unroll
          for (int kc = 0; kc < kPiece; ++kc) {
            const int src = (lane & ~3) | ((kc & 7) >> 1);
            const uint32_t hid = __shfl_sync(0xffffffffu, out, src) >> (4 * (kc >> 3) + (kc & 1));
            const float w = __shfl_sync(0xffffffffu, pr[kc >> 3][kc & 1], src);
            const float w8 = __shfl_sync(0xffffffffu, pr[kc >> 3][2 + (kc & 1)], src);
            auto add = [&](int n, int i, float v) {
              if (!(hid & 1u)) acc[n][i] = fmaf(w, v, acc[n][i]);
              if (!(hid & 4u)) acc[n][2 + i] = fmaf(w8, v, acc[n][2 + i]);
            };
            const uint32_t row = st + R::kTileB + kc * R::kRowBytes;
            if constexpr (!kQ8) {
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                const float2 v = unpack16<kHalfP>(__float_as_uint(lds32(row + ((n ^ (kc & 7)) << 4) + t4 * 4)));
                add(n, 0, v.x);
                add(n, 1, v.y);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint4 u = lds128(row + (((2 * t4 + i) ^ ((kc & 1) << 2)) << 4));
                const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                  const float2 v = unpack16<true>(e4m3x2_f16(w4[n >> 2] >> (8 * (n & 3))));
                  add(n, i, v.x);
                  add(n + 1, i, v.y);
                }
              }
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage that the next fetch overwrites
      fetch(k + R::kStages - 1);
    }
    cp_async_wait<0>();

    // ---- the four warps' results, through the rings, to one
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      rs.l[e] += __shfl_xor_sync(0xffffffffu, rs.l[e], 1);
      rs.l[e] += __shfl_xor_sync(0xffffffffu, rs.l[e], 2);
    }
    __syncwarp();
    float* wo = reinterpret_cast<float*>(smem + warp * R::kWarpB);
    float* wm = wo + kRows * kDD;  // m, then l
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g8 + 8 * e;
      if (r < rows) {
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            wo[r * kDD + (kQ8 ? 16 * (2 * t4 + i) + n : 8 * n + 2 * t4 + i)] = acc[n][2 * e + i];
        if (t4 == 0) {
          wm[r] = rs.m[e];
          wm[kRows + r] = rs.l[e];
        }
      }
    }
    __syncthreads();
    auto warp_part = [&](int w, int r, float& m, float& l) {
      const float* x = reinterpret_cast<const float*>(smem + w * R::kWarpB) + kRows * kDD;
      m = x[r];
      l = x[kRows + r];
    };
    auto warp_vec = [&](int w, int r, int c4) {
      return reinterpret_cast<const float4*>(smem + w * R::kWarpB)[r * (kDD / 4) + c4];
    };
    split_finish<kRows, kDD, kMode == kF16 || kMode == kE4m3F16>(p, sp, ss, share, it, k0, k1, kDWarps, warp_part,
                                                                warp_vec);
    split_advance<kDTile, kRows>(p, share, it, k1 - k0);
    __syncthreads();  // the rings are free again
  }
}

// Dynamic shared memory above the default, once per device and kernel.
template <int kMode>
cudaError_t launch_mode(const PagedP& p, const SplitP& sp, cudaStream_t st) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(paged_decode_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Ring<kMode>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  paged_decode_kernel<kMode><<<sp.ctas, kDThreads, Ring<kMode>::kSmem, st>>>(p, sp);
  return cudaGetLastError();
}

int decode_ctas() { return 2 * sm_count(); }  // two CTAs an SM: one's joins run under the other's copies

}  // namespace

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  static int known[64] = {};
  if (dev < 64 && known[dev]) return known[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
  if (dev < 64) known[dev] = n;
  return n;
}

bool paged_pieces_ok(const PagedP& p) {
  const CacheP& c = p.c;
  if (c.d != kDD || c.dv != kDD || p.dtype == ATTN_F32 || c.page_size % kPiece || !c.num_pages) return false;
  const int el = c.dtype == ATTN_E4M3 ? 1 : 2;
  uintptr_t bits = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                   reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.o);
  for (int i = 0; i < 3; ++i) bits |= (uintptr_t)(c.sk[i] * el) | (uintptr_t)(c.sv[i] * el);
  for (int i = 0; i < 2; ++i) bits |= (uintptr_t)(p.sq[i] * 2) | (uintptr_t)(p.so[i] * 2);
  return bits % 16 == 0;
}

bool paged_decode_supported(const PagedP& p, int32_t max_q) {
  return paged_pieces_ok(p) && (int64_t)max_q * (p.Hq / p.c.Hkv) <= kRows;
}

size_t paged_decode_workspace_bytes(size_t& zero) {
  zero = align_up((size_t)decode_ctas() * sizeof(uint32_t), 256);
  return zero + (size_t)decode_ctas() * 2 * split_part_floats<kRows, kDD>() * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedP& p, void* ws, cudaStream_t st) {
  size_t zero;
  paged_decode_workspace_bytes(zero);
  SplitP sp;
  sp.ctas = decode_ctas();
  sp.min_tiles = kMinTiles;
  sp.counters = static_cast<uint32_t*>(ws);
  sp.part = reinterpret_cast<float*>(static_cast<char*>(ws) + zero);
  if (p.c.dtype == ATTN_E4M3)
    return p.dtype == ATTN_F16 ? launch_mode<kE4m3F16>(p, sp, st) : launch_mode<kE4m3Bf16>(p, sp, st);
  return p.dtype == ATTN_F16 ? launch_mode<kF16>(p, sp, st) : launch_mode<kBf16>(p, sp, st);
}

}  // namespace attn
