// Attention over a paged cache for few new tokens per sequence (16 or 32 (token,
// head of the group) rows per K/V head, paged_decode_supported): 16-bit or e4m3
// cache, d = dv = 128, pages of a multiple of 16 positions.
//
// The arithmetic is 4 flops per cached element and row, so with up to 16 rows
// the cache's bytes bound it, and what matters is to keep enough of them in
// flight and to spend few instructions on each. Every warp streams 16-key
// pieces of its own through a private ring of asynchronous copies (no barrier
// between warps until an item ends). The products are m16n8k16 with the keys
// (then the head dimension) on the 16-row side and the query rows on the
// 8-column side, S^T = K Q^T and O^T += V^T P^T, so that eight rows cost
// half of what they would as the 16-row operand, in products and in
// registers; P^T reaches the second product's operand layout by an 8x8 register
// transpose.
//
// Work split: an item is (sequence, block of 8 or 16 rows, K/V head); its
// keys are cut into 64-key tiles (one 16-key piece per warp) and all tiles of
// all items, in order, are dealt to the CTAs in equal consecutive shares, so
// the load is even whatever the lengths are and the grid needs no length from
// the host. decode_join_kernel adds the sums of an item that several CTAs share
// in the CTAs' order, so the result does not depend on timing.
//
// Measured on the device, joins included (32 query heads over 8): 64 e4m3
// sequences of up to 8192 keys 151 us = 5.1 TB/s of cache (0.78 of the measured
// copy rate; no unit is full, the warps wait on fixed instruction latencies
// and at 166 registers 12 of them share an SM), 32 fp16 sequences of up to
// 16384 with a window of 1024 and four first keys 34.6 us = 3.9 TB/s (an item
// is 17 tiles, so starting and joining shows), one sequence of 2000 bf16 keys
// 11.2 us (two launches and their latencies; its bytes are 1.3 us).
#include <math.h>

#include "paged.cuh"
#include "paged_split.cuh"
#include "sm100_paged.h"
#include "sm100_ptx.cuh"

namespace attn {

using namespace sm100;

namespace {

constexpr int kDD = 128;          // head width
constexpr int kMaxRows = 16;      // most query rows per item: 8 or 16
constexpr int kDWarps = 4;
constexpr int kDThreads = kDWarps * 32;
constexpr int kPiece = 16;        // keys per warp and tile
constexpr int kDTile = kDWarps * kPiece;
constexpr float kLog2eD = 1.4426950408889634f;
constexpr int kMinTiles = 2;      // key tiles a CTA takes at least
constexpr float kRescaleD = 8.f;  // move the running maximum only past 2^8
constexpr float kScaleDown = 0x1p-30f, kScaleUp = 0x1p30f;  // e4m3, on V's scales

enum { kBf16 = 0, kF16 = 1, kE4m3Bf16 = 2, kE4m3F16 = 3 };  // cache type (and query type)

// kNT: 8-row column tiles of an item.
template <int kMode, int kNT>
struct Ring {
  static constexpr bool kQ8 = kMode >= kE4m3Bf16;
  static constexpr int kRowBytes = kQ8 ? kDD : 2 * kDD;
  static constexpr int kTileB = kPiece * kRowBytes;            // one of K, V
  static constexpr int kStageB = 2 * kTileB + (kQ8 ? 128 : 0); // + 16 (K scale, V scale)
  static constexpr int kStages = kQ8 ? 4 : 3;
  // CTAs an SM, against copies in flight per warp (227 KB, 65536 registers):
  // 64 e4m3 sequences of up to 8192 keys took 159 us with 3 CTAs of 4 stages,
  // 164 with 4 of 3, 184 with 4 of 2, 190 with 2 of 5; the fp16 window workload
  // of 32 sequences 35.1 us with 2 of 3, 36.6 with 3 of 2, 51 with 2 of 4.
  // (Tuned on 8 rows: with 16 rows of an e4m3 cache three CTAs leave 168
  // registers, and 100 to 176 bytes spill; two CTAs are untried there.)
  static constexpr int kCtas = kQ8 ? 3 : 2;
  static constexpr int kWarpB = kStages * kStageB;
  static constexpr int kSmem = kDWarps * kWarpB;
  static_assert(kWarpB >= 8 * kNT * (kDD + 2) * 4, "the ring also carries a warp's result to the join");
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
__device__ __forceinline__ void lds64(uint32_t addr, float& a, float& b) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(addr) : "memory");
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

// Four e4m3 codes as two packed fp16 pairs, low codes first; exact.
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// One stored element of shared memory as fp32.
template <bool kHalf>
__device__ __forceinline__ float ld16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return kHalf ? __half2float(*reinterpret_cast<const __half*>(&v)) : __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ float ld8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  __nv_fp8_e4m3 x;
  x.__x = (__nv_fp8_storage_t)v;
  return float(x);
}

// Does a word of stored values (two of 16 bits with the exponent mask expo, or
// four e4m3 codes) hold an infinity or a NaN?
__device__ __forceinline__ bool nonfinite16(uint32_t v, uint32_t expo) {
  return (v & expo) == expo || ((v >> 16) & expo) == expo;
}
__device__ __forceinline__ bool nan_e4m3(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// An 8x8 matrix of 16-bit elements spread over the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int kMode, int kNT>
__global__ void __launch_bounds__(kDThreads, (Ring<kMode, kNT>::kCtas)) paged_decode_kernel(const __grid_constant__ PagedP p,
                                                                                       const __grid_constant__ SplitP sp) {
  using R = Ring<kMode, kNT>;
  constexpr bool kQ8 = R::kQ8;
  constexpr int kRows = 8 * kNT;
  constexpr bool kHalfS = kMode != kBf16;   // K Q^T in fp16 (an e4m3 K is exact in it)
  // V^T P^T in fp16 too (e4m3 V is exact in it, and half as many instructions
  // away as bf16): a probability times its V row's scale has fp16's 2^-11,
  // and its range is kept by the running reference, below.
  constexpr bool kHalfP = kMode != kBf16;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SplitShared ss;
  const CacheP& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3, g8 = lane >> 2;
  const uint32_t ring = smem_u32(smem) + warp * R::kWarpB;
  // Errors gather in shared memory and leave with the CTA's record, so that
  // nothing has to be cleared before the launch.
  if (threadIdx.x == 0) {
    ss.errors = 0u;
    sp.rec[blockIdx.x].parts = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0) report_ragged(c, &ss.errors);
  const int group = p.Hq / c.Hkv;
  const bool causal = p.flags & ATTN_MASK_CAUSAL, window = p.flags & ATTN_MASK_WINDOW;
  const int W = (int)p.window, first = (int)p.first;

  Share share = split_share<kDTile, kRows>(p, sp, ss);
  while (share.left > 0) {
    const Item it = split_item<kDTile, kRows>(p, share);
    const int k0 = (int)share.at, k1 = (int)(it.tiles - k0 < share.left ? it.tiles : k0 + share.left);
    const int rows = it.rows;
    // Positions are below 2^31 (the cache's limit), and differences fit too.
    const int L = (int)it.s.L, pos0 = L - it.s.n;  // the first new token's position
    const int p_lo = pos0 + it.row0 / group, p_hi = pos0 + (it.row0 + rows - 1) / group;  // the rows' first and last
    // Keys some row sees: [any_lo, any_hi] and [0, first); all rows: [all_lo, all_hi] (and below first).
    const int any_hi = causal && p_hi < L - 1 ? p_hi : L - 1, all_hi = causal && p_lo < L - 1 ? p_lo : L - 1;
    const int any_lo = window && p_lo >= W ? p_lo - W + 1 : 0, all_lo = window && p_hi >= W ? p_hi - W + 1 : 0;
    const int firsts = window ? first : 0;

    // ---- the loads of one 16-key piece (tile k of the item) into its stage
    int base = k0 - 32;        // lane l holds page and offset of tile base + l
    int pg_mine = -1, off_mine = 0;
    constexpr int kChunks = R::kRowBytes / 16;  // 16-byte chunks of a row
    constexpr int kRowsAt = 32 / kChunks;       // rows a warp covers per copy instruction
    const int cr = lane / kChunks, cc = lane % kChunks;
    constexpr int kEl = kQ8 ? 1 : 2;
    const uint8_t* kb = static_cast<const uint8_t*>(c.k) + ((int64_t)it.h * c.sk[2] + cr * c.sk[1]) * kEl + cc * 16;
    const uint8_t* vb = static_cast<const uint8_t*>(c.v) + ((int64_t)it.h * c.sv[2] + cr * c.sv[1]) * kEl + cc * 16;
    const int64_t kstep = c.sk[1] * kEl * kRowsAt, vstep = c.sv[1] * kEl * kRowsAt;
    // e4m3: lanes 0-15 copy the K scales, 16-31 the V scales.
    const float* scb = nullptr;
    int64_t scp = 0, scr = 0;
    if constexpr (kQ8) {
      const int64_t* ssr = lane < 16 ? c.sks : c.svs;
      scb = (lane < 16 ? c.ks : c.vs) + (int64_t)it.h * ssr[2] + (lane & 15) * ssr[1];
      scp = ssr[0];
      scr = ssr[1];
    }
    uint32_t dead = 0;  // bit s: stage s holds a piece that no row sees, or whose page is bad
    int put = 0;        // stage of the next fetch
    auto fetch = [&](int k) {
      if (k < k1) {
        if (k - base >= 32) {
          base = k;
          const int j = it.tile_at(k + lane) * kDTile + warp * kPiece;
          pg_mine = -1;
          if (k + lane < k1 && j < L) {
            const int e = (int)((unsigned)j / (unsigned)c.page_size);
            off_mine = j - e * c.page_size;
            pg_mine = c.table[(int64_t)it.b * c.table_stride + e];
            if (pg_mine < 0 || pg_mine >= c.num_pages) {
              atomicOr(&ss.errors, ATTN_DEVERR_PAGE);
              pg_mine = -1;
            }
          }
        }
        const int pg = __shfl_sync(0xffffffffu, pg_mine, k - base), off = __shfl_sync(0xffffffffu, off_mine, k - base);
        const int j0 = it.tile_at(k) * kDTile + warp * kPiece;
        const bool live = pg >= 0 && j0 <= any_hi && (j0 + kPiece > any_lo || j0 < firsts);
        dead = live ? dead & ~(1u << put) : dead | 1u << put;
        if (live) {
          const uint32_t st = ring + put * R::kStageB;
          const uint8_t* ks = kb + (pg * c.sk[0] + off * c.sk[1]) * kEl;
          const uint8_t* vs = vb + (pg * c.sv[0] + off * c.sv[1]) * kEl;
          // (whole: some row sees every key of the piece, so all of it is copied)
          const bool whole = j0 + kPiece - 1 <= any_hi && (j0 >= any_lo || j0 + kPiece <= firsts);
#pragma unroll
          for (int i = 0; i < kPiece / kRowsAt; ++i) {
            const int r = cr + i * kRowsAt, j = j0 + r;
            const bool take = whole || (j <= any_hi && (j >= any_lo || j < firsts));
            // 16-bit rows: the 16-byte chunk index is permuted by the row so
            // that ldmatrix reads eight rows without bank conflicts; e4m3
            // rows by bit 2 of the index and the row's low bit, for the
            // K side (four chunks of two rows at a time).
            const int pc = kQ8 ? cc ^ ((r & 1) << 2) : cc ^ (r & 7);
            cp16(st + r * R::kRowBytes + pc * 16, ks + i * kstep, take);
            cp16(st + R::kTileB + r * R::kRowBytes + pc * 16, vs + i * vstep, take);
          }
          if constexpr (kQ8) {
            const int j = j0 + (lane & 15);
            cp4(st + 2 * R::kTileB + (lane & 15) * 8 + (lane >> 4) * 4, scb + pg * scp + off * scr,
                whole || (j <= any_hi && (j >= any_lo || j < firsts)));
          }
        }
      }
      put = put + 1 == R::kStages ? 0 : put + 1;
      cp_async_commit();
    };
#pragma unroll 1
    for (int k = k0; k < k0 + R::kStages - 1; ++k) fetch(k);

    // ---- Q as B fragments: column g8 of column tile nt is row 8 nt + g8 (rows past
    // the block's are zero). xs: score factor c log2(e) (over the row's power
    // of two) of the columns whose scores the thread holds, 2 t4 and 2 t4 + 1.
    uint32_t qb[kNT][8][2];
    float xs[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int r = 8 * nt + g8, rr = it.row0 + r;
      const bool live = r < rows;
      const uint16_t* qr = static_cast<const uint16_t*>(p.q) + (it.s.q0 + rr / group) * p.sq[0] +
                           (int64_t)(it.h * group + rr % group) * p.sq[1];
      float factor = p.scale * kLog2eD;
      if constexpr (!kQ8) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qb[nt][ks][0] = live ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t4) : 0u;
          qb[nt][ks][1] = live ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8 + 2 * t4) : 0u;
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
          qb[nt][ks][0] = u.x;
          qb[nt][ks][1] = u.y;
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
          const float up = __uint_as_float((uint32_t)(13 - ex + 127) << 23);  // 2^(13 - ex), ex in [-100, 127]
          factor *= __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 a = unpack16<false>(qb[nt][ks][i]);
              qb[nt][ks][i] = pack_fp16(a.x * up, a.y * up);
            }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) xs[nt][e] = __shfl_sync(0xffffffffu, factor, (2 * t4 + e) * 4);
    }

    float acc[kNT][8][4];
    float m[kNT][2], l[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    }

    int take = 0;  // stage of the piece at hand
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      cp_async_wait<R::kStages - 2>();
      __syncwarp();
      const uint32_t st = ring + take * R::kStageB;
      if (!((dead >> take) & 1u)) {
        // ---- S^T = K Q^T, even and odd steps summed apart
        float s[kNT][4], s2[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
        if constexpr (!kQ8) {
          const int r = lane & 15, hc = lane >> 4;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t a[4];
            ldsm4(st + r * R::kRowBytes + (((2 * ks + hc) ^ (r & 7)) << 4), a);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma16816<kHalfS>(ks & 1 ? s2[nt] : s[nt], a, qb[nt][ks][0], qb[nt][ks][1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = st + g8 * R::kRowBytes + (((t4 + 4 * i) ^ ((g8 & 1) << 2)) << 4);
            const uint4 u = lds128(at), v = lds128(at + 8 * R::kRowBytes);
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t a[4];  // keys g8 and g8 + 8, the step's lower and upper two d of each
              e4m3x4_f16(uw[q], a[0], a[2]);
              e4m3x4_f16(vw[q], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
                mma16816<kHalfS>(q & 1 ? s2[nt] : s[nt], a, qb[nt][4 * i + q][0], qb[nt][4 * i + q][1]);
            }
          }
        }
        // ---- scale, mask, running summary. Element e: key j0 + g8 + 8 (e >> 1),
        // row 8 nt + 2 t4 + (e & 1).
        // The running reference m of an e4m3 row is that of s + log2(v), v being
        // 2^-30 times V's scale, so that the operand 2^(s - m) v stays within 2^8
        // of its largest value whatever the scales are; the sum takes 2^(s - m)
        // itself, in fp32. (v below 2^-90 counts as that there. With the 2^-30 the
        // sum's largest term is between 2^-90 and 2^98 for scales from 2^-60 to
        // 2^120, so that terms 2^36 times smaller still count.)
        float ksc[2] = {1.f, 1.f}, vsc[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
        if constexpr (kQ8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lds64(st + 2 * R::kTileB + (g8 + 8 * i) * 8, ksc[i], vsc[i]);
            vsc[i] *= kScaleDown;
            lv[i] = fminf(fmaxf(__log2f(fabsf(vsc[i])), -90.f), 90.f);
          }
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][e] = (s[nt][e] + s2[nt][e]) * xs[nt][e & 1];
            if constexpr (kQ8) s[nt][e] *= ksc[e >> 1];
          }
        const int j0 = it.tile_at(k) * kDTile + warp * kPiece;
        const bool full = j0 + kPiece - 1 <= all_hi && p_lo >= 0 && (j0 >= all_lo || j0 + kPiece <= firsts);
        uint32_t out = 0;  // bit 4 nt + e: masked
        if (!full) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 8 * nt + 2 * t4 + (e & 1), j = j0 + g8 + 8 * (e >> 1);
              const int pos = pos0 + (it.row0 + r) / group;
              bool ok = j < L && r < rows && pos >= 0;
              if (causal) ok = ok && j <= pos;
              if (window) ok = ok && (j > pos - W || j < first);
              if (!ok) {
                s[nt][e] = -INFINITY;
                out |= 1u << (4 * nt + e);
              }
            }
        }
        float al[kNT][2];
        bool moved = false;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[nt][e] + lv[0], s[nt][e + 2] + lv[1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            float mn = m[nt][e];
            if (mx > mn + kRescaleD) mn = mx;  // (mn = -inf: any finite mx)
            al[nt][e] = mn == m[nt][e] ? 1.f : ex2(m[nt][e] - mn);
            moved = moved || mn != m[nt][e];
            m[nt][e] = mn;
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt][j][e] *= al[nt][e & 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) l[nt][e] *= al[nt][e];
          }
        }
        uint32_t pb[kNT][2];  // P^T as B fragments
        float pr[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = ex2(s[nt][e] - (m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1]));  // 0 where masked
            l[nt][e & 1] += w;
            pr[nt][e] = kQ8 ? w * vsc[e >> 1] : w;
          }
        }
        // A key that some rows see and others do not may hold anything in its
        // V row, and 0 times an infinity is not 0: such a piece, if its V rows
        // are not all finite, is added key by key.
        bool plain = true;
        if (!full) {
          if constexpr (kQ8) {  // nor may a masked row's scale count
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) pr[nt][e] = (out >> (4 * nt + e)) & 1u ? 0.f : pr[nt][e];
          }
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
        // ---- O^T += V^T P^T
        const uint32_t vt = st + R::kTileB;
        if (plain) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) pb[nt][i] = transpose8(pack16<kHalfP>(pr[nt][2 * i], pr[nt][2 * i + 1]));
          if constexpr (!kQ8) {
            const int r = (lane & 7) + ((lane >> 4) << 3), hc = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t a[4];
              ldsm4t(vt + r * R::kRowBytes + (((2 * j + hc) ^ (r & 7)) << 4), a);
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt) mma16816<kHalfP>(acc[nt][j], a, pb[nt][0], pb[nt][1]);
            }
          } else {
            // Rows g8 and g8 + 8 of m-tile j stand for d = 16 g8 + 2 j and
            // 16 g8 + 2 j + 1: a thread reads whole 16-byte chunks of its
            // four keys and pairs their bytes.
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
                // bytes (w0[2y], w1[2y], w0[2y + 1], w1[2y + 1]): d = .. 2y and 2y + 1 of two keys
                const uint32_t sel = y ? 0x7362u : 0x5140u;
                uint32_t a[4];
                e4m3x4_f16(__byte_perm(w[0], w[1], sel), a[0], a[1]);
                e4m3x4_f16(__byte_perm(w[2], w[3], sel), a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) mma16816<true>(acc[nt][2 * q + y], a, pb[nt][0], pb[nt][1]);
              }
            }
          }
        } else {
#pragma unroll 1
          for (int kc = 0; kc < kPiece; ++kc) {
            const int src = (kc & 7) * 4 + t4;
            const uint32_t hid = __shfl_sync(0xffffffffu, out, src) >> (2 * (kc >> 3));
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e)
                w[e] = __shfl_sync(0xffffffffu, kc < 8 ? pr[nt][e] : pr[nt][2 + e], src);
              const uint32_t row = vt + kc * R::kRowBytes;
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float v;
                  if constexpr (!kQ8) {
                    const int at = 2 * j + i;  // 16-byte chunk of d = 16 j + 8 i + g8
                    v = ld16<kHalfP>(row + ((at ^ (kc & 7)) << 4) + 2 * g8);
                  } else {
                    v = ld8(row + ((g8 ^ ((kc & 1) << 2)) << 4) + 2 * j + i);
                  }
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (!((hid >> (4 * nt + e)) & 1u)) acc[nt][j][2 * i + e] = fmaf(w[e], v, acc[nt][j][2 * i + e]);
                }
            }
          }
        }
      }
      take = take + 1 == R::kStages ? 0 : take + 1;
      __syncwarp();  // every lane has read the stage that the next fetch overwrites
      fetch(k + R::kStages - 1);
    }
    cp_async_wait<0>();

    // ---- the four warps' results, through the rings, to one
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
      }
    __syncwarp();
    float* wo = reinterpret_cast<float*>(smem + warp * R::kWarpB);
    float* wm = wo + kRows * kDD;  // m, then l
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e;
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            wo[r * kDD + (kQ8 ? 16 * g8 + 2 * j + i : 16 * j + 8 * i + g8)] =
                kQ8 ? acc[nt][j][2 * i + e] * kScaleUp : acc[nt][j][2 * i + e];
        if (g8 == 0) {
          wm[r] = m[nt][e];
          wm[kRows + r] = l[nt][e];
        }
      }
    __syncthreads();
    auto warp_part = [&](int w, int r, float& mm, float& ll) {
      const float* x = reinterpret_cast<const float*>(smem + w * R::kWarpB) + kRows * kDD;
      mm = x[r];
      ll = x[kRows + r];
    };
    auto warp_vec = [&](int w, int r, int c4) {
      return reinterpret_cast<const float4*>(smem + w * R::kWarpB)[r * (kDD / 4) + c4];
    };
    split_finish<kRows, kDD, kMode == kF16 || kMode == kE4m3F16>(p, sp, share, it, k0, k1, kDWarps, warp_part, warp_vec);
    split_advance<kDTile, kRows>(p, share, it, k1 - k0);
    __syncthreads();  // the rings are free again
  }
  __syncthreads();
  if (threadIdx.x == 0) sp.rec[blockIdx.x].errors = ss.errors;
}

template <int kRows, bool kHalf>
__global__ void __launch_bounds__(kJoinRows * 32) decode_join_kernel(const PagedP p, const SplitP sp) {
  wait_for_previous();
  join_record<kRows, kDD, kHalf>(p, sp.rec, sp.ctas, true, [&](int i, int e) {
    return split_slot<kRows, kDD>(sp, i + e, e == 0 ? 1 : 0);
  });
}

// Dynamic shared memory above the default, once per device and kernel.
template <int kMode, int kNT>
cudaError_t launch_mode(const PagedP& p, SplitP sp, cudaStream_t st) {
  using R = Ring<kMode, kNT>;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(paged_decode_kernel<kMode, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  sp.ctas = R::kCtas * sm_count();
  paged_decode_kernel<kMode, kNT><<<sp.ctas, kDThreads, R::kSmem, st>>>(p, sp);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_after(decode_join_kernel<8 * kNT, kMode == kF16 || kMode == kE4m3F16>, dim3(sp.ctas, kNT),
                      kJoinRows * 32, 0, st, p, sp);
}

// Blocks of 8 or 16 rows. A 16-bit cache is bound by its bytes either way (64
// sequences of 8192 keys: 317 us with 8 rows and with 16); an e4m3 one by
// instructions, 206 us with 8 rows against 320 with 16 (whose form also spills,
// see Ring), so that three blocks of 8 take less than two of 16 (20 rows: 574
// against 626 us) and two of 8 more than one of 16 (12 rows: 386 against 318 us).
template <int kMode>
cudaError_t launch_rows(const PagedP& p, int rows, const SplitP& sp, cudaStream_t st) {
  const bool eights = rows <= 8 || (kMode >= kE4m3Bf16 && rows > 16 && rows <= 24);
  return eights ? launch_mode<kMode, 1>(p, sp, st) : launch_mode<kMode, 2>(p, sp, st);
}

constexpr int kMostCtas = 4;  // of any form, an SM

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

// Where this kernel is taken and not the chunk kernel, measured with 32 heads
// over 8 (this kernel / the chunk kernel, us). Up to 16 rows always: 64 sequences
// of 8192 keys, 16 rows, bf16 334 / 566, e4m3 320 / 717. Up to 32 rows, where the
// cache is read twice, for e4m3 (64 of 8192: 20 rows 572 / 691, 32 rows 679 / 709;
// 16 of 2048: 57 / 67; one of 32768: 56 / 65), and for 16-bit caches where there
// are fewer K/V heads than SMs to share out (16 of 2048: 49-52 / 53; one of 32768:
// 54-56 / 57; one of 2048: 15 / 21), but not beyond (64 of 8192: 694 / 601). From
// 48 rows on the chunk kernel (16 of 2048, e4m3: 75 / 68).
bool paged_decode_supported(const PagedP& p, int32_t max_q) {
  const bool twice = p.c.dtype == ATTN_E4M3 || (int64_t)p.c.batch * p.c.Hkv <= sm_count();
  return paged_pieces_ok(p) && (int64_t)max_q * (p.Hq / p.c.Hkv) <= (twice ? 2 : 1) * kMaxRows;
}

size_t paged_decode_workspace_bytes() {
  const size_t ctas = (size_t)kMostCtas * sm_count();
  return align_up(ctas * sizeof(JoinRec), 256) + ctas * 2 * split_part_floats<kMaxRows, kDD>() * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedP& p, int32_t max_q, void* ws, cudaStream_t st) {
  SplitP sp;
  sp.ctas = 0;
  sp.min_tiles = kMinTiles;
  sp.rec = static_cast<JoinRec*>(ws);
  sp.part = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                     align_up((size_t)kMostCtas * sm_count() * sizeof(JoinRec), 256));
  const int rows = max_q * (p.Hq / p.c.Hkv);
  if (p.c.dtype == ATTN_E4M3)
    return p.dtype == ATTN_F16 ? launch_rows<kE4m3F16>(p, rows, sp, st) : launch_rows<kE4m3Bf16>(p, rows, sp, st);
  return p.dtype == ATTN_F16 ? launch_rows<kF16>(p, rows, sp, st) : launch_rows<kBf16>(p, rows, sp, st);
}

}  // namespace attn
