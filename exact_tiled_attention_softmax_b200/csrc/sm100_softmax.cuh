// One S row per thread -> P, in TMEM: the running-summary update of the
// tensor-core forward kernels (dense and paged), for a 128-key tile whose row
// is the calling thread's TMEM lane.
#pragma once

#include <math.h>

#include "sm100_ptx.cuh"

namespace attn {

namespace {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // move the running max only past 2^8
constexpr int kPolyEvery = 4;              // forward: every k-th pair of exponentials on the FMA pipe (0: none)

// Does pair e of a 16-pair chunk take its exponentials on the FMA pipe? Not
// with dropout: there the softmax warps also run Philox4x32-10, whose
// multiplies share the pipe the polynomial would use.
template <bool kDrop>
__host__ __device__ constexpr bool poly_pair(int e) {
  return !kDrop && kPolyEvery > 0 && e % (kPolyEvery > 0 ? kPolyEvery : 1) == kPolyEvery - 1;
}

// Bits lo..hi (inclusive, within [0, 63]) of a 64-bit word; 0 when lo > hi.
__device__ __forceinline__ uint64_t range_bits64(int64_t lo, int64_t hi) {
  if (lo > hi || hi < 0 || lo > 63) return 0ull;
  lo = lo < 0 ? 0 : lo;
  hi = hi > 63 ? 63 : hi;
  const uint64_t upto = hi >= 63 ? ~0ull : ((1ull << (hi + 1)) - 1ull);
  return upto & ~((1ull << lo) - 1ull);
}

// New running maximum after a tile whose (scaled, base-2) maximum is mx:
// moved only when mx exceeds it by more than the threshold (or on the first
// tile with an allowed key). Returns the factor alpha = 2^(m_old - m_new) that
// rescales the earlier terms (0 when there were none, 1 when m stays).
__device__ __forceinline__ float move_max(float mx, float& m_run) {
  float m_new = m_run;
  if (mx > -INFINITY && (m_run == -INFINITY || mx > m_run + kRescaleThreshold)) m_new = fmaxf(mx, m_run);
  const float alpha = (m_new == m_run) ? 1.f : ex2(m_run - m_new);
  m_run = m_new;
  return alpha;
}

// 2^x of two by a polynomial: x below -125 counts as that or, with kFine, below
// -127 as minus infinity: at -127 the polynomial is 1 and its exponent field
// becomes 0, so the result is 0 (between the two it is below 2^-125).
template <bool kFine>
__device__ __forceinline__ uint64_t exp2_pair(float x0, float x1) {
  return kFine ? exp2_fma2_fine(f2_pack(fmaxf(x0, -127.f), fmaxf(x1, -127.f)))
               : exp2_fma2(f2_pack(fmaxf(x0, -125.f), fmaxf(x1, -125.f)));
}

// One S row (128 keys, all allowed, no dropout) of the calling thread's TMEM
// lane -> P (bf16 pairs written over the row's first 64 columns), with the
// running summary (m_run, l_run) updated. The maximum takes two 64-column
// TMEM loads and the exponentials four 32-column reloads, so that no more
// than 64 scores are live at once (the forward then needs no spill slots);
// x = s c log2(e) - m is formed on packed fp32 pairs and every kPolyEvery-th
// pair of exponentials runs on the FMA pipe instead of MUFU. Returns alpha.
// kStrict: the polynomial is the quartic; a NaN or +inf score makes l_run NaN (the polynomial and the plain
// maximum drop a NaN), and a row of -inf scores adds nothing.
template <bool kH, bool kDrop, bool kStrict = false>
__device__ __forceinline__ float softmax_full_tile(uint32_t tS, float scale_log2, float& m_run, float& l_run,
                                                   uint64_t kb0, uint64_t kb1) {
  float mx;
  {
    auto hi3 = [](float a, float b, float c) { return kStrict ? max3nan(a, b, c) : max3f(a, b, c); };
    auto lo3 = [](float a, float b, float c) { return kStrict ? min3nan(a, b, c) : min3f(a, b, c); };
    const bool pos = scale_log2 >= 0.f;
    float e0 = pos ? -INFINITY : INFINITY, e1 = e0, e2 = e0, e3 = e0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t s0[32], s1[32];
      tmem_ld32(tS + 64 * hf, s0);
      tmem_ld32(tS + 64 * hf + 32, s1);
      tmem_wait_ld();
      if (pos) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          e0 = hi3(e0, __uint_as_float(s0[e]), __uint_as_float(s0[e + 1]));
          e1 = hi3(e1, __uint_as_float(s0[e + 2]), __uint_as_float(s0[e + 3]));
          e2 = hi3(e2, __uint_as_float(s1[e]), __uint_as_float(s1[e + 1]));
          e3 = hi3(e3, __uint_as_float(s1[e + 2]), __uint_as_float(s1[e + 3]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          e0 = lo3(e0, __uint_as_float(s0[e]), __uint_as_float(s0[e + 1]));
          e1 = lo3(e1, __uint_as_float(s0[e + 2]), __uint_as_float(s0[e + 3]));
          e2 = lo3(e2, __uint_as_float(s1[e]), __uint_as_float(s1[e + 1]));
          e3 = lo3(e3, __uint_as_float(s1[e + 2]), __uint_as_float(s1[e + 3]));
        }
      }
    }
    mx = (pos ? hi3(e0, e1, kStrict ? max3nan(e2, e3, e3) : fmaxf(e2, e3))
              : lo3(e0, e1, kStrict ? min3nan(e2, e3, e3) : fminf(e2, e3))) * scale_log2;
  }
  const bool poison = kStrict && !(mx < INFINITY);
  if (poison) mx = -INFINITY;
  const float alpha = move_max(mx, m_run);
  const float msub = kStrict && m_run == -INFINITY ? 0.f : m_run;
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-msub, -msub);
  uint64_t acc0 = 0ull, acc1 = 0ull;  // two packed partial sums (pairs of +0.0f)
  auto chunk = [&](const uint32_t (&r)[32], int q) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t x = f2_fma(f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sc2, nm2);
      float x0, x1;
      f2_unpack(x, x0, x1);
      const uint64_t pp = poly_pair<kDrop>(e)
                              ? exp2_pair<kStrict>(x0, x1)
                              : f2_pack(ex2(x0), ex2(x1));
      if (e & 1)
        acc1 = f2_add(acc1, pp);
      else
        acc0 = f2_add(acc0, pp);
      float p0, p1;
      f2_unpack(pp, p0, p1);
      if constexpr (kDrop) {  // xi only in the P operand; the sum keeps every term
        const uint64_t kw = q < 2 ? kb0 : kb1;
        const int bit = (q & 1) * 32 + 2 * e;
        p0 = ((kw >> bit) & 1ull) ? p0 : 0.f;
        p1 = ((kw >> (bit + 1)) & 1ull) ? p1 : 0.f;
      }
      pk[e] = pack16<kH>(p0, p1);
    }
    tmem_st16(tS + q * 16, pk);
  };
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t r[32];
    tmem_ld32(tS + 32 * q, r);
    tmem_wait_ld();
    chunk(r, q);
  }
  float a0, a1, b0, b1;
  f2_unpack(acc0, a0, a1);
  f2_unpack(acc1, b0, b1);
  l_run = poison ? NAN : l_run * alpha + ((a0 + a1) + (b0 + b1));
  return alpha;
}

// The general row: allowed-key bits (mw0, mw1) and dropout keep bits
// (kb0, kb1) per key; two TMEM passes of 64 columns for the maximum, then 32
// columns per pass for the exponentials. The sum and the maximum use
// every allowed key (undropped); P carries only the kept ones (the 1/(1-rho)
// factor is applied to O in fp32 at the end). Returns alpha.
template <bool kH>
__device__ __forceinline__ float softmax_masked_tile(uint32_t tS, float scale_log2, uint64_t mw0, uint64_t mw1,
                                                     uint64_t kb0, uint64_t kb1, float& m_run, float& l_run) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t r0[32], r1[32];
    tmem_ld32(tS + hf * 64, r0);
    tmem_ld32(tS + hf * 64 + 32, r1);
    tmem_wait_ld();
    const uint64_t mw = hf ? mw1 : mw0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if ((mw >> e) & 1ull) mx = fmaxf(mx, __uint_as_float(r0[e]) * scale_log2);
      if ((mw >> (32 + e)) & 1ull) mx = fmaxf(mx, __uint_as_float(r1[e]) * scale_log2);
    }
  }
  const float alpha = move_max(mx, m_run);
  const float msub = m_run == -INFINITY ? 0.f : m_run;
  float sum = 0.f;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t r[32];
    tmem_ld32(tS + q * 32, r);
    tmem_wait_ld();
    const uint64_t mw = q < 2 ? mw0 : mw1;
    const uint64_t kw = q < 2 ? kb0 : kb1;
    const int base = (q & 1) * 32;
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int bit = base + 2 * e;
      const float p0 = ((mw >> bit) & 1ull) ? ex2(__uint_as_float(r[2 * e]) * scale_log2 - msub) : 0.f;
      const float p1 = ((mw >> (bit + 1)) & 1ull) ? ex2(__uint_as_float(r[2 * e + 1]) * scale_log2 - msub) : 0.f;
      sum += p0 + p1;
      pk[e] = pack16<kH>(((kw >> bit) & 1ull) ? p0 : 0.f, ((kw >> (bit + 1)) & 1ull) ? p1 : 0.f);
    }
    tmem_st16(tS + q * 16, pk);
  }
  l_run = l_run * alpha + sum;
  return alpha;
}

}  // namespace

}  // namespace attn
