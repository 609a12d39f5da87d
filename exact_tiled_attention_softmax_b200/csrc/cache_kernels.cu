// Writing new tokens into a paged K/V cache and reading a cache back.
//
// Both are copies of rows between a dense array and the pool, through the
// block table, with the e4m3 form's arithmetic on the way: a row x is stored
// as s = max|x| / 448 and e4m3(x / s) (448 is e4m3's largest finite value), so
// a code is off by at most 2^-4 of its value, or by half the smallest
// subnormal step (2^-10 s) for the smallest entries. Both quotients are the
// correctly rounded fp32 ones: multiplying by a rounded 1/s instead moves
// values that lie on a border between two codes, which 16-bit inputs often do.
// What bounds them is the bytes: a row is read once and written once, in
// 16-byte pieces, K and V in the same launch. With a full division per
// element the write of an 8192-token prompt was bound by instructions.
// Measured on the device (8 heads of 128): the new tokens of 64 bf16 sequences
// 3.0 us (a launch), a bf16 prompt of 8192 tokens as it is 13.9 us with its
// rows in HBM (4.8 TB/s, 0.74 of the measured copy rate; one round of loads and
// stores per warp) and 8.6 us with them in L2, into e4m3 17.4 and 15.1-15.8 us
// (3.2 TB/s; 62 % of the issue slots, the quotients' chains bound it), eight
// ragged e4m3 sequences of up to 4096 read back as bf16 27.4 us (5.5 TB/s, 0.84
// of the measured copy rate), 1000 fp16 positions read back 3.2 us.
#include <math.h>

#include "paged.cuh"

namespace attn {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kMaxWidth = 576;  // widest head row
constexpr int kHeadBlock = 4;   // heads a warp writes: 4 loads of 16 bytes a lane in flight

// e4m3 codes of two values, rounded to nearest even, saturated at +-448
// (callers never pass more; NaN stays NaN).
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Two e4m3 codes as fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The scale of a row whose largest magnitude is a (NaN in a: the row holds
// one). 1 for a row of zeros, and for one so small that the quotient is 0.
__device__ __forceinline__ float row_scale(float a) {
  const float s = __fdiv_rn(a, kE4m3Max);
  return s == 0.f ? 1.f : s;
}
// The same for a in [2^-80, 2^96]; usual: false outside (and for a NaN).
__device__ __forceinline__ float row_scale_usual(float a, bool& usual) {
  constexpr float r = 1.f / kE4m3Max;
  usual = a >= 0x1p-80f && a <= 0x1p96f;
  const float q = a * r;
  return fmaf(fmaf(-q, kE4m3Max, a), r, q);
}

// max that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Quotients and reciprocals without branches, by the remainder corrections of
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor" (1990): 1/s from an estimate r as r + r (1 - r s), and x / s from
// q = x r as q + r (x - q s), each residual exact in one fma. Correctly rounded
// while nothing leaves the normal range; callers take them for scales in
// [2^-90, 2^90], where a quotient that could still round to a nonzero code
// (at least 2^-11) has a normal remainder.
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(r, fmaf(-r, s, 1.f), r);
}
// Two quotients in packed fp32. (The correction loses the sign of -0: it is put
// back.)
__device__ __forceinline__ void quotients(float& x0, float& x1, float s, float r) {
  const float s0 = x0, s1 = x1;
  asm("{\n\t.reg .b64 x, q, d, ns, rr;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 ns, {%2, %2};\n\tmov.b64 rr, {%3, %3};\n\t"
      "mul.rn.f32x2 q, x, rr;\n\tfma.rn.f32x2 d, q, ns, x;\n\tfma.rn.f32x2 q, d, rr, q;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(-s), "f"(r));
  x0 = copysignf(x0, s0);
  x1 = copysignf(x1, s1);
}

template <typename T>
struct Vec8;  // eight elements as loaded
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  // Largest magnitude; NaN if any element is one.
  __device__ __forceinline__ float top() const {
    const float4 p = a, q = b;
    return max_nan(max_nan(max_nan(fabsf(p.x), fabsf(p.y)), max_nan(fabsf(p.z), fabsf(p.w))),
                   max_nan(max_nan(fabsf(q.x), fabsf(q.y)), max_nan(fabsf(q.z), fabsf(q.w))));
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <typename T2, typename T>
struct Vec8of16 {
  uint4 u;
  __device__ __forceinline__ float top() const {  // two elements at a time
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    T2 m = __habs2(*reinterpret_cast<const T2*>(&w[0]));
#pragma unroll
    for (int e = 1; e < 4; ++e) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const T2*>(&w[e])));
    return max_nan(ld(&m.x), ld(&m.y));
  }
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <>
struct Vec8<__nv_bfloat16> : Vec8of16<__nv_bfloat162, __nv_bfloat16> {
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&t);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<__half> : Vec8of16<__half2, __half> {
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 t = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&t);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Where new token t goes: its sequence's page and the position in it, for the
// whole warp; false when it goes nowhere (no sequence, a negative position, a
// page outside the pool).
__device__ __forceinline__ bool slot_of(const CacheP& c, int t, int64_t& pg, int64_t& off) {
  const int b = warp_seq_of(c, t);
  if (b < 0) return false;
  const SeqView s = warp_seq_view(c, b);
  const int pos = (int)s.L - s.n + (t - s.q0);
  if (pos < 0 || pos >= (int)s.L) return false;
  pg = page_of(c, b, pos);
  off = (unsigned)pos % (unsigned)c.page_size;
  return pg >= 0;
}

// Rows whose width, strides and addresses allow 16-byte pieces. One warp per
// (new token, kHeadBlock heads): the lower half-warp takes K, the upper V,
// lane l of a half elements 8 l .. 8 l + 7 of every 128 (kCh such pieces).
template <typename TS, bool kQuant, int kCh>
__global__ void __launch_bounds__(256)
cache_write_vec(CacheP c, const TS* k, int64_t snk0, int64_t snk1, const TS* v, int64_t snv0, int64_t snv1) {
  if (blockIdx.x == 0 && blockIdx.y == 0) report_ragged(c);
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), h0 = blockIdx.y * kHeadBlock;
  if (t >= c.rows) return;
  const int lane = threadIdx.x & 31, hl = lane & 15;
  const bool isv = lane >= 16;
  const int width = isv ? c.dv : c.d;
  const TS* src = (isv ? v : k) + (int64_t)t * (isv ? snv0 : snk0);
  const int64_t sh = isv ? snv1 : snk1;
  Vec8<TS> x[kHeadBlock][kCh];
#pragma unroll
  for (int e = 0; e < kHeadBlock; ++e)
#pragma unroll
    for (int ch = 0; ch < kCh; ++ch)
      if (h0 + e < c.Hkv && ch * 128 + hl * 8 < width) x[e][ch].load(src + (h0 + e) * sh + ch * 128 + hl * 8);
  int64_t pg, off;
  if (!slot_of(c, t, pg, off)) return;
  // (strides as selected values: a selected pointer into the parameters would
  // make every use an indexed constant load)
  const int64_t sp = isv ? c.sv[0] : c.sk[0], so = isv ? c.sv[1] : c.sk[1], sc = isv ? c.sv[2] : c.sk[2];
  uint8_t* pool = const_cast<uint8_t*>(static_cast<const uint8_t*>(isv ? c.v : c.k));
  const int64_t base = pg * sp + off * so + (int64_t)h0 * sc;
  [[maybe_unused]] float* scale_at = nullptr;
  [[maybe_unused]] int64_t scale_step = 0;
  if constexpr (kQuant) {
    scale_step = isv ? c.svs[2] : c.sks[2];
    scale_at = const_cast<float*>(isv ? c.vs : c.ks) + pg * (isv ? c.svs[0] : c.sks[0]) +
               off * (isv ? c.svs[1] : c.sks[1]) + (int64_t)h0 * scale_step;
  }
#pragma unroll
  for (int e = 0; e < kHeadBlock; ++e) {
    if (h0 + e >= c.Hkv) break;
    const int64_t row = base + e * sc;
    if constexpr (!kQuant) {
      TS* dst = reinterpret_cast<TS*>(pool) + row;
#pragma unroll
      for (int ch = 0; ch < kCh; ++ch)
        if (ch * 128 + hl * 8 < width) x[e][ch].store(dst + ch * 128 + hl * 8);
    } else {
      float a = 0.f;
#pragma unroll
      for (int ch = 0; ch < kCh; ++ch)
        if (ch * 128 + hl * 8 < width) a = max_nan(a, x[e][ch].top());
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));  // within the half-warp
      bool usual;
      float s = row_scale_usual(a, usual);
      if (!usual) s = row_scale(a);
      const float rs = reciprocal(s);
      uint8_t* dst = pool + row;
#pragma unroll
      for (int ch = 0; ch < kCh; ++ch)
        if (ch * 128 + hl * 8 < width) {
          float f[8];
          x[e][ch].get(f);
          if (usual) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) quotients(f[i], f[i + 1], s, rs);
          } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              // one division in the code, for the element that i selects
              float g = f[0];
#pragma unroll
              for (int b = 1; b < 8; ++b) g = i == b ? f[b] : g;
              g = __fdiv_rn(g, s);
#pragma unroll
              for (int b = 0; b < 8; ++b) f[b] = i == b ? g : f[b];
            }
          }
          uint32_t w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[i] = (uint32_t)e4m3x2(f[4 * i], f[4 * i + 1]) | ((uint32_t)e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16);
          *reinterpret_cast<uint2*>(dst + ch * 128 + hl * 8) = make_uint2(w[0], w[1]);
        }
      if (hl == 0) scale_at[e * scale_step] = s;
    }
  }
}

// Any width and stride: one warp per (new token, head), K then V, element by element.
template <typename TS, bool kQuant>
__global__ void __launch_bounds__(256)
cache_write_any(CacheP c, const TS* k, int64_t snk0, int64_t snk1, const TS* v, int64_t snv0, int64_t snv1) {
  if (blockIdx.x == 0) report_ragged(c);
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (warp >= (int64_t)c.rows * c.Hkv) return;
  const int lane = threadIdx.x & 31;
  const int t = (int)(warp / c.Hkv), h = (int)(warp % c.Hkv);
  int64_t pg, off;
  if (!slot_of(c, t, pg, off)) return;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const TS* src = w ? v + (int64_t)t * snv0 + h * snv1 : k + (int64_t)t * snk0 + h * snk1;
    const int64_t* sc = w ? c.sv : c.sk;
    const int64_t row = pg * sc[0] + off * sc[1] + h * sc[2];
    const int width = w ? c.dv : c.d;
    if constexpr (!kQuant) {
      TS* dst = const_cast<TS*>(static_cast<const TS*>(w ? c.v : c.k)) + row;
      for (int i = lane; i < width; i += 32) dst[i] = src[i];
    } else {
      float a = 0.f;
      for (int i = lane; i < width; i += 32) a = max_nan(a, fabsf(ld(src + i)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s = row_scale(a);
      uint8_t* dst = const_cast<uint8_t*>(static_cast<const uint8_t*>(w ? c.v : c.k)) + row;
      for (int i = lane; i < width; i += 32) dst[i] = (uint8_t)(e4m3x2(__fdiv_rn(ld(src + i), s), 0.f) & 0xffu);
      const int64_t* ss = w ? c.svs : c.sks;
      if (lane == 0) const_cast<float*>(w ? c.vs : c.ks)[pg * ss[0] + off * ss[1] + h * ss[2]] = s;
    }
  }
}

// ------------------------------------------------------------------- read

constexpr int kReadRows = 64;  // positions a block reads: 16 half-warps x 4 each

// Two e4m3 codes times a scale, rounded once to the output type.
template <typename TO>
__device__ __forceinline__ void scaled8(const uint2& u, float scale, Vec8<TO>& out) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = e4m3x2_to_float2((uint16_t)((i < 2 ? u.x : u.y) >> (16 * (i & 1))));
    f[2 * i] = p.x * scale;
    f[2 * i + 1] = p.y * scale;
  }
  out.set(f);
}

// One block per (64 positions, head, sequence), for pages of a multiple of four
// positions. A half-warp reads the four rows at 4 g of the block, which share
// a page: one lookup and one address for the four, K and V of all in flight
// at once. (With a lookup and an address per row the read was bound by
// instructions: 31.7 us for eight e4m3 sequences of up to 4096.)
template <typename TO, bool kQuant, int kCh>
__global__ void __launch_bounds__(256)
cache_read_vec(CacheP c, TO* k, int64_t sk0, int64_t sk1, int64_t sk2, TO* v, int64_t sv0, int64_t sv1, int64_t sv2,
               int T, int jblocks) {
  const unsigned bh = blockIdx.x / (unsigned)jblocks;
  const int b = (int)(bh / (unsigned)c.Hkv), h = (int)(bh % (unsigned)c.Hkv);
  const int g = threadIdx.x >> 4, hl = threadIdx.x & 15;
  const int j = (int)(blockIdx.x % (unsigned)jblocks) * kReadRows + 4 * g;  // the half-warp's first position
  if (blockIdx.x == 0) report_ragged(c);
  const SeqView s = seq_view(c, b);
  const int n = (int)(s.L < T ? s.L : T);
  if (j >= n) return;
  const int64_t pg = page_of(c, b, j);
  if (pg < 0) return;
  const int64_t off = (unsigned)j % (unsigned)c.page_size;
  const int rows = n - j < 4 ? n - j : 4;
  float xs[4], ys[4];
  if constexpr (kQuant) {
    const float* ks = c.ks + pg * c.sks[0] + off * c.sks[1] + h * c.sks[2];
    const float* vs = c.vs + pg * c.svs[0] + off * c.svs[1] + h * c.svs[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      xs[e] = e < rows ? ks[e * c.sks[1]] : 0.f;
      ys[e] = e < rows ? vs[e * c.svs[1]] : 0.f;
    }
  }
#pragma unroll
  for (int ch = 0; ch < kCh; ++ch) {
    const int at = ch * 128 + hl * 8;
    const int64_t kat = pg * c.sk[0] + off * c.sk[1] + h * c.sk[2] + at;
    const int64_t vat = pg * c.sv[0] + off * c.sv[1] + h * c.sv[2] + at;
    TO* ko = k + b * sk0 + h * sk1 + j * sk2 + at;
    TO* vo = v + b * sv0 + h * sv1 + j * sv2 + at;
    const bool hask = at < c.d, hasv = at < c.dv;
    if constexpr (!kQuant) {
      Vec8<TO> x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e < rows && hask) x[e].load(static_cast<const TO*>(c.k) + kat + e * c.sk[1]);
        if (e < rows && hasv) y[e].load(static_cast<const TO*>(c.v) + vat + e * c.sv[1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e < rows && hask) x[e].store(ko + e * sk2);
        if (e < rows && hasv) y[e].store(vo + e * sv2);
      }
    } else {
      uint2 x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e < rows && hask)
          x[e] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + kat + e * c.sk[1]);
        if (e < rows && hasv)
          y[e] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + vat + e * c.sv[1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        Vec8<TO> out;
        if (e < rows && hask) {
          scaled8(x[e], xs[e], out);
          out.store(ko + e * sk2);
        }
        if (e < rows && hasv) {
          scaled8(y[e], ys[e], out);
          out.store(vo + e * sv2);
        }
      }
    }
  }
}

// Any width and stride: one warp per (position, head, sequence).
template <typename TO, typename TC>
__global__ void __launch_bounds__(256)
cache_read_any(CacheP c, TO* k, int64_t sk0, int64_t sk1, int64_t sk2, TO* v, int64_t sv0, int64_t sv1, int64_t sv2,
               int T) {
  if (blockIdx.x == 0) report_ragged(c);
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (warp >= (int64_t)c.batch * c.Hkv * T) return;
  const int lane = threadIdx.x & 31;
  const int j = (int)(warp % T), h = (int)((warp / T) % c.Hkv), b = (int)(warp / ((int64_t)T * c.Hkv));
  if (j >= seq_view(c, b).L) return;
  const int64_t pg = page_of(c, b, j), off = j % c.page_size;
  if (pg < 0) return;
  const float xs = c.ks ? c.ks[pg * c.sks[0] + off * c.sks[1] + h * c.sks[2]] : 1.f;
  const float ys = c.vs ? c.vs[pg * c.svs[0] + off * c.svs[1] + h * c.svs[2]] : 1.f;
  const TC* ck = static_cast<const TC*>(c.k) + pg * c.sk[0] + off * c.sk[1] + h * c.sk[2];
  const TC* cv = static_cast<const TC*>(c.v) + pg * c.sv[0] + off * c.sv[1] + h * c.sv[2];
  for (int i = lane; i < c.d; i += 32) st(k + b * sk0 + h * sk1 + j * sk2 + i, c.ks ? ld(ck + i) * xs : ld(ck + i));
  for (int i = lane; i < c.dv; i += 32) st(v + b * sv0 + h * sv1 + j * sv2 + i, c.vs ? ld(cv + i) * ys : ld(cv + i));
}

// May rows at base with these element strides be moved in pieces of `bytes`?
bool pieces_ok(const void* base, const int64_t* s, int ns, int width, int elem, int bytes) {
  if (reinterpret_cast<uintptr_t>(base) % bytes || width % 8) return false;
  for (int i = 0; i < ns; ++i)
    if ((s[i] * elem) % bytes) return false;
  return true;
}

int elem_bytes(int32_t dt) { return dt == ATTN_F32 ? 4 : dt == ATTN_E4M3 ? 1 : 2; }

bool pool_pieces_ok(const CacheP& c) {
  const int e = elem_bytes(c.dtype), piece = e == 1 ? 8 : 16;
  return pieces_ok(c.k, c.sk, 3, c.d, e, piece) && pieces_ok(c.v, c.sv, 3, c.dv, e, piece);
}

unsigned grid_for(int64_t warps) { return (unsigned)((warps + 7) / 8); }

template <typename TS, bool kQuant>
cudaError_t write_as(const CacheP& c, const void* kv, const int64_t snk[2], const void* vv, const int64_t snv[2],
                     int32_t src_dtype, cudaStream_t st) {
  const TS* k = static_cast<const TS*>(kv);
  const TS* v = static_cast<const TS*>(vv);
  const int e = elem_bytes(src_dtype);
  if (pool_pieces_ok(c) && c.Hkv <= 65535 * kHeadBlock && pieces_ok(k, snk, 2, c.d, e, 16) && pieces_ok(v, snv, 2, c.dv, e, 16)) {
    const dim3 g(grid_for(c.rows), (c.Hkv + kHeadBlock - 1) / kHeadBlock);
    if (c.d <= 128 && c.dv <= 128)
      cache_write_vec<TS, kQuant, 1><<<g, 256, 0, st>>>(c, k, snk[0], snk[1], v, snv[0], snv[1]);
    else
      cache_write_vec<TS, kQuant, (kMaxWidth + 127) / 128><<<g, 256, 0, st>>>(c, k, snk[0], snk[1], v, snv[0], snv[1]);
  } else {
    cache_write_any<TS, kQuant><<<grid_for((int64_t)c.rows * c.Hkv), 256, 0, st>>>(c, k, snk[0], snk[1], v, snv[0],
                                                                                  snv[1]);
  }
  return cudaGetLastError();
}

template <typename TO>
cudaError_t read_as(const CacheP& c, void* kv, const int64_t sok[3], void* vv, const int64_t sov[3], int T,
                    int32_t out_dtype, cudaStream_t st) {
  TO* k = static_cast<TO*>(kv);
  TO* v = static_cast<TO*>(vv);
  const int e = elem_bytes(out_dtype);
  const bool quant = c.dtype == ATTN_E4M3;
  if (pool_pieces_ok(c) && c.page_size % 4 == 0 && pieces_ok(k, sok, 3, c.d, e, 16) && pieces_ok(v, sov, 3, c.dv, e, 16)) {
    const int jb = (T + kReadRows - 1) / kReadRows;
    const unsigned g = (unsigned)((int64_t)jb * c.Hkv * c.batch);
    constexpr int kWide = (kMaxWidth + 127) / 128;
    const bool narrow = c.d <= 128 && c.dv <= 128;
#define ATTN_READ(Q, CH) \
  cache_read_vec<TO, Q, CH><<<g, 256, 0, st>>>(c, k, sok[0], sok[1], sok[2], v, sov[0], sov[1], sov[2], T, jb)
    if (quant) {
      if (narrow) ATTN_READ(true, 1);
      else ATTN_READ(true, kWide);
    } else {
      if (narrow) ATTN_READ(false, 1);
      else ATTN_READ(false, kWide);
    }
#undef ATTN_READ
  } else {
    const unsigned g = grid_for((int64_t)c.batch * c.Hkv * T);
    if (quant)
      cache_read_any<TO, __nv_fp8_e4m3><<<g, 256, 0, st>>>(c, k, sok[0], sok[1], sok[2], v, sov[0], sov[1], sov[2], T);
    else
      cache_read_any<TO, TO><<<g, 256, 0, st>>>(c, k, sok[0], sok[1], sok[2], v, sov[0], sov[1], sov[2], T);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheP& c, const void* k, const int64_t snk[2], const void* v,
                               const int64_t snv[2], int32_t src_dtype, cudaStream_t st) {
  const bool quant = c.dtype == ATTN_E4M3;
  if (src_dtype == ATTN_F32)
    return quant ? write_as<float, true>(c, k, snk, v, snv, src_dtype, st)
                 : write_as<float, false>(c, k, snk, v, snv, src_dtype, st);
  if (src_dtype == ATTN_F16)
    return quant ? write_as<__half, true>(c, k, snk, v, snv, src_dtype, st)
                 : write_as<__half, false>(c, k, snk, v, snv, src_dtype, st);
  return quant ? write_as<__nv_bfloat16, true>(c, k, snk, v, snv, src_dtype, st)
               : write_as<__nv_bfloat16, false>(c, k, snk, v, snv, src_dtype, st);
}

cudaError_t launch_cache_read(const CacheP& c, void* k, const int64_t sok[3], void* v, const int64_t sov[3], int T,
                              int32_t out_dtype, cudaStream_t st) {
  if (out_dtype == ATTN_F32) return read_as<float>(c, k, sok, v, sov, T, out_dtype, st);
  if (out_dtype == ATTN_F16) return read_as<__half>(c, k, sok, v, sov, T, out_dtype, st);
  return read_as<__nv_bfloat16>(c, k, sok, v, sov, T, out_dtype, st);
}

}  // namespace attn
