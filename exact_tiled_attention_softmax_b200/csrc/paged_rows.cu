// Attention of new tokens over a paged cache, one warp per (new token, query
// head): every dtype, head width (<= 576), page size and stride order. The
// path for shapes that the tensor-core kernels do not take, and the simplest
// statement of the operator: per allowed key the score (times the key's scale
// for an e4m3 cache), the running-summary update, and the value row weighted by
// the probability (times the row's scale). Keys no set allows are never read,
// so what their rows hold cannot reach the result.
#include <math.h>

#include "paged.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;

template <typename TQ, typename TC, int N>
__global__ void __launch_bounds__(kWarps * 32) paged_rows_kernel(PagedP p) {
  const CacheP& c = p.c;
  if (blockIdx.x == 0) report_ragged(c);
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (warp >= (int64_t)c.rows * p.Hq) return;
  const int t = (int)(warp / p.Hq), h = (int)(warp % p.Hq);
  const int b = warp_seq_of(c, t);
  if (b < 0) return;
  const SeqView s = warp_seq_view(c, b);
  const int64_t pos = s.L - s.n + (t - s.q0);  // the query's key position
  const int kvh = h / (p.Hq / c.Hkv);
  const TQ* q = static_cast<const TQ*>(p.q) + t * p.sq[0] + h * p.sq[1];
  float qr[N], acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    qr[e] = lane + 32 * e < c.d ? ld(q + lane + 32 * e) : 0.f;
    acc[e] = 0.f;
  }
  const bool window = p.flags & ATTN_MASK_WINDOW;
  int64_t hi = s.L - 1;
  if ((p.flags & ATTN_MASK_CAUSAL) && pos < hi) hi = pos;
  if (t - s.q0 >= s.n || pos < 0) hi = -1;
  const int64_t wlo = window ? pos - p.window + 1 : 0;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j <= hi; ++j) {
    if (j >= p.first && j < wlo) j = wlo;  // from the first keys to the window
    if (j > hi) break;
    const int64_t pg = page_of(c, b, j);
    if (pg < 0) continue;
    const int64_t off = j % c.page_size;
    const TC* kr = static_cast<const TC*>(c.k) + pg * c.sk[0] + off * c.sk[1] + kvh * c.sk[2];
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (lane + 32 * e < c.d) x = fmaf(qr[e], ld(kr + lane + 32 * e), x);
    x = warp_sum(x);
    if (c.ks) x *= c.ks[pg * c.sks[0] + off * c.sks[1] + kvh * c.sks[2]];
    x *= p.scale;
    if (x == -INFINITY) continue;  // exp(-inf): no share
    const float mn = fmaxf(m, x);
    const float alpha = m == -INFINITY && l == 0.f ? 0.f : expf(m - mn);
    const float w = expf(x - mn);
    l = l * alpha + w;
    m = mn;
    const float wv = c.vs ? w * c.vs[pg * c.svs[0] + off * c.svs[1] + kvh * c.svs[2]] : w;
    const TC* vr = static_cast<const TC*>(c.v) + pg * c.sv[0] + off * c.sv[1] + kvh * c.sv[2];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float y = lane + 32 * e < c.dv ? ld(vr + lane + 32 * e) : 0.f;
      acc[e] = fmaf(wv, y, acc[e] * alpha);
    }
  }
  const bool has_sink = p.sink != nullptr;
  const float z = has_sink ? p.sink[h] : -INFINITY;
  const bool empty = l == 0.f;  // a NaN score leaves l NaN, and the row with it
  float lse, osc;
  if (empty) {
    lse = z;
    osc = 0.f;
  } else {
    const float M = has_sink ? fmaxf(m, z) : m;
    const float tot = l * expf(m - M) + (has_sink ? expf(z - M) : 0.f);
    osc = expf(m - M) / tot;
    lse = M + logf(tot);
  }
  TQ* o = static_cast<TQ*>(p.o) + t * p.so[0] + h * p.so[1];
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (lane + 32 * e < c.dv) st(o + lane + 32 * e, empty ? 0.f : acc[e] * osc);
  if (lane == 0) {
    float out = lse;
    if (p.lse_fmt & ATTN_LSE_KV_ONLY) out = empty ? -INFINITY : m + logf(l);
    if (p.lse_fmt & ATTN_LSE_NEG_LOG2) out *= -1.4426950408889634f;
    p.lse[t * p.sl[0] + h * p.sl[1]] = out;
  }
}

template <typename TQ, typename TC>
cudaError_t launch_width(const PagedP& p, cudaStream_t st) {
  const int w = p.c.d > p.c.dv ? p.c.d : p.c.dv;
  const unsigned g = (unsigned)(((int64_t)p.c.rows * p.Hq + kWarps - 1) / kWarps);
  if (w <= 64)
    paged_rows_kernel<TQ, TC, 2><<<g, kWarps * 32, 0, st>>>(p);
  else if (w <= 128)
    paged_rows_kernel<TQ, TC, 4><<<g, kWarps * 32, 0, st>>>(p);
  else
    paged_rows_kernel<TQ, TC, 18><<<g, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename TQ>
cudaError_t launch_types(const PagedP& p, cudaStream_t st) {
  return p.c.dtype == ATTN_E4M3 ? launch_width<TQ, __nv_fp8_e4m3>(p, st) : launch_width<TQ, TQ>(p, st);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedP& p, cudaStream_t st) {
  if (p.dtype == ATTN_F32) return launch_types<float>(p, st);
  if (p.dtype == ATTN_F16) return launch_types<__half>(p, st);
  return launch_types<__nv_bfloat16>(p, st);
}

}  // namespace attn
