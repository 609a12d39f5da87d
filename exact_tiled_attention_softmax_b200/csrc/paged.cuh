// Paged K/V caches: the parameter block that every paged kernel takes, the
// checked view of one sequence, and the launchers (internal; the C entry
// points are in api.cu).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace attn {

struct CacheP {
  const void* k;  // [num_pages, page_size, Hkv, d] (write: also the destination)
  const void* v;
  int64_t sk[3], sv[3];    // strides of (page, position in page, head), in elements
  const float* ks;         // scales [num_pages, page_size, Hkv], null unless dtype is ATTN_E4M3
  const float* vs;
  int64_t sks[3], svs[3];
  const int32_t* table;    // [batch, max_pages]
  int64_t table_stride;
  int32_t max_pages, num_pages, page_size, batch;
  const int32_t* lens;     // [batch]
  int32_t Hkv, d, dv;
  int32_t dtype;           // attn_dtype of the pool
  const int32_t* cu_q;     // [batch + 1] or null: rows / batch new tokens each
  int32_t rows;            // new tokens in all
  uint32_t* status;        // may be null
};

struct PagedP {
  CacheP c;
  const void* q;  // [rows, Hq, d]
  int64_t sq[2];
  void* o;        // [rows, Hq, dv]
  int64_t so[2];
  float* lse;     // [rows, Hq]
  int64_t sl[2];
  int32_t Hq;
  int32_t dtype;  // attn_dtype of q and o
  uint32_t flags; // ATTN_MASK_CAUSAL | WINDOW | FIRST
  int64_t window, first;
  const float* sink;
  uint32_t lse_fmt;
  float scale;
};

// One sequence's new tokens [q0, q0 + n) and cached length L, clamped into
// range whatever the device arrays hold.
struct SeqView {
  int q0, n;
  int64_t L;
};

__device__ __forceinline__ SeqView seq_view(const CacheP& c, int b) {
  SeqView s;
  int lo, hi;
  if (c.cu_q) {
    lo = c.cu_q[b];
    hi = c.cu_q[b + 1];
    lo = lo < 0 ? 0 : (lo > c.rows ? c.rows : lo);
    hi = hi < 0 ? 0 : (hi > c.rows ? c.rows : hi);
  } else {
    const int each = c.rows / c.batch;
    lo = b * each;
    hi = lo + each;
  }
  s.q0 = lo;
  s.n = hi > lo ? hi - lo : 0;
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  const int64_t L = c.lens[b];
  s.L = L < 0 ? 0 : (L > cap ? cap : L);
  return s;
}

// The same for a whole (converged) warp: one reading, so that its lanes agree even
// while someone else writes the arrays.
__device__ __forceinline__ SeqView warp_seq_view(const CacheP& c, int b) {
  SeqView s = seq_view(c, b);
  s.q0 = __shfl_sync(0xffffffffu, s.q0, 0);
  s.n = __shfl_sync(0xffffffffu, s.n, 0);
  s.L = __shfl_sync(0xffffffffu, (int)s.L, 0);  // below 2^30
  return s;
}

// Reports cu_q and seq_lens entries that seq_view clamps, or whose new tokens
// do not fit their sequence. For one block of a launch, all threads.
__device__ __forceinline__ void report_ragged(const CacheP& c, uint32_t* status) {
  if (!status) return;
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  bool bad = false;
  for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
    const int64_t L = c.lens[b];
    const int64_t lo = c.cu_q ? c.cu_q[b] : 0, hi = c.cu_q ? c.cu_q[b + 1] : (c.rows / c.batch);
    bad = bad || L < 0 || L > cap || lo < 0 || hi < lo || hi > c.rows || hi - lo > L;
  }
  if (bad) set_status(status, ATTN_DEVERR_RAGGED);
}
__device__ __forceinline__ void report_ragged(const CacheP& c) { report_ragged(c, c.status); }

// The sequence that holds new token t, found by the whole (converged) warp:
// the number of sequences that end at or before t. -1 when none does.
__device__ __forceinline__ int warp_seq_of(const CacheP& c, int t) {
  if (!c.cu_q) {
    const int each = c.rows / c.batch;
    return t / each < c.batch ? t / each : -1;
  }
  const int lane = threadIdx.x & 31;
  int b = 0;  // (the same in every lane: it counts ballots)
  for (int b0 = 0; b0 < c.batch; b0 += 32) {
    const bool ends = b0 + lane < c.batch && c.cu_q[b0 + lane + 1] <= t;
    b += __popc(__ballot_sync(0xffffffffu, ends));
  }
  if (b >= c.batch) return -1;
  return __all_sync(0xffffffffu, c.cu_q[b] <= t && t < c.cu_q[b + 1]) ? b : -1;
}

// The page that holds position pos (below 2^30) of sequence b, or -1 when the table names
// a page outside the pool (reported).
__device__ __forceinline__ int64_t page_of(const CacheP& c, int b, int64_t pos) {
  const int64_t pg = c.table[(int64_t)b * c.table_stride + (unsigned)pos / (unsigned)c.page_size];
  if (pg < 0 || pg >= c.num_pages) {
    set_status(c.status, ATTN_DEVERR_PAGE);
    return -1;
  }
  return pg;
}

__device__ __forceinline__ float ld(const __nv_fp8_e4m3* p) { return float(*p); }

cudaError_t launch_cache_write(const CacheP& c, const void* k, const int64_t snk[2], const void* v,
                               const int64_t snv[2], int32_t src_dtype, cudaStream_t st);
cudaError_t launch_cache_read(const CacheP& c, void* k, const int64_t sok[3], void* v, const int64_t sov[3], int T,
                              int32_t out_dtype, cudaStream_t st);
// Any head width up to 576, page size, dtype and stride: one warp per (row, head).
cudaError_t launch_paged_rows(const PagedP& p, cudaStream_t st);

}  // namespace attn
