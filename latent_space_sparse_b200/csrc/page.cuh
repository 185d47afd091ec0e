// page.cuh -- the paged 8-bit cache: plan, arguments and device helpers shared
// by the append (page_append.cu), the attention (page_attend.cu) and the
// entry points (page_api.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace salsc {

constexpr int kPageMaxGroup = 16;   // query heads per KV head
constexpr int kPageMaxHeadDim = 128;

// One step's sizes, pointers to the caller's lengths and tables, and the
// rotation's frequencies: passed to the kernels by value.
struct PageStep {
  int B, Hq, U, G, d, T;  // batch, query heads, KV heads, heads per KV head, head dim, page size
  int n_pages, max_pages, n_tokens, max_q;
  int window;  // 0: none
  int rotate;  // 0: keys and queries are taken as they are
  float scale;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* offs;  // null: row b is sequence b's one token
  uint32_t* flags;
  // frequency of pair i in turns per position: base^(-2i/d) / 2pi
  double turns[kPageMaxHeadDim / 2];
};

// One sequence's part of a step, cut to the step's bounds.
struct PageSeq {
  int n;     // tokens in the cache, new ones included
  int m;     // new tokens (at most max_q)
  int row0;  // row of the first of them
};

__device__ __forceinline__ PageSeq page_seq(const PageStep& s, int b) {
  PageSeq q;
  bool bad = false;
  q.n = s.lens[b];
  const int cap = s.max_pages * s.T;
  if (q.n < 0 || q.n > cap) {
    bad = true;
    q.n = q.n < 0 ? 0 : cap;
  }
  if (s.offs) {
    int o0 = s.offs[b], o1 = s.offs[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > s.n_tokens) {
      bad = true;
      o0 = min(max(o0, 0), s.n_tokens);
      o1 = min(max(o1, o0), s.n_tokens);
    }
    q.row0 = o0;
    q.m = o1 - o0;
    if (q.m > s.max_q) {
      bad = true;
      q.m = s.max_q;
    }
  } else {
    q.row0 = b;
    q.m = 1;
  }
  if (bad) atomicOr(s.flags, FLAG_BAD_INDEX);
  return q;
}

// Page j of sequence b, or -1 (and the anomaly flag) for an entry outside the pool.
__device__ __forceinline__ int page_of(const PageStep& s, int b, int j) {
  const int pg = s.table[(size_t)b * s.max_pages + j];
  if ((unsigned)pg < (unsigned)s.n_pages) return pg;
  atomicOr(s.flags, FLAG_BAD_INDEX);
  return -1;
}

// Block-wide: item x of a list in which sequence b has count(b) items; the
// sequence (-1 when x is past the end) and the item's index in it.  `sm`: 34
// ints of shared memory.  Every thread calls it, with the same x.
template <typename F>
__device__ __forceinline__ void page_find(int B, int x, int* sm, F count, int& b_out, int& r_out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) sm[32] = -1;
  int left = x;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + tid;
    const int c = b < B ? count(b) : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += sm[w];
      total += sm[w];
    }
    const int end = before + inc;
    if (left >= end - c && left < end) {
      sm[32] = b;
      sm[33] = left - (end - c);
    }
    __syncthreads();
    if (left < total) break;
    left -= total;
  }
  __syncthreads();
  b_out = sm[32];
  r_out = sm[33];
}

// cos and sin of position pos at `turns` turns per position: the angle is
// formed and reduced to half a turn in fp64, so that far positions keep fp32's
// accuracy.
__device__ __forceinline__ void page_cs(int pos, double turns, float& c, float& s) {
  const double a = (double)pos * turns;
  sincospif((float)(2.0 * (a - rint(a))), &s, &c);
}

// Host side: launchers.
cudaError_t launch_page_append(const PageStep& s, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, void* k_pages, void* v_pages, float* k_scales,
                               float* v_scales, salsc_dtype dt, cudaStream_t stream);
cudaError_t launch_page_attend(const PageStep& s, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void* part, salsc_dtype dt,
                               cudaStream_t stream);
size_t page_attend_workspace(const PageStep& s, salsc_dtype dt);

}  // namespace salsc
