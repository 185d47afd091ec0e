// page_append.cu -- append to the paged 8-bit cache: rotation, scales, codes.
//
// For every page that the step touches and every KV head, keys and values
// apart:
//   x_t   = RoPE(K_new[t], position)            or V_new[t]
//   a     = max over the page's new tokens of |k_i| + |k_{i+d/2}| (keys that
//           are rotated: it bounds sqrt(k_i^2 + k_{i+d/2}^2), which the
//           rotation keeps, so the scale follows from the inputs alone and
//           does not depend on how an angle rounds), or of |k|, |v|
//   scale = 2^e, the least e with a <= 448 * 2^e, and no less than the size of
//           the page's scale where it holds earlier tokens
//   code  = e4m3(x / scale)
// A power of two costs e4m3 nothing (its relative step is the same at every
// scale; at most one of its 16 binades is left unused) and makes growth cheap:
// recoding an earlier token with a larger power of two is exact unless the
// value falls below the normal range, 2^-6 of the new scale.
//
// The work is one pass over memory: 2 (or 4) bytes in and 1 byte out per
// element.  One (page, head, K or V) item is T x d elements on T*d/32 threads,
// 32 elements a thread held in registers between the maximum and the codes.
// A thread's 16-element chunks are 8 elements of either half of a row, so a
// rotated pair is one thread's and global accesses are 16-byte loads and
// 8-byte stores.  A CTA takes some items of one page; how many is a balance:
// cos and sin of the page's positions are computed once per CTA, and few items
// to a CTA keep more loads in flight, with the loads issued before cos and sin
// are computed.
//
// What bounds it: instructions, half of the issue slots, and the latency of the
// loads.  16.7K tokens of prompts (8 heads of 128, bf16): 30 us, 3.3 TB/s (28.2 us
// from a graph); with sizes taken one by one and fp64 angles it was 47.  Single
// tokens, from a graph: 3.5 us for 4 sequences of 8 heads, one dependent load after
// another (lengths, table, the page's scale beside the new values); 7.6 for 64 of 32
// heads, where an item's threads are those of a whole page and most have no token.
#include <algorithm>

#include "page.cuh"

namespace salsc {
namespace {

constexpr int kMinExp = -100;  // exponent of the scale of a page that holds only zeros
constexpr int kTargetCtas = 4 * 148;  // CTAs that run at once (64 registers of 256 threads each)

// The least 2^e >= a / 448, e >= kMinExp (a finite, >= 0).  448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kMinExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_or_zero(float x) { return fabsf(x) <= 3.402823466e38f ? fabsf(x) : 0.f; }
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldg((const uint4*)p + i);
  return r;
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x), x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z), x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The larger of a and the elements' sizes; NaN if one of them is.
__device__ __forceinline__ float max_size(const Raw8<float>& r, float a) {
  float x[8];
  widen8(r, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(x[i]));
  return a;
}
__device__ __forceinline__ float max_size(const Raw8<__nv_bfloat16>& r, float a) {
  auto two = [](uint32_t w) { return __habs2(*(const __nv_bfloat162*)&w); };
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(two(r.v[0].x), two(r.v[0].y)),
                                       __hmax2_nan(two(r.v[0].z), two(r.v[0].w)));
  return max_nan(a, max_nan(__low2float(m), __high2float(m)));
}
// The larger of a and the sums of sizes of pairs.
template <typename T>
__device__ __forceinline__ float max_pair(const Raw8<T>& r0, const Raw8<T>& r1, float a) {
  float x[8], y[8];
  widen8(r0, x);
  widen8(r1, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(x[i]) + fabsf(y[i]));
  return a;
}
// The same for any values: what is not finite does not count.
template <typename T>
__device__ __noinline__ float max_finite(const Raw8<T> r0, const Raw8<T> r1, bool pairs) {
  float x[8], y[8], a = 0.f;
  widen8(r0, x);
  widen8(r1, y);
  for (int i = 0; i < 8; ++i) {
    const float x0 = finite_or_zero(x[i]), y0 = finite_or_zero(y[i]);
    a = fmaxf(a, pairs ? fminf(x0 + y0, 3.402823466e38f) : fmaxf(x0, y0));
  }
  return a;
}

__device__ __forceinline__ uint2 codes8(float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mul2(x[2 * i], x[2 * i + 1], inv);
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Two pairs (a, b) rotated.
__device__ __forceinline__ void turn2(float& a0, float& a1, float& b0, float& b1, float c0, float c1,
                                      float s0, float s1) {
  asm("{\n\t.reg .b64 a, b, c, s, m, n, p, q;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
      "mov.b64 s, {%6, %7};\n\tmov.b64 n, {%8, %9};\n\t"
      "mul.rn.f32x2 m, a, c;\n\tfma.rn.f32x2 m, b, n, m;\n\t"
      "mul.rn.f32x2 p, b, c;\n\tfma.rn.f32x2 p, a, s, p;\n\t"
      "mov.b64 {%0, %1}, m;\n\tmov.b64 {%2, %3}, p;\n\t}"
      : "+f"(a0), "+f"(a1), "+f"(b0), "+f"(b1)
      : "f"(c0), "f"(c1), "f"(s0), "f"(s1), "f"(-s0), "f"(-s1));
}

__device__ __forceinline__ uint2 recode8(uint2 v, float ratio) {
  float x[8];
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  return codes8(x, ratio);
}

// D: head dim.  Block of 256 threads (512 for T * D = 16384); grid (touched
// pages at most, parts of a page's items).
template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 1024 : 768) / kThreads)
page_append_kernel(const __grid_constant__ PageStep s, const T* __restrict__ K, int64_t k_stride,
                   const T* __restrict__ V, int64_t v_stride, uint8_t* __restrict__ k_pages,
                   uint8_t* __restrict__ v_pages, float* __restrict__ k_scales,
                   float* __restrict__ v_scales, int part) {
  extern __shared__ __align__(16) float cs[];  // [T][D/2] cos of the new tokens' slots, [T][D/2] sin
  __shared__ float red[2][kThreads / 32];
  constexpr int kHalf = D / 2;
  constexpr int kRowChunks = D / 16;  // 16-element chunks of a row
  const int tid = threadIdx.x;
  grid_dependency_wait();
  allow_dependent_launch();

  // the x-th touched page of the step; without offsets a sequence touches one
  int b = blockIdx.x, j = 0;
  if (s.offs) {
    int64_t x;
    int b0;
    const bool any = page_find(
        s.B,
        [&](int i) -> int64_t {
          const PageSeq q = page_seq<false>(s, i);
          const int m = min(q.m, q.n);
          return m > 0 ? ((q.n - 1) >> s.log_t) - ((q.n - m) >> s.log_t) + 1 : 0;
        },
        [&](int64_t) { return (int64_t)blockIdx.x; }, x, b, b0);
    if (!any) return;
    j = (int)x;
  }
  const PageSeq q = page_seq<false>(s, b);
  const int m = min(q.m, q.n), start = q.n - m;
  if (m <= 0) return;
  j += start >> s.log_t;
  const int pg = page_of<false>(s, b, j);
  if (pg < 0) return;
  const int lo = max(start - j * s.T, 0), hi = min(q.n - j * s.T, s.T);  // new slots
  // row of slot 0 (may lie before the first new row)
  const int64_t row0 = (int64_t)q.row0 + (q.m - m) + ((int64_t)j * s.T - start);

  constexpr int kLogD = D == 128 ? 7 : 6, kLogThreads = kThreads == 512 ? 9 : 8;
  const int log_per = s.log_t + kLogD - 5, per = 1 << log_per;  // threads of an item
  const int log_items = kLogThreads - log_per, items = 1 << log_items;  // items of a pass
  const int ti = tid & (per - 1), warps = per >> 5;
  // this CTA's passes over the page's items, keys first, then values
  const int passes = (2 * s.U + items - 1) >> log_items;
  const int first = blockIdx.y * part, last = min(first + part, passes);
  for (int pass = first; pass < last; ++pass) {
    const int it = pass * items + (tid >> log_per);
    const bool live = it < 2 * s.U;
    const bool val = it >= s.U;
    const int u = val ? it - s.U : it;
    const T* X = val ? V : K;
    const int64_t stride = val ? v_stride : k_stride;
    const bool turn = s.rotate && !val;
    float* scales = (val ? v_scales : k_scales) + (size_t)pg * s.U + u;
    uint8_t* page = (val ? v_pages : k_pages) + ((size_t)pg * s.U + u) * s.T * D;
    Raw8<T> x[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int ch = ti + k * per, slot = ch / kRowChunks, i0 = ch % kRowChunks * 8;
      if (live && slot >= lo && slot < hi) {
        const T* p = X + (row0 + slot) * stride + u * D + i0;
        x[k][0] = load8(p);
        x[k][1] = load8(p + kHalf);
      }
    }
    float old = 0.f;
    if (live && lo > 0) old = *scales;
    if (pass == first) {
      // with the first loads in flight
      if (s.rotate && pass * items < s.U) {
        for (int e = tid; e < (hi - lo) * kHalf; e += kThreads) {
          const int slot = lo + e / kHalf, i = e % kHalf;
          float c, sn;
          page_cs(j * s.T + slot, s.turns[i], c, sn);
          cs[slot * kHalf + i] = c;
          cs[(s.T + slot) * kHalf + i] = sn;
        }
      }
      __syncthreads();
    }
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int slot = (ti + k * per) / kRowChunks;
      if (live && slot >= lo && slot < hi)
        a = turn ? max_pair(x[k][0], x[k][1], a) : max_size(x[k][1], max_size(x[k][0], a));
    }
    if (!(a <= 3.402823466e38f)) {
      a = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int slot = (ti + k * per) / kRowChunks;
        if (live && slot >= lo && slot < hi) a = fmaxf(a, max_finite(x[k][0], x[k][1], turn));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    // the item's threads meet; each has read the old scale before one of them writes it
    if (warps > 1) {
      float* r = red[pass & 1];
      if ((tid & 31) == 0) r[tid >> 5] = a;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + (tid >> log_per)), "r"(per) : "memory");
      const int w0 = (tid >> 5) & -warps;
      for (int w = 0; w < warps; ++w) a = fmaxf(a, r[w0 + w]);
    } else {
      __syncwarp();
    }
    if (!live) continue;
    old += old - old;  // NaN if it is not finite: then it does not count, and earlier codes become NaN
    const float sc = fmaxf(pow2_scale(a), fabsf(old)), inv = 1.f / sc;
    if (lo > 0 && old != sc) {  // earlier codes stand for code * old, whatever its sign
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int ch = ti + k * per, slot = ch / kRowChunks, i0 = ch % kRowChunks * 8;
        uint8_t* row = page + slot * D + i0;
        if (slot < lo) {
          *(uint2*)row = recode8(*(const uint2*)row, old * inv);
          *(uint2*)(row + kHalf) = recode8(*(const uint2*)(row + kHalf), old * inv);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int ch = ti + k * per, slot = ch / kRowChunks, i0 = ch % kRowChunks * 8;
      uint8_t* row = page + slot * D + i0;
      if (slot >= lo && slot < hi) {
        float y[2][8];
        widen8(x[k][0], y[0]);
        widen8(x[k][1], y[1]);
        if (turn) {
          const float* c = cs + slot * kHalf + i0;
          const float* sn = c + s.T * kHalf;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 c4 = *(const float4*)(c + i), s4 = *(const float4*)(sn + i);
            turn2(y[0][i], y[0][i + 1], y[1][i], y[1][i + 1], c4.x, c4.y, s4.x, s4.y);
            turn2(y[0][i + 2], y[0][i + 3], y[1][i + 2], y[1][i + 3], c4.z, c4.w, s4.z, s4.w);
          }
        }
        *(uint2*)row = codes8(y[0], inv);
        *(uint2*)(row + kHalf) = codes8(y[1], inv);
      }
    }
    if (ti == 0) *scales = sc;
  }
}

template <typename T, int D, int kThreads>
cudaError_t launch(const PageStep& s, const void* K, int64_t k_stride, const void* V,
                   int64_t v_stride, void* k_pages, void* v_pages, float* k_scales,
                   float* v_scales, cudaStream_t stream) {
  static int done[kMaxDevices];
  auto kern = page_append_kernel<T, D, kThreads>;
  const size_t smem = 2 * sizeof(float) * s.T * (D / 2);
  const cudaError_t e = ensure_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  // a sequence with m new tokens touches at most floor((m + T - 2) / T) + 1 <= m pages
  int64_t pages = s.B;
  if (s.offs) {
    pages = (int64_t)s.n_tokens / s.T + 2 * (int64_t)s.B;
    if (pages > s.n_tokens) pages = s.n_tokens;
  }
  const int per = s.T * D / 32, items = kThreads / per, passes = (2 * s.U + items - 1) / items;
  // Passes of a CTA: so many that it computes one cos and sin a thread for
  // each (16.7K tokens, pages of 16, when it was chosen: four passes 28.8 us, two
  // 29.9, one 33.2); fewer where the step is small and CTAs would be missing (64
  // single tokens of 32 heads: two passes 7.6 us, one 8.9).
  int64_t part = std::max(1, s.T * (D / 2) / kThreads);
  part = std::min(part, std::max<int64_t>(1, (passes * pages + kTargetCtas - 1) / kTargetCtas));
  const int64_t parts = (passes + part - 1) / part;
  return launch_k(kern, dim3((unsigned)pages, (unsigned)parts), dim3(kThreads), smem, stream, true,
                  s, (const T*)K, k_stride, (const T*)V, v_stride, (uint8_t*)k_pages,
                  (uint8_t*)v_pages, k_scales, v_scales, (int)part);
}

template <typename T>
cudaError_t launch_t(const PageStep& s, const void* K, int64_t k_stride, const void* V,
                     int64_t v_stride, void* k_pages, void* v_pages, float* k_scales,
                     float* v_scales, cudaStream_t stream) {
  if (s.d == 64)
    return launch<T, 64, 256>(s, K, k_stride, V, v_stride, k_pages, v_pages, k_scales, v_scales,
                              stream);
  if (s.T == 128)
    return launch<T, 128, 512>(s, K, k_stride, V, v_stride, k_pages, v_pages, k_scales, v_scales,
                               stream);
  return launch<T, 128, 256>(s, K, k_stride, V, v_stride, k_pages, v_pages, k_scales, v_scales,
                             stream);
}

}  // namespace

cudaError_t launch_page_append(const PageStep& s, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, void* k_pages, void* v_pages, float* k_scales,
                               float* v_scales, salsc_dtype dt, cudaStream_t stream) {
  return dt == SALSC_BF16 ? launch_t<__nv_bfloat16>(s, K, k_stride, V, v_stride, k_pages, v_pages,
                                                    k_scales, v_scales, stream)
                          : launch_t<float>(s, K, k_stride, V, v_stride, k_pages, v_pages, k_scales,
                                            v_scales, stream);
}

}  // namespace salsc
