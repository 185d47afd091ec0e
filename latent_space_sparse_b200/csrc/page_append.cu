// page_append.cu -- append to the paged 8-bit cache: rotation, scales, codes.
//
// For every page that the step touches and every KV head, keys and values
// apart:
//   x_t   = RoPE(K_new[t], position)            or V_new[t]
//   a     = max over the page's new tokens of |k_i| + |k_{i+d/2}| (keys that
//           are rotated: it bounds sqrt(k_i^2 + k_{i+d/2}^2), which the
//           rotation keeps, so the scale follows from the inputs alone and
//           does not depend on how an angle rounds), or of |k|, |v|
//   scale = 2^e, the least e with a <= 448 * 2^e, and no less than the page's
//           scale where it holds earlier tokens
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
// 8-byte stores.  A CTA takes one page and every gridDim.y-th group of its
// items, so that the cos/sin table of the page's positions is computed once
// per CTA and not once per head.
#include "page.cuh"

namespace salsc {
namespace {

constexpr int kMinExp = -100;  // exponent of the scale of a page that holds only zeros
constexpr int kTargetCtas = 2 * 148;

// The least 2^e >= a / 448, e >= kMinExp (a finite, >= 0).  448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kMinExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_or_zero(float x) { return fabsf(x) <= 3.402823466e38f ? fabsf(x) : 0.f; }

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *(const uint4*)p;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
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
// pages at most, head parts).
template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads)
page_append_kernel(const __grid_constant__ PageStep s, const T* __restrict__ K, int64_t k_stride,
                   const T* __restrict__ V, int64_t v_stride, uint8_t* __restrict__ k_pages,
                   uint8_t* __restrict__ v_pages, float* __restrict__ k_scales,
                   float* __restrict__ v_scales) {
  extern __shared__ float2 cs[];  // [T][D/2] cos, sin of the new tokens' slots
  __shared__ int find[34];
  __shared__ float red[kThreads / 32];
  constexpr int kHalf = D / 2;
  constexpr int kRowChunks = D / 16;  // 16-element chunks of a row
  const int tid = threadIdx.x;
  grid_dependency_wait();
  allow_dependent_launch();

  // the x-th touched page of the step
  int b, j;
  page_find(s.B, blockIdx.x, find, [&](int i) {
    const PageSeq q = page_seq(s, i);
    const int m = min(q.m, q.n);
    return m > 0 ? (q.n - 1) / s.T - (q.n - m) / s.T + 1 : 0;
  }, b, j);
  if (b < 0) return;
  const PageSeq q = page_seq(s, b);
  const int m = min(q.m, q.n), start = q.n - m;
  j += start / s.T;
  const int pg = page_of(s, b, j);
  if (pg < 0) return;
  const int lo = max(start - j * s.T, 0), hi = min(q.n - j * s.T, s.T);  // new slots
  // row of slot 0 (may lie before the first new row)
  const int64_t row0 = (int64_t)q.row0 + (q.m - m) + ((int64_t)j * s.T - start);

  if (s.rotate) {
    for (int e = tid; e < (hi - lo) * kHalf; e += kThreads) {
      const int slot = lo + e / kHalf, i = e % kHalf;
      float c, sn;
      page_cs(j * s.T + slot, s.turns[i], c, sn);
      cs[slot * kHalf + i] = make_float2(c, sn);
    }
  }
  __syncthreads();

  const int per = s.T * D / 32;       // threads of an item
  const int items = kThreads / per;   // items of a pass
  const int ti = tid % per, warps = per / 32;
  for (int it0 = blockIdx.y * items; it0 < 2 * s.U; it0 += gridDim.y * items) {
    const int it = it0 + tid / per;
    const bool live = it < 2 * s.U;
    const bool val = it >= s.U;  // keys first, then values
    const int u = val ? it - s.U : it;
    const T* X = val ? V : K;
    const int64_t stride = val ? v_stride : k_stride;
    const bool turn = s.rotate && !val;
    float x[2][2][8];
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int ch = ti + k * per, slot = ch / kRowChunks, i0 = ch % kRowChunks * 8;
      if (live && slot >= lo && slot < hi) {
        const T* p = X + (row0 + slot) * stride + u * D + i0;
        load8(p, x[k][0]);
        load8(p + kHalf, x[k][1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a0 = finite_or_zero(x[k][0][i]), a1 = finite_or_zero(x[k][1][i]);
          a = fmaxf(a, turn ? fminf(__fadd_rn(a0, a1), 3.402823466e38f) : fmaxf(a0, a1));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (warps > 1) {
      if ((tid & 31) == 0) red[tid >> 5] = a;
      __syncthreads();
      const int w0 = (tid >> 5) / warps * warps;
      for (int w = 0; w < warps; ++w) a = fmaxf(a, red[w0 + w]);
      __syncthreads();
    }
    if (!live) continue;
    float* scales = (val ? v_scales : k_scales) + (size_t)pg * s.U + u;
    uint8_t* page = (val ? v_pages : k_pages) + ((size_t)pg * s.U + u) * s.T * D;
    float sc = pow2_scale(a), ratio = 1.f;
    if (lo > 0) {
      const float old = *scales;
      if (old > 0.f && old <= 3.402823466e38f) {
        ratio = old / sc;
        if (ratio >= 1.f) {
          sc = old;
          ratio = 1.f;
        }
      }
    }
    const float inv = 1.f / sc;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int ch = ti + k * per, slot = ch / kRowChunks, i0 = ch % kRowChunks * 8;
      uint8_t* row = page + slot * D + i0;
      if (slot >= lo && slot < hi) {
        if (turn) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 r = cs[slot * kHalf + i0 + i];
            const float x0 = x[k][0][i], x1 = x[k][1][i];
            x[k][0][i] = x0 * r.x - x1 * r.y;
            x[k][1][i] = x1 * r.x + x0 * r.y;
          }
        }
        *(uint2*)row = codes8(x[k][0], inv);
        *(uint2*)(row + kHalf) = codes8(x[k][1], inv);
      } else if (slot < lo && ratio != 1.f) {
        *(uint2*)row = recode8(*(const uint2*)row, ratio);
        *(uint2*)(row + kHalf) = recode8(*(const uint2*)(row + kHalf), ratio);
      }
    }
    // every thread of the item has read the old scale before one of them writes it
    if (warps > 1) {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + tid / per), "r"(per) : "memory");
    } else {
      __syncwarp();
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
  const size_t smem = sizeof(float2) * s.T * (D / 2);
  const cudaError_t e = ensure_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  // a sequence with m new tokens touches at most floor((m + T - 2) / T) + 1 <= m pages
  int64_t pages = s.B;
  if (s.offs) {
    pages = (int64_t)s.n_tokens / s.T + 2 * (int64_t)s.B;
    if (pages > s.n_tokens) pages = s.n_tokens;
  }
  const int per = s.T * D / 32, passes = (2 * s.U * per + kThreads - 1) / kThreads;
  int64_t parts = (kTargetCtas + pages - 1) / pages;
  if (parts > passes) parts = passes;
  return launch_k(kern, dim3((unsigned)pages, (unsigned)parts), dim3(kThreads), smem, stream, true,
                  s, (const T*)K, k_stride, (const T*)V, v_stride, (uint8_t*)k_pages,
                  (uint8_t*)v_pages, k_scales, v_scales);
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
