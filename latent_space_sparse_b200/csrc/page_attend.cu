// page_attend.cu -- attention over the paged 8-bit cache, plain form: one CTA
// per (new token, KV head), fp32 arithmetic on the CUDA cores.
#include "page.cuh"

namespace salsc {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 128;

__device__ __forceinline__ float code_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
page_attend_kernel(const __grid_constant__ PageStep s, const T* __restrict__ q, int64_t q_stride,
                   const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   T* __restrict__ out) {
  __shared__ int find[34];
  __shared__ float qr[kPageMaxGroup][D];
  __shared__ float p[kPageMaxGroup][kTile];
  __shared__ float m_s[kPageMaxGroup], l_s[kPageMaxGroup], al_s[kPageMaxGroup];
  __shared__ int pages[kTile];
  const int tid = threadIdx.x, u = blockIdx.y, G = s.G;
  grid_dependency_wait();
  allow_dependent_launch();
  int b, i;
  page_find(s.B, blockIdx.x, find, [&](int x) { return page_seq(s, x).m; }, b, i);
  if (b < 0) return;
  const PageSeq sq = page_seq(s, b);
  const int pos = sq.n - sq.m + i, end = pos + 1;
  const int beg = s.window ? max(0, end - s.window) : 0;
  const int64_t row = sq.row0 + i;
  for (int e = tid; e < G * (D / 2); e += kThreads) {
    const int g = e / (D / 2), k = e % (D / 2);
    const T* x = q + row * q_stride + (u * G + g) * D;
    float c = 1.f, sn = 0.f;
    if (s.rotate) page_cs(pos, s.turns[k], c, sn);
    const float x0 = to_f32(x[k]), x1 = to_f32(x[k + D / 2]);
    qr[g][k] = (x0 * c - x1 * sn) * s.scale;
    qr[g][k + D / 2] = (x1 * c + x0 * sn) * s.scale;
  }
  if (tid < G) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  float acc[kPageMaxGroup];
  for (int g = 0; g < kPageMaxGroup; ++g) acc[g] = 0.f;
  for (int t0 = beg / kTile * kTile; t0 < end; t0 += kTile) {
    __syncthreads();
    const int t = t0 + tid;
    int pg = -1;
    if (t >= beg && t < end) pg = page_of(s, b, t / s.T);
    pages[tid] = pg;
    const size_t base = ((size_t)max(pg, 0) * s.U + u) * s.T + t % s.T;
    const float sc = pg >= 0 ? ks[(size_t)pg * s.U + u] : 0.f;
    for (int g = 0; g < G; ++g) {
      float dot = 0.f;
      if (pg >= 0)
        for (int k = 0; k < D; ++k) dot = fmaf(qr[g][k], code_f32(kp[base * D + k]), dot);
      p[g][tid] = pg >= 0 ? dot * sc : -INFINITY;
    }
    __syncthreads();
    if (tid < G) {
      float m = m_s[tid];
      for (int k = 0; k < kTile; ++k) m = fmaxf(m, p[tid][k]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float al = expf(m_s[tid] - ref);
      float l = l_s[tid] * al;
      for (int k = 0; k < kTile; ++k) {
        p[tid][k] = expf(p[tid][k] - ref);
        l += p[tid][k];
      }
      m_s[tid] = m;
      l_s[tid] = l;
      al_s[tid] = al;
    }
    __syncthreads();
    if (tid < D) {
      for (int g = 0; g < G; ++g) acc[g] *= al_s[g];
      for (int k = 0; k < kTile; ++k) {
        if (pages[k] < 0) continue;
        const size_t e = ((size_t)pages[k] * s.U + u) * s.T + (t0 + k) % s.T;
        const float v = code_f32(vp[e * D + tid]) * vs[(size_t)pages[k] * s.U + u];
        for (int g = 0; g < G; ++g) acc[g] = fmaf(p[g][k], v, acc[g]);
      }
    }
  }
  __syncthreads();
  if (tid < D)
    for (int g = 0; g < G; ++g)
      out[(row * s.Hq + u * G + g) * D + tid] = from_f32<T>(l_s[g] > 0.f || l_s[g] != l_s[g] ? acc[g] / l_s[g] : 0.f);
}

template <typename T, int D>
cudaError_t launch(const PageStep& s, const void* q, int64_t q_stride, const void* kp,
                   const void* vp, const float* ks, const float* vs, void* out,
                   cudaStream_t stream) {
  return launch_k(page_attend_kernel<T, D>, dim3((unsigned)s.n_tokens, (unsigned)s.U),
                  dim3(kThreads), 0, stream, true, s, (const T*)q, q_stride, (const uint8_t*)kp,
                  (const uint8_t*)vp, ks, vs, (T*)out);
}

}  // namespace

size_t page_attend_workspace(const PageStep&, salsc_dtype) { return 0; }

cudaError_t launch_page_attend(const PageStep& s, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void*, salsc_dtype dt,
                               cudaStream_t stream) {
  if (dt == SALSC_BF16)
    return s.d == 64 ? launch<__nv_bfloat16, 64>(s, q, q_stride, k_pages, v_pages, k_scales,
                                                 v_scales, out, stream)
                     : launch<__nv_bfloat16, 128>(s, q, q_stride, k_pages, v_pages, k_scales,
                                                  v_scales, out, stream);
  return s.d == 64 ? launch<float, 64>(s, q, q_stride, k_pages, v_pages, k_scales, v_scales, out,
                                       stream)
                   : launch<float, 128>(s, q, q_stride, k_pages, v_pages, k_scales, v_scales, out,
                                        stream);
}

}  // namespace salsc
