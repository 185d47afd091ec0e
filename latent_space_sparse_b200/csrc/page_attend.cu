// page_attend.cu -- attention over the paged 8-bit cache: the plan of a call,
// and the merge of units whose tiles several CTAs shared.
#include "page.cuh"

namespace salsc {
namespace {

constexpr int kMergeWarps = 4;  // rows of a merge CTA
// What a unit takes besides its tiles, in tiles.
constexpr int kOverFew = 2, kOverMany = 3;

// out[row] = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i over the pieces i
// of a unit.  CTA c's second slot holds a unit's first piece, the following
// CTAs' first slots the others.  A warp per row, D / 32 dimensions a lane; the
// pieces' maxima are read first, 32 at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
page_merge_kernel(const __grid_constant__ PageStep s, const __grid_constant__ PageWork w,
                  T* __restrict__ out) {
  constexpr int kV = D / 32;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  allow_dependent_launch();
  const int4 info = w.info[c];
  if (r >= info.z) return;
  const int n = info.w - c + 1;  // pieces
  auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * w.rows + r; };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, w.ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.f;
    if (i0 + lane < n) {
      const float2 ml = w.ml[slot(i0 + lane)];
      // a piece without a token (m = -inf) weighs nothing; a NaN stays one
      f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
      l += f * ml.y;
    }
    const int top = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < top; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float* a = w.acc + slot(i0 + i) * D + lane * kV;
      if constexpr (kV == 4) {
        const float4 x = *(const float4*)a;
        acc[0] = fmaf(fi, x.x, acc[0]);
        acc[1] = fmaf(fi, x.y, acc[1]);
        acc[2] = fmaf(fi, x.z, acc[2]);
        acc[3] = fmaf(fi, x.w, acc[3]);
      } else {
        const float2 x = *(const float2*)a;
        acc[0] = fmaf(fi, x.x, acc[0]);
        acc[1] = fmaf(fi, x.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int i = r / s.G, g = r - i * s.G;
  T* dst = out + ((int64_t)(info.x + i) * s.Hq + info.y * s.G + g) * D + lane * kV;
#pragma unroll
  for (int k = 0; k < kV; ++k) dst[k] = from_f32<T>(l == 0.f ? 0.f : acc[k] / l);
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Partial results of a kernel whose row blocks have `rows` rows, from p + off on; off moves behind
// them.
PageWork layout(const PageStep& s, int rows, void* part, size_t& off) {
  PageWork w{};
  w.rows = rows;
  char* p = (char*)part;
  w.info = (int4*)(p + off);
  off = align_up(off + sizeof(int4) * kPageGrid);
  w.ml = (float2*)(p + off);
  off = align_up(off + sizeof(float2) * 2 * kPageGrid * rows);
  w.acc = (float*)(p + off);
  off = align_up(off + sizeof(float) * 2 * kPageGrid * rows * s.d);
  return w;
}

// The kernels of a step: sequences with at most `few.max_rows` rows per KV head
// go to page_few, the others (bf16 only) to page_many.
struct Plan {
  PageWork few, many;
  bool has_many;
  size_t bytes;
};

Plan make_plan(const PageStep& s, salsc_dtype dt, void* part) {
  Plan p{};
  const int rows = page_few_rows(s, dt);
  p.few = layout(s, rows, part, p.bytes);
  p.few.tb = rows / s.G;
  p.few.over = kOverFew;
  p.few.min_rows = 1;
  p.few.max_rows = INT32_MAX;
  p.has_many = dt == SALSC_BF16 && (int64_t)s.max_q * s.G > rows;
  if (p.has_many) {
    p.many = layout(s, kPageManyRows, part, p.bytes);
    p.many.tb = 2 * (kPageManyRows / 2 / s.G);
    p.many.qrot = (char*)part + p.bytes;
    p.bytes = align_up(p.bytes + (size_t)s.n_tokens * s.Hq * s.d * 2);
    p.many.qexp = (int8_t*)part + p.bytes;
    p.bytes = align_up(p.bytes + (size_t)s.n_tokens * s.Hq);
    p.many.over = kOverMany;
    p.many.min_rows = rows + 1;
    p.many.max_rows = INT32_MAX;
    p.few.max_rows = rows;
  }
  return p;
}

}  // namespace

size_t page_attend_workspace(const PageStep& s, salsc_dtype dt) {
  return make_plan(s, dt, nullptr).bytes;
}

cudaError_t launch_page_merge(const PageStep& s, const PageWork& w, void* out, salsc_dtype dt,
                              cudaStream_t stream) {
  const dim3 grid(kPageGrid, (unsigned)((w.rows + kMergeWarps - 1) / kMergeWarps));
  const dim3 block(kMergeWarps * 32);
  if (dt == SALSC_BF16)
    return s.d == 64 ? launch_k(page_merge_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, true,
                                s, w, (__nv_bfloat16*)out)
                     : launch_k(page_merge_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, true,
                                s, w, (__nv_bfloat16*)out);
  return s.d == 64
             ? launch_k(page_merge_kernel<float, 64>, grid, block, 0, stream, true, s, w, (float*)out)
             : launch_k(page_merge_kernel<float, 128>, grid, block, 0, stream, true, s, w,
                        (float*)out);
}

cudaError_t launch_page_attend(const PageStep& s, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void* part, salsc_dtype dt,
                               cudaStream_t stream) {
  const Plan p = make_plan(s, dt, part);
  cudaError_t e = cudaSuccess;
  if (p.has_many) {
    e = launch_page_many(s, p.many, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, stream);
    if (e == cudaSuccess) e = launch_page_merge(s, p.many, out, dt, stream);
  }
  if (e == cudaSuccess)
    e = launch_page_few(s, p.few, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, dt, stream);
  if (e == cudaSuccess) e = launch_page_merge(s, p.few, out, dt, stream);
  return e;
}

}  // namespace salsc
