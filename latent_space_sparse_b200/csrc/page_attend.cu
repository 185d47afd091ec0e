// page_attend.cu -- attention over the paged 8-bit cache: the plan of a call,
// and the merge of page_many's units whose tiles several CTAs shared.
#include "page.cuh"

namespace salsc {
namespace {

constexpr int kMergeWarps = 4, kMergeRows = 4;  // warps of a merge CTA, rows of a warp
// What a unit takes besides its tiles, in tiles: without it the CTAs with many
// short units were last (a prompt of 4K 442 us, with it 261 at the time). The choice
// is flat: 1, 2, 3, 4 and 6 for page_few gave 67, 61, 53, 53 and 55 us on 64 short
// sequences, 2, 3, 4, 6 and 8 for page_many 227, 227, 225, 228 and 232 us on a
// prompt of 4K (both when they were chosen).
constexpr int kOverFew = 3, kOverMany = 3;

// A warp takes kMergeRows rows of the unit that CTA c starts (usually of two
// pieces): lane (row, piece) reads a piece's maximum and normaliser, and the
// pieces' outputs of all rows are loaded together.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
page_merge_kernel(const __grid_constant__ PageStep s, const __grid_constant__ PageWork w,
                  __nv_bfloat16* __restrict__ out) {
  constexpr int kV = D / 32, kPieces = 32 / kMergeRows;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r0 = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * kMergeRows;
  grid_dependency_wait();
  allow_dependent_launch();
  const int4 info = w.info[c];
  if (r0 >= info.z) return;
  const int n = info.w - c + 1;  // pieces
  auto slot = [&](int i, int r) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * w.rows + r; };
  const int mr = lane / kPieces, mp = lane % kPieces, rr = min(r0 + mr, info.z - 1);
  float m = -INFINITY;
  for (int i = mp; i < n; i += kPieces) m = fmaxf(m, w.ml[slot(i, rr)].x);
#pragma unroll
  for (int o = kPieces / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[kMergeRows][kV];
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r)
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[r][k] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kPieces) {
    float f = 0.f;
    if (i0 + mp < n) {
      const float2 ml = w.ml[slot(i0 + mp, rr)];
      f = page_factor(ml, m, l);
    }
    const int top = min(kPieces, n - i0);
#pragma unroll 2
    for (int i = 0; i < top; ++i) {
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        const float fi = __shfl_sync(0xffffffffu, f, r * kPieces + i);
        const float* a = w.acc + slot(i0 + i, min(r0 + r, info.z - 1)) * D + lane * kV;
        if constexpr (kV == 4) {
          const float4 x = *(const float4*)a;
          acc[r][0] = fmaf(fi, x.x, acc[r][0]);
          acc[r][1] = fmaf(fi, x.y, acc[r][1]);
          acc[r][2] = fmaf(fi, x.z, acc[r][2]);
          acc[r][3] = fmaf(fi, x.w, acc[r][3]);
        } else {
          const float2 x = *(const float2*)a;
          acc[r][0] = fmaf(fi, x.x, acc[r][0]);
          acc[r][1] = fmaf(fi, x.y, acc[r][1]);
        }
      }
    }
  }
#pragma unroll
  for (int o = kPieces / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r) {
    const float lr = __shfl_sync(0xffffffffu, l, r * kPieces);
    if (r0 + r >= info.z) break;
    const int i = (r0 + r) / s.G, g = r0 + r - i * s.G;
    __nv_bfloat16* dst = out + ((int64_t)(info.x + i) * s.Hq + info.y * s.G + g) * D + lane * kV;
#pragma unroll
    for (int k = 0; k < kV; k += 2)
      *(__nv_bfloat162*)(dst + k) = __floats2bfloat162_rn(lr == 0.f ? 0.f : acc[r][k] / lr,
                                                          lr == 0.f ? 0.f : acc[r][k + 1] / lr);
  }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Partial results of a kernel of `grid` CTAs whose row blocks have `rows` rows,
// from p + off on; off moves behind them.
PageWork layout(const PageStep& s, int rows, int grid, void* part, size_t& off) {
  PageWork w{};
  w.rows = rows;
  w.grid = grid;
  char* p = (char*)part;
  w.info = (int4*)(p + off);
  off = align_up(off + sizeof(int4) * grid);
  w.ml = (float2*)(p + off);
  off = align_up(off + sizeof(float2) * 2 * grid * rows);
  w.acc = (float*)(p + off);
  off = align_up(off + sizeof(float) * 2 * grid * rows * s.d);
  return w;
}

// The kernels of a step.  page_few takes sequences of up to 16 rows (new tokens
// times heads per KV head) and all of fp32 storage, page_many the others: at 16
// rows page_few takes 53 us and page_many 84 (8 sequences of 8192 tokens, 4 of
// them new, 32 heads on 8; 53 and 83 us for 2 sequences, 16 new, 32 heads on 32),
// at 20 rows page_many 50 us (4 sequences of 8192, 5 new), where a page_few for 32
// rows took 95 when there was one.  A step that has both
// kinds sends page_few the sequences with a single new token only: its time
// grows with the rows that it is built for (eight requests of 1 to 1024 new
// tokens, when it was chosen: 237 us with one for 32 rows, 208 with one for 4).
// fp32 storage pays for that rule at prompts: the cache is read once for every 16
// rows, so that a prompt of 4K takes 2.8 ms, 14 times as long as in bf16.
struct Plan {
  PageWork few, many;
  bool has_many;
  size_t bytes;
};

Plan make_plan(const PageStep& s, salsc_dtype dt, void* part) {
  Plan p{};
  int rows = page_few_rows((int64_t)s.max_q * s.G);
  p.has_many = dt == SALSC_BF16 && (int64_t)s.max_q * s.G > rows;
  if (p.has_many) rows = page_few_rows(s.G);
  // page_few's counters come first, and nothing else lies there whatever the
  // descriptor: salsc_page_prepare clears them, and each call leaves them so
  p.bytes = align_up(page_attend_cleared());
  p.few = layout(s, rows, page_few_grid(rows, dt), part, p.bytes);
  p.few.done = (uint32_t*)part;
  p.few.tb = rows / s.G;
  p.few.over = kOverFew;
  p.few.min_rows = 1;
  p.few.max_rows = INT32_MAX;
  if (p.has_many) {
    p.many = layout(s, kPageManyRows, kPageGrid, part, p.bytes);
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

cudaError_t launch_merge(const PageStep& s, const PageWork& w, void* out, cudaStream_t stream) {
  const dim3 grid(w.grid, (unsigned)(w.rows / (kMergeWarps * kMergeRows)));
  return launch_k(s.d == 64 ? page_merge_kernel<64> : page_merge_kernel<128>, grid, dim3(kMergeWarps * 32),
                  0, stream, true, s, w, (__nv_bfloat16*)out);
}

}  // namespace

size_t page_attend_cleared() { return sizeof(uint32_t) * 2 * kPageGrid; }

size_t page_attend_workspace(const PageStep& s, salsc_dtype dt) {
  return make_plan(s, dt, nullptr).bytes;
}

cudaError_t launch_page_attend(const PageStep& s, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void* part, salsc_dtype dt,
                               cudaStream_t stream) {
  Plan p = make_plan(s, dt, part);
  cudaError_t e = cudaSuccess;
  if (p.has_many) {
    e = launch_page_many(s, p.many, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, stream);
    // page_few may begin beside page_many only right behind it: page_many begins when the
    // rotation in front of it has waited for all earlier work, and page_few waits for both at
    // its end, before anything that waits for page_few goes on
    p.few.overlaps = 1;
  }
  if (e == cudaSuccess)
    e = launch_page_few(s, p.few, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, dt, stream);
  if (p.has_many && e == cudaSuccess) e = launch_merge(s, p.many, out, stream);
  return e;
}

}  // namespace salsc
