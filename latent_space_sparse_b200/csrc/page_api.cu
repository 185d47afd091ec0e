// page_api.cu -- the extern "C" boundary of the paged 8-bit cache: checks,
// the step's plan and the launches.
#include <math.h>

#include "page.cuh"

namespace {

constexpr size_t kFlagsBytes = salsc::kWsAlign;  // the anomaly word's region

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

salsc_status make_step(const salsc_page_desc* D, salsc::PageStep* S) {
  if (!D) return SALSC_ERR_INVALID_ARG;
  if (D->batch < 1 || D->n_q_heads < 1 || D->n_kv_heads < 1 || D->head_dim < 1 ||
      D->page_size < 1 || D->n_pages < 1 || D->max_pages < 1 || D->n_tokens < 0 || D->max_q < 0 ||
      D->window < 0)
    return SALSC_ERR_INVALID_ARG;
  if (D->n_q_heads % D->n_kv_heads != 0) return SALSC_ERR_INVALID_ARG;
  if (D->dtype != SALSC_F32 && D->dtype != SALSC_BF16) return SALSC_ERR_INVALID_ARG;
  if (D->rope_base != 0.0 && (!(D->rope_base > 1.0) || !isfinite(D->rope_base)))
    return SALSC_ERR_INVALID_ARG;
  if (!(D->softmax_scale >= 0.0f) || !isfinite(D->softmax_scale)) return SALSC_ERR_INVALID_ARG;
  if (!D->page_table_dev || !D->seq_lens_dev) return SALSC_ERR_INVALID_ARG;
  // without offsets, row b is sequence b's token
  if (!D->q_offsets_dev && D->n_tokens < D->batch) return SALSC_ERR_INVALID_ARG;
  if (D->head_dim != 64 && D->head_dim != 128) return SALSC_ERR_UNSUPPORTED;
  if (D->page_size != 16 && D->page_size != 32 && D->page_size != 64 && D->page_size != 128)
    return SALSC_ERR_UNSUPPORTED;
  if (D->n_kv_heads > salsc::kMaxUnits) return SALSC_ERR_UNSUPPORTED;
  if (D->n_q_heads / D->n_kv_heads > salsc::kPageMaxGroup) return SALSC_ERR_UNSUPPORTED;
  // rows of the pool and positions are 32-bit numbers
  if ((int64_t)D->n_pages * D->n_kv_heads * D->page_size > INT32_MAX) return SALSC_ERR_UNSUPPORTED;
  if ((int64_t)D->max_pages * D->page_size > INT32_MAX) return SALSC_ERR_UNSUPPORTED;

  salsc::PageStep s{};
  s.B = D->batch;
  s.Hq = D->n_q_heads;
  s.U = D->n_kv_heads;
  s.G = s.Hq / s.U;
  s.d = D->head_dim;
  s.T = D->page_size;
  while ((1 << s.log_t) < s.T) ++s.log_t;
  s.n_pages = D->n_pages;
  s.max_pages = D->max_pages;
  s.n_tokens = D->n_tokens;
  s.max_q = D->q_offsets_dev || D->max_q < 1 ? D->max_q : 1;
  s.window = D->window;
  s.rotate = D->rope_base != 0.0;
  s.scale = D->softmax_scale != 0.0f ? D->softmax_scale : (float)(1.0 / sqrt((double)s.d));
  s.table = D->page_table_dev;
  s.lens = D->seq_lens_dev;
  s.offs = D->q_offsets_dev;
  if (s.rotate) {
    // products of the first power in 64-bit fixed point: 64 roundings of 2^-64 of a
    // turn, below 2^-27 of a turn at position 2^31
    const long double two64 = 18446744073709551616.0L;
    const long double step = powl((long double)D->rope_base, -2.0L / s.d) * two64;
    const uint64_t step64 = step < two64 - 1.0L ? (uint64_t)step : UINT64_MAX;
    uint64_t f = 0x28BE60DB9391054Aull;  // 1 / 2pi
    for (int i = 0; i < s.d / 2; ++i) {
      s.turns[i] = f;
      f = (uint64_t)(((unsigned __int128)f * step64 + (1ull << 63)) >> 64);
    }
  }
  *S = s;
  return SALSC_OK;
}

salsc_status check_ws(const salsc_page_desc* desc, salsc::PageStep& s, void* ws, size_t ws_bytes) {
  if (!ws || ((uintptr_t)ws % salsc::kWsAlign) != 0 ||
      ws_bytes < kFlagsBytes + salsc::page_attend_workspace(s, desc->dtype))
    return SALSC_ERR_WORKSPACE;
  s.flags = (uint32_t*)ws;
  return SALSC_OK;
}

// Row stride in elements: 0 means contiguous rows of `row` elements.
bool fix_stride(int64_t& stride, int64_t row) {
  if (stride == 0) stride = row;
  return stride >= row && stride % 8 == 0;
}

}  // namespace

extern "C" {

size_t salsc_page_workspace_size(const salsc_page_desc* desc) {
  salsc::PageStep s;
  if (make_step(desc, &s) != SALSC_OK) return 0;
  return kFlagsBytes + salsc::page_attend_workspace(s, desc->dtype);
}

salsc_status salsc_page_prepare(const salsc_page_desc* desc, void* ws, size_t ws_bytes,
                                salsc_stream stream) {
  salsc::PageStep s;
  salsc_status st = make_step(desc, &s);
  if (st != SALSC_OK) return st;
  if ((st = check_ws(desc, s, ws, ws_bytes)) != SALSC_OK) return st;
  const cudaError_t e =
      cudaMemsetAsync(ws, 0, kFlagsBytes + salsc::page_attend_cleared(), (cudaStream_t)stream);
  return e == cudaSuccess ? SALSC_OK : salsc::record_cuda_error(e);
}

salsc_status salsc_page_append(const salsc_page_desc* desc, const void* K_new, int64_t k_stride,
                               const void* V_new, int64_t v_stride, void* k_pages, void* v_pages,
                               float* k_scales, float* v_scales, void* ws, size_t ws_bytes,
                               salsc_stream stream) {
  salsc::PageStep s;
  salsc_status st = make_step(desc, &s);
  if (st != SALSC_OK) return st;
  if (!k_pages || !v_pages || !k_scales || !v_scales) return SALSC_ERR_INVALID_ARG;
  if (s.n_tokens > 0 && (!K_new || !V_new)) return SALSC_ERR_INVALID_ARG;
  if (!aligned16(K_new) || !aligned16(V_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
      ((uintptr_t)k_scales & 3u) || ((uintptr_t)v_scales & 3u))
    return SALSC_ERR_INVALID_ARG;
  if (!fix_stride(k_stride, (int64_t)s.U * s.d) || !fix_stride(v_stride, (int64_t)s.U * s.d))
    return SALSC_ERR_INVALID_ARG;
  if ((st = check_ws(desc, s, ws, ws_bytes)) != SALSC_OK) return st;
  if (s.n_tokens == 0 || s.max_q == 0) return SALSC_OK;
  const cudaError_t e =
      salsc::launch_page_append(s, K_new, k_stride, V_new, v_stride, k_pages, v_pages, k_scales,
                                v_scales, desc->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SALSC_OK : salsc::record_cuda_error(e);
}

salsc_status salsc_page_attend(const salsc_page_desc* desc, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void* ws, size_t ws_bytes,
                               salsc_stream stream) {
  salsc::PageStep s;
  salsc_status st = make_step(desc, &s);
  if (st != SALSC_OK) return st;
  if (!k_pages || !v_pages || !k_scales || !v_scales) return SALSC_ERR_INVALID_ARG;
  if (s.n_tokens > 0 && (!q || !out)) return SALSC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_pages) || !aligned16(v_pages) ||
      ((uintptr_t)k_scales & 3u) || ((uintptr_t)v_scales & 3u))
    return SALSC_ERR_INVALID_ARG;
  if (!fix_stride(q_stride, (int64_t)s.Hq * s.d)) return SALSC_ERR_INVALID_ARG;
  if (s.n_tokens > 0) {  // pieces of a row's work read its queries after others wrote its output
    const uintptr_t e = desc->dtype == SALSC_BF16 ? 2 : 4, row = (uintptr_t)s.Hq * s.d;
    const uintptr_t q0 = (uintptr_t)q, q1 = q0 + ((uintptr_t)(s.n_tokens - 1) * q_stride + row) * e;
    const uintptr_t o0 = (uintptr_t)out, o1 = o0 + (uintptr_t)s.n_tokens * row * e;
    if (q0 < o1 && o0 < q1) return SALSC_ERR_INVALID_ARG;
  }
  if ((st = check_ws(desc, s, ws, ws_bytes)) != SALSC_OK) return st;
  if (s.n_tokens == 0 || s.max_q == 0) return SALSC_OK;
  const cudaError_t e = salsc::launch_page_attend(s, q, q_stride, k_pages, v_pages, k_scales,
                                                  v_scales, out, (char*)ws + kFlagsBytes,
                                                  desc->dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? SALSC_OK : salsc::record_cuda_error(e);
}

}  // extern "C"
