// page.cuh -- the paged 8-bit cache: plan, arguments and device helpers shared
// by the append (page_append.cu), the attention (page_attend.cu) and the
// entry points (page_api.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "page_sched.cuh"

namespace salsc {

constexpr int kPageMaxGroup = 16;   // query heads per KV head
constexpr int kPageMaxHeadDim = 128;

// One step's sizes, pointers to the caller's lengths and tables, and the
// rotation's frequencies: passed to the kernels by value.
struct PageStep {
  int B, Hq, U, G, d, T;  // batch, query heads, KV heads, heads per KV head, head dim, page size
  int log_t;              // T = 2^log_t
  int n_pages, max_pages, n_tokens, max_q;
  int window;  // 0: none
  int rotate;  // 0: keys and queries are taken as they are
  float scale;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* offs;  // null: row b is sequence b's one token
  uint32_t* flags;
  // frequency of pair i in turns per position, base^(-2i/d) / 2pi, in units of 2^-64
  uint64_t turns[kPageMaxHeadDim / 2];
};

// One sequence's part of a step, cut to the step's bounds.
struct PageSeq {
  int n;     // tokens in the cache, new ones included
  int m;     // new tokens (at most max_q)
  int row0;  // row of the first of them
};

// An integer of the caller's.  kL2: past L1, which may hold lines from before the
// work that wrote it. page_many and the page_few behind it need that, for lengths,
// offsets, tables, scales and queries: they begin when a kernel of their own step
// has waited for all earlier work, but wait themselves only later. (The append has
// waited itself, and all threads of its blocks read the same lengths: from L2 64
// single tokens of 32 heads took 22.9 us instead of 7.7.)
template <bool kL2>
__device__ __forceinline__ int32_t load_int(const int32_t* p) {
  return kL2 ? __ldcg(p) : *p;
}

template <bool kL2>
__device__ __forceinline__ PageSeq page_seq(const PageStep& s, int b) {
  PageSeq q;
  bool bad = false;
  q.n = load_int<kL2>(s.lens + b);
  const int cap = s.max_pages * s.T;
  if (q.n < 0 || q.n > cap) {
    bad = true;
    q.n = q.n < 0 ? 0 : cap;
  }
  if (s.offs) {
    int o0 = load_int<kL2>(s.offs + b), o1 = load_int<kL2>(s.offs + b + 1);
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
template <bool kL2>
__device__ __forceinline__ int page_of(const PageStep& s, int b, int j) {
  const int pg = load_int<kL2>(s.table + (size_t)b * s.max_pages + j);
  if ((unsigned)pg < (unsigned)s.n_pages) return pg;
  atomicOr(s.flags, FLAG_BAD_INDEX);
  return -1;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A byte of w is the NaN code 0x7F or 0xFF.
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
}

// Two fp32 at a time.
__device__ __forceinline__ void fma2(float& a0, float& a1, float m, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mov.b64 z, {%3, %3};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(m), "f"(c));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

__device__ __forceinline__ void mul2(float& a0, float& a1, float m) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(m));
}

// Item x of a list in which sequence b has cost(b) items: the sequence (false
// when x is past the end), and x becomes the item's index in it.  A warp finds
// it for itself, without a barrier: each lane adds up a 32nd of the sequences,
// then of those of the lane that holds x, and so on.  After the last round lane
// i has called cost(b0 + i) last, and the sequence is that of lane b - b0.
// start(total) says what x is once the length of the list is known.
template <typename F, typename S>
__device__ __forceinline__ bool page_find(int B, F cost, S start, int64_t& x, int& b, int& b0) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  for (bool first = true;; first = false) {
    const int c = (n + 31) / 32;
    int64_t sum = 0;
#pragma unroll 1
    for (int i = 0; i < c; ++i) {
      const int k = lane * c + i;
      if (k < n) sum += cost(lo + k);
    }
    int64_t end = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += t;
    }
    if (first) {
      const int64_t total = __shfl_sync(0xffffffffu, end, 31);
      x = start(total);
      if (x >= total) return false;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, x < end)) - 1;
    x -= __shfl_sync(0xffffffffu, end - sum, l);
    b0 = lo;
    lo += l * c;
    n = min(c, n - l * c);
    if (c == 1) break;
  }
  b = lo;
  return true;
}

// cos and sin of position pos at `turns` (of 2^64) turns per position: the
// product's low 64 bits are the angle in parts of a turn, exact to 2^-33 of a
// turn at every position below 2^31, so that far positions keep fp32's accuracy.
__device__ __forceinline__ void page_cs(int pos, uint64_t turns, float& c, float& s) {
  const int32_t a = (int32_t)(((uint64_t)(uint32_t)pos * turns) >> 32);
  sincospif((float)a * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
}

// ---------------------------------------------------------------- attention

// A page's value scale as f * 2^e.  Finite scales from 2^-99 on have 1 <= |f| < 2.
// Smaller ones, which the append writes for pages of zeros, would have weights of
// 2^-126 and less beside scales above 2^26 and drop out of the normaliser: they take
// an e that lies 24 below the largest, `big`, that was met so far (-100 at least,
// which leaves them exact where nothing larger is).  What is not finite is NaN.
// down = 2^-e.
struct ValueScale {
  float f, e, down;
};
constexpr int kNoScale = -1000;  // no scale from 2^-99 on was met
__device__ __forceinline__ int scale_exponent(float v) {
  const int ex = (int)((__float_as_uint(v) >> 23) & 255u);
  return ex < 28 || ex == 255 ? kNoScale : ex - 127;
}
__device__ __forceinline__ ValueScale value_scale(float v, int big) {
  const int ex = (int)((__float_as_uint(v) >> 23) & 255u);
  const int e = ex < 28 ? max(big - 24, -100) : ex - 127;
  const float down = __uint_as_float(e == 127 ? 0x00400000u : (uint32_t)(127 - e) << 23);
  if (ex == 255) return ValueScale{__uint_as_float(0x7FC00000u), 0.f, 1.f};
  return ValueScale{v * down, (float)e, down};
}
// A key scale: NaN if it is not finite, so that scores of -inf hide no token.
__device__ __forceinline__ float key_scale(float k) { return k + (k - k); }

// Which sequences a kernel of the attention takes, and how it cuts them.
struct PageWork {
  int min_rows, max_rows;  // sequences with min_rows <= new tokens * G <= max_rows
  int tb;                  // new tokens of a row block
  int over;                // tiles' worth of time that a unit takes besides its tiles
  int rows;                // rows of a partial slot (>= tb * G)
  int grid;                // CTAs
  int overlaps;            // page_few behind page_many of the same step, which need not have ended
  // Partial results of units that several CTAs share: CTA c's slots 2c (a
  // piece that starts inside a unit) and 2c + 1 (one that starts a unit and
  // does not end it), of `rows` rows each
  float* acc;     // [2 * grid][rows][d] unnormalised outputs
  float2* ml;     // [2 * grid][rows] running maximum (log2 units) and normaliser
  // few rows: pieces of the unit that CTA c starts that are done (0 between calls)
  uint32_t* done;  // [grid]
  // many rows
  int4* info;     // [grid] of slot 2c + 1: first row's token row, KV head, rows, last CTA of the unit
  void* qrot;     // rotated queries and their rows' exponents (page_many.cu)
  int8_t* qexp;
};

// A cursor over the step's units and tiles, for one warp or thread (every
// thread that uses one advances it alike).
struct PageCursor {
  const PageStep& s;
  const PageWork& w;
  int b, u, k;      // sequence, KV head, row block
  PageBlocks blk;   // of sequence b
  int row0;         // row of the sequence's first new token
  int tiles;        // tiles of the unit
  int tile;         // tile inside the unit (0-based from the block's first tile)
  int64_t base;     // the unit's first place in the list

  __device__ __forceinline__ PageCursor(const PageStep& s_, const PageWork& w_) : s(s_), w(w_) {}
  __device__ __forceinline__ void load() {
    const PageSeq q = page_seq<true>(s, b);
    blk = PageBlocks{q.n, q.m, w.tb, s.window, w.over};
    row0 = q.row0;
  }
  __device__ __forceinline__ bool mine() const {
    const int64_t r = (int64_t)blk.m * s.G;
    return r >= w.min_rows && r <= w.max_rows;
  }
  // tiles from `tile` on of a range that ends at place x1 (0 or less: none)
  __device__ __forceinline__ int upto(int64_t x1) const {
    return (int)(min((int64_t)tiles, x1 - base - w.over) - tile);
  }
  __device__ __forceinline__ bool whole(int n) const { return tile == 0 && n == tiles; }
  // the unit's last tile's place
  __device__ __forceinline__ int64_t last() const { return base + w.over + tiles - 1; }
  // to the next unit; false past the last one
  __device__ __forceinline__ bool next_unit() {
    tile = 0;
    base += w.over + tiles;
    if (++u < s.U) return true;
    u = 0;
    if (++k < blk.count()) {
      tiles = blk.tiles(k);
      return true;
    }
    k = 0;
    while (++b < s.B) {
      load();
      if (mine()) {
        tiles = blk.tiles(0);
        return true;
      }
    }
    return false;
  }
};

// Warp-wide: the length of the list of the kernel's sequences, the end x1 of
// this CTA's range of it, and the cursor at the range's start; false for an
// empty range.  Every warp that needs it finds it for itself: no barrier.
__device__ __forceinline__ bool page_begin(PageCursor& c, int64_t& total, int64_t& x1) {
  const PageStep& s = c.s;
  const PageWork& w = c.w;
  const int lane = threadIdx.x & 31;
  PageSeq q{};  // of the sequence that the lane looked at last
  int64_t x, x0;
  int b0;
  const bool any = page_find(
      s.B,
      [&](int b) -> int64_t {
        q = page_seq<true>(s, b);
        const int64_t r = (int64_t)q.m * s.G;
        if (r < w.min_rows || r > w.max_rows) return 0;
        const PageBlocks p{q.n, q.m, w.tb, s.window, w.over};
        return (int64_t)s.U * p.before(p.count());
      },
      [&](int64_t all) {
        total = all;
        const int64_t each = div_small(all, gridDim.x), more = all - each * gridDim.x;
        x0 = blockIdx.x * each + min((int64_t)blockIdx.x, more);  // share_begin
        x1 = x0 + each + (blockIdx.x < more ? 1 : 0);
        return x0 < x1 ? x0 : all;
      },
      x, c.b, b0);
  if (!any) return false;
  const int l = c.b - b0;
  c.blk = PageBlocks{__shfl_sync(0xffffffffu, q.n, l), __shfl_sync(0xffffffffu, q.m, l), w.tb, s.window, w.over};
  c.row0 = __shfl_sync(0xffffffffu, q.row0, l);
  // the row block: its U KV heads have U * cost behind U * before(k); 32 tries at a time
  const int64_t y = div_small(x, s.U);
  int lo = 0, n = c.blk.count();  // the block is one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, k = lo + lane * step;
    const bool at = k < lo + n && c.blk.before(k) <= y;
    const int hit = __popc(__ballot_sync(0xffffffffu, at)) - 1;  // before() grows with k
    n = min(step, n - hit * step);
    lo += hit * step;
  }
  c.k = lo;
  c.tiles = c.blk.tiles(c.k);
  x -= (int64_t)s.U * c.blk.before(c.k);
  const int unit = w.over + c.tiles;
  c.u = (int)div_small(x, unit);
  x -= (int64_t)c.u * unit;
  c.base = x0 - x;
  c.tile = x > w.over ? (int)(x - w.over) : 0;
  return true;
}

// A piece's factor 2^(m_i - m), with l += 2^(m_i - m) l_i. In two steps: pieces of
// small value scales have a large l_i and an m_i far below. A piece without a token
// (m_i = -inf) weighs nothing; a NaN stays one.
__device__ __forceinline__ float page_factor(float2 ml, float m, float& l) {
  const float h = ml.x == -INFINITY ? 0.f : exp2f(0.5f * (ml.x - m));
  l += h * ml.y * h;
  return h * h;
}

// One row of a unit whose pieces are those of CTAs c0 .. c0 + n - 1:
//   out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i
// CTA c0's second slot holds the unit's first piece, the following CTAs' first
// slots the others.  A warp to a row, D / 32 dimensions a lane; the pieces'
// maxima are read first, 32 at a time.  Reads past L1: other SMs wrote.
template <typename T, int D>
__device__ __forceinline__ void page_merge_row(const PageWork& w, int c0, int n, int r, T* dst) {
  constexpr int kV = D / 32;
  const int lane = threadIdx.x & 31;
  auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * w.rows + r; };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(&w.ml[slot(i)]).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.f;
    if (i0 + lane < n) {
      const float2 ml = __ldcg(&w.ml[slot(i0 + lane)]);
      f = page_factor(ml, m, l);
    }
    const int top = min(32, n - i0);
#pragma unroll 8
    for (int i = 0; i < top; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float* a = w.acc + slot(i0 + i) * D + lane * kV;
      if constexpr (kV == 4) {
        const float4 x = __ldcg((const float4*)a);
        acc[0] = fmaf(fi, x.x, acc[0]);
        acc[1] = fmaf(fi, x.y, acc[1]);
        acc[2] = fmaf(fi, x.z, acc[2]);
        acc[3] = fmaf(fi, x.w, acc[3]);
      } else {
        const float2 x = __ldcg((const float2*)a);
        acc[0] = fmaf(fi, x.x, acc[0]);
        acc[1] = fmaf(fi, x.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
  for (int k = 0; k < kV; ++k) dst[lane * kV + k] = from_f32<T>(l == 0.f ? 0.f : acc[k] / l);
}

// Host side: launchers.
constexpr int kPageGrid = 148;  // SMs
cudaError_t launch_page_append(const PageStep& s, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, void* k_pages, void* v_pages, float* k_scales,
                               float* v_scales, salsc_dtype dt, cudaStream_t stream);
cudaError_t launch_page_attend(const PageStep& s, const void* q, int64_t q_stride,
                               const void* k_pages, const void* v_pages, const float* k_scales,
                               const float* v_scales, void* out, void* part, salsc_dtype dt,
                               cudaStream_t stream);
size_t page_attend_workspace(const PageStep& s, salsc_dtype dt);
size_t page_attend_cleared();  // bytes at the workspace's start that are 0 between calls
// The attention of few rows (page_few.cu): rows of its row blocks, and its launch.
int page_few_rows(int64_t rows);  // for sequences of up to `rows` rows
int page_few_grid(int rows, salsc_dtype dt);
cudaError_t launch_page_few(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                            const void* k_pages, const void* v_pages, const float* k_scales,
                            const float* v_scales, void* out, salsc_dtype dt, cudaStream_t stream);
// The attention of many rows (page_many.cu; bf16): rows of its row blocks, and its launch.
constexpr int kPageManyRows = 256;
cudaError_t launch_page_many(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                             const void* k_pages, const void* v_pages, const float* k_scales,
                             const float* v_scales, void* out, cudaStream_t stream);

}  // namespace salsc
