// page_few.cu -- attention of few query rows over the paged 8-bit cache:
// single tokens (serving) and short runs of tokens; every row count for fp32.
//
//   s_t = RoPE(q) . K_t,  p = softmax(scale * s),  out = sum_t p_t V_t
//
// A row block is up to RC rows: the query heads of one KV head, for one or
// more new tokens.  With few rows the work is the read of the cache, one byte
// per element, so the e4m3 codes go from HBM to the tensor cores as they are
// (TMA into shared memory, no conversion on the way):
//   S^T [128 tokens x N] = K tile (M = tokens, K-major)  x  Q   (tcgen05 kind::f8f6f4)
//   O^T [d x N]         += V tile (M = d, MN-major)      x  P
// The other operand is cut into e4m3 terms, x = x0 + x1/32 + x2/32^2 + ...,
// each the rounding of 32 times what the terms before it left: a term takes 4
// bits, the products are exact and the accumulators fp32.  3 terms hold 12
// bits (relative 2^-12; bf16 storage has 8), 6 terms 24 (fp32 storage), of
// numbers down to 2^-13 of the largest; of smaller ones what lies above 2^-27
// (2^-42) of it.  (32 is the largest step whose terms stay below 448: a rounding
// is off by 2^-5 of a number below 256.)  The
// terms are columns of the same MMA (N = terms * RC), so they cost nothing
// while N is small.
//
// Scales: a page's key scale multiplies its scores; its value scale
// v = f * 2^e, 1 <= f < 2, enters the softmax as t = s + e (log2 units), the
// weights as p * f and the normaliser as p * 2^-e, so that one running
// maximum keeps the weights within e4m3's range whatever the scales are.
//
// Work: tiles of 128 tokens of all units in one list, cut into equal ranges
// for two persistent CTAs per SM (page_sched.cuh); pieces of units that several
// CTAs share leave (maximum, normaliser, sums), and the CTA whose piece is done
// last merges them.
// Warps: 0-3 softmax (a thread per token; in the epilogue per output
// dimension), 4 TMA producer (lanes issue a tile's pages), 5 MMA issuer.
//
// What bounds it: long caches the read of the codes.  Single tokens of four
// sequences of 32K (32 heads on 8), replayed from a graph: 50 us, 5.3 TB/s or 0.81
// of the measured copy rate; 16K to 128K: 84 us, 6.0 TB/s or 0.91.  The rest is about 9 us of
// start and end: lengths, table, scales and codes one after another from
// memory, the pipeline's first tile, and the merge.  With one CTA per SM (six
// tiles in flight instead of three in each of two) 60 and 96 us, and 64 short
// sequences 91 us instead of 53, for which the overlap of one CTA's unit
// boundaries with the other's tiles counts most.  Short caches (4K tokens of 32
// heads: 13 us; 8K tokens of fp32 storage: 14) are that chain.
#include "page.cuh"
#include "tc.cuh"

namespace salsc {
namespace {

constexpr int kThreads = 192;
constexpr int kSoftmax = 128;
constexpr float kPScale = 128.f;  // weights p * f <= 2 become <= 256
constexpr float kStep = 32.f;     // a term counts 1 / kStep of the one before it
constexpr int kMaxPages = 8;      // pages of a tile (page size >= 16)

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 6 : 3;

template <typename T, int D, int RC>
struct Few {
  static constexpr int kN = (kTerms<T> * RC + 15) / 16 * 16;
  static constexpr int kTmem = 3 * kN <= 64 ? 64 : 3 * kN <= 128 ? 128 : 3 * kN <= 256 ? 256 : 512;
  // Two CTAs to an SM where tensor memory allows: one's tiles fly while the
  // other is at a softmax or between units.
  static constexpr int kCtas = kTmem <= 256 ? 2 : 1;
  static constexpr int kTileBytes = kPageTile * D;  // of K, and of V
  // tiles in flight: what fits with 4 KB for the static arrays
  static constexpr int kStages = (226 * 1024 / kCtas - 5 * 1024 - 3 * kN * 128) / (2 * kTileBytes);
  static constexpr int kOffQ = kStages * 2 * kTileBytes;
  static constexpr int kOffP = kOffQ + kN * 128;
  static constexpr int kSmem = kOffP + 2 * kN * 128 + 1024;  // + alignment
  static_assert(kStages >= 2, "tiles in flight");
};

// Scales and extent of one tile, written by the producer.
struct TileMeta {
  float ks[kMaxPages];   // key scale
  float vf[kMaxPages];   // value scale's mantissa f
  float ve[kMaxPages];   // its exponent e
  float ive[kMaxPages];  // 2^-e
  uint32_t loaded;       // pages that were loaded
};

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 f32x2(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
}

// Atomic add that other threads' stores before the last barrier precede, and
// that the block's loads after the next one follow, for the whole GPU.
__device__ __forceinline__ uint32_t add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

template <typename T, int D, int RC>
__global__ void __launch_bounds__(kThreads, Few<T, D, RC>::kCtas)
page_few_kernel(const __grid_constant__ PageStep s, const __grid_constant__ PageWork w,
                const T* __restrict__ q, int64_t q_stride, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const float* __restrict__ k_scales,
                const float* __restrict__ v_scales, T* __restrict__ out) {
  using C = Few<T, D, RC>;
  constexpr int kN = C::kN, kStages = C::kStages, kTile = C::kTileBytes, kT = kTerms<T>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TileMeta meta[kStages];
  __shared__ alignas(8) uint64_t bars[3 * kStages + 8];
  __shared__ alignas(16) float wmax[2][4][RC];
  __shared__ alignas(16) float wsum[4][RC];
  __shared__ float qfac[RC];     // softmax scale * log2(e) / the row's power of two
  __shared__ int rpos[RC];       // position of the row (a row that does not exist: -1)
  __shared__ int64_t rout[RC];   // its element offset in out
  __shared__ uint32_t tmem_base;
  __shared__ bool joins;         // this CTA's piece is the last of its unit to be done

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sm0 = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sm0 - tc::smem_u32(smem_raw));
  const uint32_t bar0 = tc::smem_u32(bars);
  auto kfull = [&](int i) { return bar0 + 8u * i; };
  auto vfull = [&](int i) { return bar0 + 8u * (kStages + i); };
  auto free_ = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto sready = [&](int i) { return bar0 + 8u * (3 * kStages + i); };
  auto pready = [&](int i) { return bar0 + 8u * (3 * kStages + 2 + i); };
  auto pvdone = [&](int i) { return bar0 + 8u * (3 * kStages + 4 + i); };
  const uint32_t qready = bar0 + 8u * (3 * kStages + 6), drained = bar0 + 8u * (3 * kStages + 7);

  if (tid == 0) {
    for (int i = 0; i < 3 * kStages; ++i) tc::mbar_init(bar0 + 8u * i, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(sready(i), 1);
      tc::mbar_init(pready(i), kSoftmax);
      tc::mbar_init(pvdone(i), 1);
    }
    tc::mbar_init(qready, kSoftmax);
    tc::mbar_init(drained, 1);
    tc::mbar_fence_init();
  }
  if (warp == 4 && lane < 2) tc::tma_prefetch_desc(lane ? &vmap : &kmap);
  // Behind page_many, which runs on other sequences and starts when all that
  // came before the step is done: this kernel's CTAs start where its CTAs have
  // ended, and wait for all of them at their own end.
  if (!w.overlaps) grid_dependency_wait();
  // (tensor memory last: a kernel before that starts to allocate must not find it taken
  // by one that waits for it)
  if (warp == 5) tc::tmem_alloc(tc::smem_u32(&tmem_base), C::kTmem);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  allow_dependent_launch();  // (a kernel that uses tensor memory must not come first to it)
  const uint32_t tmem = tmem_base;
  bool dead = false;  // a wait gave up: skip the others, so that the kernel ends
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead && !tc::mbar_wait(bar, parity, s.flags)) dead = true;
  };

  PageCursor cur(s, w);
  int64_t total, x1;
  if (page_begin(cur, total, x1)) {
    int it = 0;  // tiles so far
    const int npg = kPageTile / s.T;

    if (warp == 4) {
      // ------------------------------------------------ TMA producer
      bool gone = false;  // a lane gave up: the warp stops
      while (!gone) {
        const int n = cur.upto(x1);
        if (n <= 0) break;
        const int t0 = cur.blk.tile0(cur.k) + cur.tile;
        const int lo = cur.blk.lo(cur.k), hi = cur.blk.pos1(cur.k);
        // a batch of 32 pages: lane i holds page i; its loads fly one batch ahead
        const int per = 32 / npg;  // tiles of a batch
        auto look = [&](int tile) {
          const int64_t first = (int64_t)(t0 + tile) * kPageTile + (int64_t)lane * s.T;
          const bool need = tile + lane / npg < n && first <= hi && first + s.T > lo;
          return need ? page_of<true>(s, cur.b, (int)(first / s.T)) : -1;
        };
        int pg = look(0), big = kNoScale;
        float ks = 0.f, vs = 0.f;
        if (pg >= 0) {
          ks = __ldcg(k_scales + (size_t)pg * s.U + cur.u);
          vs = __ldcg(v_scales + (size_t)pg * s.U + cur.u);
        }
        for (int i0 = 0; i0 < n && !gone; i0 += per) {
          const int pg_n = i0 + per < n ? look(i0 + per) : -1;
          float ks_n = 0.f, vs_n = 0.f;
          for (int i = i0; i < min(n, i0 + per); ++i, ++it) {
            const int st = it % kStages;
            if (i == min(n, i0 + per) - 1 && pg_n >= 0) {
              ks_n = __ldcg(k_scales + (size_t)pg_n * s.U + cur.u);
              vs_n = __ldcg(v_scales + (size_t)pg_n * s.U + cur.u);
            }
            wait(free_(st), ((it / kStages) & 1) ^ 1);
            if ((gone = __any_sync(0xffffffffu, dead))) break;
            const bool mine = lane / npg == i - i0;
            const int sub = lane % npg;
            const uint32_t got = __ballot_sync(0xffffffffu, mine && pg >= 0);
            // the copies first: the scales may still be on their way
            if (mine && pg >= 0) {
              const uint32_t dst = sm0 + (uint32_t)st * 2 * kTile + (uint32_t)sub * s.T * D;
              const int row = (pg * s.U + cur.u) * s.T;
              tc::tma_load_2d(dst, &kmap, 0, row, kfull(st));
              tc::tma_load_2d(dst + kTile, &vmap, 0, row, vfull(st));
            }
            big = max(big, __reduce_max_sync(0xffffffffu, mine ? scale_exponent(vs) : kNoScale));
            if (mine) {
              const ValueScale v = value_scale(vs, big);
              meta[st].ks[sub] = key_scale(ks);
              meta[st].vf[sub] = v.f;
              meta[st].ve[sub] = v.e;
              meta[st].ive[sub] = v.down;
              if (sub == 0) meta[st].loaded = got >> (npg * (i - i0));
            }
            __syncwarp();
            const uint32_t bytes = (uint32_t)__popc(got) * s.T * D;
            if (lane == 0) {
              tc::mbar_expect_tx(kfull(st), bytes);
              tc::mbar_expect_tx(vfull(st), bytes);
            }
            __syncwarp();
          }
          pg = pg_n;
          ks = ks_n;
          vs = vs_n;
        }
        if (!cur.next_unit()) break;
      }
      // the copies in flight land before the block ends
      if (gone)
        for (int k = max(it - kStages, 0); k < it; ++k) {
          tc::mbar_wait(kfull(k % kStages), (k / kStages) & 1, s.flags);
          tc::mbar_wait(vfull(k % kStages), (k / kStages) & 1, s.flags);
        }
    } else if (warp == 5) {
      // ------------------------------------------------ MMA issuer
      if (tc::elect_one()) {
        const uint32_t id_s = tc::idesc_e4m3_f32(128, kN, false);
        const uint32_t id_o = tc::idesc_e4m3_f32(128, kN, true);
        const uint32_t qs = sm0 + C::kOffQ;
        auto scores = [&](int i) {
          const int st = i % kStages;
          const uint32_t k = sm0 + (uint32_t)st * 2 * kTile;
          wait(kfull(st), (i / kStages) & 1);
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            tc::mma_f8(tmem + (i & 1) * kN,
                       D == 128 ? tc::sdesc_kmajor_sw128(k + kk * 32)
                                : tc::sdesc_sw64(k + kk * 32, 16, 512),
                       tc::sdesc_kmajor_sw128(qs + kk * 32), id_s, kk > 0);
          tc::mma_commit(sready(i & 1));
        };
        auto values = [&](int i, bool first) {
          const int st = i % kStages;
          const uint32_t v = sm0 + (uint32_t)st * 2 * kTile + kTile;
          const uint32_t p = sm0 + C::kOffP + (i & 1) * kN * 128;
          wait(vfull(st), (i / kStages) & 1);
          wait(pready(i & 1), (i >> 1) & 1);
          tc::fence_after_sync();
          // 32 tokens to an MMA; for d = 64 the second 64 rows of D repeat the first
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_f8(tmem + 2 * kN,
                       D == 128 ? tc::sdesc_mnmajor_sw128(v + kk * 4096, 16384, 1024)
                                : tc::sdesc_sw64(v + kk * 2048, 0, 512),
                       tc::sdesc_kmajor_sw128(p + kk * 32), id_o, !first || kk > 0);
          tc::mma_commit(pvdone(i & 1));
          tc::mma_commit(free_(st));
        };
        for (int seg = 0;; ++seg) {
          const int n = cur.upto(x1);
          if (n <= 0) break;
          wait(qready, seg & 1);
          scores(it);
          for (int i = 0; i < n; ++i, ++it) {
            if (i + 1 < n) scores(it + 1);
            values(it, i == 0);
          }
          if (!cur.next_unit()) break;
        }
        if (dead) {  // and so do the MMAs, before tensor memory is given back
          tc::mma_commit(drained);
          tc::mbar_wait(drained, 0, s.flags);
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------ softmax
      const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
      const int weff = s.window ? s.window : INT32_MAX;
      while (true) {
        const int n = cur.upto(x1);
        if (n <= 0) break;
        const int t0 = cur.blk.tile0(cur.k) + cur.tile;
        const int p0 = cur.blk.pos0(cur.k), p1 = cur.blk.pos1(cur.k);
        const int rows = (p1 - p0 + 1) * s.G;
        const int row0 = cur.row0 + cur.k * w.tb;
        // tokens that every row sees: [all_lo, p0]
        const int all_lo = p1 - p0 < weff && s.window ? max(p1 - weff + 1, 0) : (s.window ? INT32_MAX : 0);
        const int any_lo = cur.blk.lo(cur.k);

        // the rows' terms: a warp per row
        for (int r = warp; r < RC; r += 4) {
          const int i = r / s.G, g = r - i * s.G;
          float x2[D / 64][2];
          float amax = 0.f;
          if (r < rows) {
            const T* src = q + (int64_t)(row0 + i) * q_stride + (cur.u * s.G + g) * D;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
              const int e = lane + 32 * j;
              const float a = to_f32(__ldcg(src + e)), c2 = to_f32(__ldcg(src + e + D / 2));
              float c = 1.f, sn = 0.f;
              if (s.rotate) page_cs(p0 + i, s.turns[e], c, sn);
              x2[j][0] = a * c - c2 * sn;
              x2[j][1] = c2 * c + a * sn;
              // e4m3 has no infinity: NaN, as the scores would be
              x2[j][0] += x2[j][0] - x2[j][0];
              x2[j][1] += x2[j][1] - x2[j][1];
              amax = fmaxf(amax, fmaxf(fabsf(x2[j][0]), fabsf(x2[j][1])));
            }
          } else {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) x2[j][0] = x2[j][1] = 0.f;
          }
          amax = warp_max(amax);
          // power of two that brings the row's largest element into [128, 256)
          int ex = (int)(__float_as_uint(amax) >> 23) - 127 - 7;
          ex = max(ex, -119);
          const float mul = __uint_as_float((uint32_t)(127 - ex) << 23);
          if (lane == 0) {
            qfac[r] = s.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + ex) << 23);
            rpos[r] = r < rows ? p0 + i : -1;
            rout[r] = ((int64_t)(row0 + i) * s.Hq + cur.u * s.G + g) * D;
          }
          unsigned char* dst = smem + C::kOffQ;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            float a = x2[j][0] * mul, c2 = x2[j][1] * mul;
            const int e = lane + 32 * j;
#pragma unroll
            for (int t = 0; t < kT; ++t) {
              const uint32_t c = e4m3x2(a, c2);
              const float2 f = f32x2(c);
              const int nrow = t * RC + r;
              dst[nrow * 128 + (e ^ ((nrow & 7) << 4))] = (unsigned char)c;
              dst[nrow * 128 + ((e + D / 2) ^ ((nrow & 7) << 4))] = (unsigned char)(c >> 8);
              a = (a - f.x) * kStep;
              c2 = (c2 - f.y) * kStep;
            }
          }
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(qready);
        tc::named_sync(1, kSoftmax);  // qfac, rpos, rout

        float m[RC], l[RC];
#pragma unroll
        for (int r = 0; r < RC; ++r) {
          m[r] = -INFINITY;
          l[r] = 0.f;
        }
        for (int i = 0; i < n; ++i, ++it) {
          const int st = it % kStages, buf = it & 1;
          const int64_t tile0 = (int64_t)(t0 + i) * kPageTile;
          const int tok = (int)min(tile0 + tid, (int64_t)INT32_MAX);
          wait(kfull(st), (it / kStages) & 1);
          wait(sready(buf), (it >> 1) & 1);
          tc::fence_after_sync();
          const TileMeta& mt = meta[st];
          const int pgi = tid / s.T;
          const float ks = mt.ks[pgi], ve = mt.ve[pgi], ive = mt.ive[pgi];
          float vf = mt.vf[pgi];
          const bool full = tile0 >= all_lo && tile0 + kPageTile - 1 <= p0 &&
                            mt.loaded == (1u << npg) - 1u;
          float t[RC];
#pragma unroll
          for (int r0 = 0; r0 < RC; r0 += (RC < 8 ? RC : 8)) {
            constexpr int kW = RC < 8 ? RC : 8;
            if constexpr (RC < 8) {
              // all terms in one load
              uint32_t v[16];
              tc::tmem_ld16(lanes + buf * kN, v);
              uint32_t v2[16];
              if constexpr (kN > 16) tc::tmem_ld16(lanes + buf * kN + 16, v2);
              tc::tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < RC; ++r) {
                float a = 0.f;
#pragma unroll
                for (int k = kT - 1; k >= 0; --k) {
                  const int c = k * RC + r;
                  const float vv = __uint_as_float(c < 16 ? v[c] : v2[c - 16]);
                  a = k == kT - 1 ? vv : fmaf(a, 1.f / kStep, vv);
                }
                t[r] = a;
              }
            } else {
              uint32_t v[kT][8];
#pragma unroll
              for (int k = 0; k < kT; ++k) tc::tmem_ld8(lanes + buf * kN + k * RC + r0, v[k]);
              tc::tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < kW; ++r) {
                float a = __uint_as_float(v[kT - 1][r]);
#pragma unroll
                for (int k = kT - 2; k >= 0; --k) a = fmaf(a, 1.f / kStep, __uint_as_float(v[k][r]));
                t[r0 + r] = a;
              }
            }
          }
#pragma unroll
          for (int r = 0; r < RC; ++r) t[r] = fmaf(t[r], qfac[r] * ks, ve);
          if (!full) {
            const bool there = (mt.loaded >> pgi) & 1u;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
              const int pos = rpos[r];
              if (!there || tok > pos || pos - tok >= weff) t[r] = -INFINITY;
            }
            // Values that no row sees may be anything, and values that some rows
            // do not see may be NaN, which a weight of zero would not hide: such
            // rows of the tile become zeros, and a NaN is handed to the rows that
            // see it by their weights.
            wait(vfull(st), (it / kStages) & 1);
            uint4* vrow = (uint4*)(smem + (size_t)st * 2 * kTile + kTile + tid * D);
            bool clear = !there || tok > p1 || tok < any_lo;
            if (!clear) {
              bool nan = false;
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint4 c = vrow[k];
                nan |= has_nan(c.x) || has_nan(c.y) || has_nan(c.z) || has_nan(c.w);
              }
              if (nan) {
                clear = true;
                vf = __uint_as_float(0x7FC00000u);
              }
            }
            if (clear) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) vrow[k] = make_uint4(0, 0, 0, 0);
            }
          }
          // the tile's maximum, over the four warps
          {
            float tm[RC];
#pragma unroll
            for (int r = 0; r < RC; ++r) tm[r] = warp_max(t[r]);
            if (lane == 0) {
#pragma unroll
              for (int r = 0; r < RC; r += 4)
                *(float4*)&wmax[buf][warp][r] = make_float4(tm[r], tm[r + 1], tm[r + 2], tm[r + 3]);
            }
          }
          tc::named_sync(1, kSoftmax);
          float al[RC];
          bool grew = false;
#pragma unroll
          for (int r = 0; r < RC; r += 4) {
            float4 a = *(const float4*)&wmax[buf][0][r];
#pragma unroll
            for (int k = 1; k < 4; ++k) {
              const float4 c = *(const float4*)&wmax[buf][k][r];
              a.x = fmaxf(a.x, c.x);
              a.y = fmaxf(a.y, c.y);
              a.z = fmaxf(a.z, c.z);
              a.w = fmaxf(a.w, c.w);
            }
            const float nm[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float mm = fmaxf(m[r + k], nm[k]);
              al[r + k] = m[r + k];
              grew |= !(mm == m[r + k]);
              m[r + k] = mm;
            }
          }
          if (grew) {
#pragma unroll
            for (int r = 0; r < RC; ++r) {
              // in two steps, as page_factor
              const float h = al[r] == m[r] ? 1.f : ex2(0.5f * (al[r] - m[r]));
              l[r] = l[r] * h * h;
              al[r] = h * h;
            }
            if (i > 0) {  // the sums so far (of this piece) follow the maximum
              wait(pvdone(buf ^ 1), ((it - 1) >> 1) & 1);
              tc::fence_after_sync();
#pragma unroll
              for (int c0 = 0; c0 < kN; c0 += 16) {
                uint32_t v[16];
                tc::tmem_ld16(lanes + 2 * kN + c0, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  v[c] = __float_as_uint(__uint_as_float(v[c]) * al[(c0 + c) % RC]);
                tc::tmem_st16(lanes + 2 * kN + c0, v);
              }
              tc::tmem_st_wait();
            }
          }
          if (it >= 2) wait(pvdone(buf), ((it - 2) >> 1) & 1);  // P's buffer is free
          unsigned char* dst = smem + C::kOffP + buf * kN * 128;
          const float vfp = vf * kPScale;
#pragma unroll
          for (int r = 0; r < RC; r += 2) {
            // (a row that has seen nothing: its t are -inf, whatever they refer to)
            const float p0 = ex2(t[r] - (m[r] == -INFINITY ? 0.f : m[r]));
            const float p1 = ex2(t[r + 1] - (m[r + 1] == -INFINITY ? 0.f : m[r + 1]));
            l[r] = fmaf(p0, ive, l[r]);
            l[r + 1] = fmaf(p1, ive, l[r + 1]);
            float y0 = p0 * vfp, y1 = p1 * vfp;
            if (!full) {  // vf may be a NaN that not all rows see
              y0 = t[r] == -INFINITY ? 0.f : y0;
              y1 = t[r + 1] == -INFINITY ? 0.f : y1;
            }
#pragma unroll
            for (int k = 0; k < kT; ++k) {
              const uint32_t c = e4m3x2(y0, y1);
              const int n0 = k * RC + r;
              dst[n0 * 128 + (tid ^ ((n0 & 7) << 4))] = (unsigned char)c;
              dst[(n0 + 1) * 128 + (tid ^ (((n0 + 1) & 7) << 4))] = (unsigned char)(c >> 8);
              if (k + 1 < kT) {
                const float2 f = f32x2(c);
                add2(y0, y1, -f.x, -f.y);
                mul2(y0, y1, kStep);
              }
            }
          }
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();
          tc::mbar_arrive(pready(buf));
        }

        // ---- the piece's result
#pragma unroll
        for (int r = 0; r < RC; ++r) {
          float a = l[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          if (lane == 0) wsum[warp][r] = a;
        }
        wait(pvdone((it - 1) & 1), ((it - 1) >> 1) & 1);
        tc::fence_after_sync();
        tc::named_sync(1, kSoftmax);
        const bool whole = cur.whole(n);
        const int slot = 2 * blockIdx.x + (cur.tile == 0 ? 1 : 0);
        if (!whole && tid < rows) {
          float mm = 0.f;
#pragma unroll
          for (int r = 0; r < RC; ++r)
            if (r == tid) mm = m[r];
          const float ll = wsum[0][tid] + wsum[1][tid] + wsum[2][tid] + wsum[3][tid];
          w.ml[(size_t)slot * w.rows + tid] = make_float2(mm, ll);
        }
        if (warp * 32 < D) {
#pragma unroll
          for (int r0 = 0; r0 < RC; r0 += 4) {
            uint32_t v[kT][2][2];
#pragma unroll
            for (int k = 0; k < kT; ++k) {
              tc::tmem_ld2(lanes + 2 * kN + k * RC + r0, v[k][0]);
              tc::tmem_ld2(lanes + 2 * kN + k * RC + r0 + 2, v[k][1]);
            }
            tc::tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (r0 + r < rows) {
                float a = __uint_as_float(v[kT - 1][r / 2][r % 2]);
#pragma unroll
                for (int k = kT - 2; k >= 0; --k) a = fmaf(a, 1.f / kStep, __uint_as_float(v[k][r / 2][r % 2]));
                a *= 1.f / kPScale;
                if (whole) {
                  const float ll = wsum[0][r0 + r] + wsum[1][r0 + r] + wsum[2][r0 + r] + wsum[3][r0 + r];
                  out[rout[r0 + r] + tid] = from_f32<T>(ll == 0.f ? 0.f : a / ll);
                } else {
                  w.acc[((size_t)slot * w.rows + r0 + r) * D + tid] = a;
                }
              }
            }
          }
        }
        if (!whole) {
          // the CTA whose piece is done last merges the unit's
          const int c0 = (int)share_of_tile(cur.base + w.over, total, gridDim.x);
          const int pieces = (int)share_of_tile(cur.last(), total, gridDim.x) - c0 + 1;
          tc::named_sync(1, kSoftmax);
          if (tid == 0) {
            joins = add_acq_rel(&w.done[c0], 1u) == (uint32_t)pieces - 1;
            if (joins) w.done[c0] = 0;
          }
          tc::named_sync(1, kSoftmax);
          if (joins)
            for (int r = warp; r < rows; r += 4) page_merge_row<T, D>(w, c0, pieces, r, out + rout[r]);
        }
        tc::fence_before_sync();
        tc::named_sync(1, kSoftmax);  // wsum, qfac, rpos, rout are free
        if (!cur.next_unit()) break;
      }
    }
  }
  __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tmem, C::kTmem);
  if (w.overlaps) grid_dependency_wait();
}

template <typename T, int D, int RC>
cudaError_t launch(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                   const void* kp, const void* vp, const float* ks, const float* vs, void* out,
                   cudaStream_t stream) {
  static int done[kMaxDevices];
  using C = Few<T, D, RC>;
  auto kern = page_few_kernel<T, D, RC>;
  const cudaError_t e = ensure_smem(kern, C::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)s.n_pages * s.U * s.T;
  if (!make_tmap_u8_rows(&km, kp, rows, D, s.T) || !make_tmap_u8_rows(&vm, vp, rows, D, s.T))
    return cudaErrorInvalidValue;
  return launch_k(kern, dim3(w.grid), dim3(kThreads), C::kSmem, stream, true, s, w, (const T*)q,
                  q_stride, km, vm, ks, vs, (T*)out);
}

template <typename T, int D>
cudaError_t launch_d(int rc, const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                     const void* kp, const void* vp, const float* ks, const float* vs, void* out,
                     cudaStream_t stream) {
  switch (rc) {
    case 4: return launch<T, D, 4>(s, w, q, q_stride, kp, vp, ks, vs, out, stream);
    case 8: return launch<T, D, 8>(s, w, q, q_stride, kp, vp, ks, vs, out, stream);
    default: return launch<T, D, 16>(s, w, q, q_stride, kp, vp, ks, vs, out, stream);
  }
}

}  // namespace

int page_few_rows(int64_t want) {
  int rc = 4;
  while (rc < 16 && rc < want) rc *= 2;
  return rc;
}

int page_few_grid(int rows, salsc_dtype dt) {
  const int n = (dt == SALSC_F32 ? kTerms<float> : kTerms<__nv_bfloat16>) * rows;
  return n > 80 ? kPageGrid : 2 * kPageGrid;  // as Few::kCtas
}

cudaError_t launch_page_few(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                            const void* k_pages, const void* v_pages, const float* k_scales,
                            const float* v_scales, void* out, salsc_dtype dt, cudaStream_t stream) {
  if (dt == SALSC_BF16)
    return s.d == 64 ? launch_d<__nv_bfloat16, 64>(w.rows, s, w, q, q_stride, k_pages, v_pages,
                                                   k_scales, v_scales, out, stream)
                     : launch_d<__nv_bfloat16, 128>(w.rows, s, w, q, q_stride, k_pages, v_pages,
                                                    k_scales, v_scales, out, stream);
  return s.d == 64 ? launch_d<float, 64>(w.rows, s, w, q, q_stride, k_pages, v_pages, k_scales,
                                         v_scales, out, stream)
                   : launch_d<float, 128>(w.rows, s, w, q, q_stride, k_pages, v_pages, k_scales,
                                          v_scales, out, stream);
}

}  // namespace salsc
