// page_many.cu -- attention of many query rows over the paged 8-bit cache
// (prompts and chunks of prompts, bf16 storage).
//
//   s_t = RoPE(q) . K_t,  p = softmax(scale * s),  out = sum_t p_t V_t
//
// A row block is two halves of 128 rows: each half the query heads of one KV
// head for floor(128 / G) consecutive new tokens.  Per tile of 128 tokens and
// half, on tcgen05 kind::f16 with fp32 accumulators in TMEM:
//   S [128 x 128 tokens]  = Q (K-major)         x  K tile (K-major)
//   O [128 x d]          += P (A from TMEM)     x  V tile (MN-major)
// e4m3 codes are exact in f16, which also gives the rotated queries and the
// weights 11 bits.  Codes are read once per tile and both halves use them.
//
// Scales: a page's key scale multiplies its scores; its value scale
// v = f * 2^e, 1 <= |f| < 2, enters the softmax as t = s + e (log2 units) and
// the normaliser as p * 2^-e; f goes into the f16 values (nothing, and exact,
// for the powers of two that the append writes; two roundings of 2^-12 for
// others).
// So the weights 2^(t - m) stay in f16's range whatever the scales are.
//
// The weights refer to a maximum that follows the rows' only when it must: a
// tile's weights are computed with what is at hand, and only if their sum
// reaches kMost (none is larger then, and f16 holds them as well) computed again
// with the tile's own maximum, when O is rescaled too.  So no maximum stands
// between the scores and the exponentials of most tiles.  What they refer to lies
// 2^kUp below the maximum, in the middle between f16's largest number and kMost's
// room to grow: weights keep 11 bits down to 2^-21 of the largest, and smaller
// ones what lies above 2^-32 of it.
//
// Roles (512 threads, one CTA per SM): warps 0-3 and 4-7 softmax of a half (a
// thread per row), warps 8-11 cache tiles (codes to f16), warp 12 issues the
// MMAs, warp 13 copies queries and pages to shared memory (warps 14 and 15 are
// there because registers are shared out by four warps).  Each role's loop is
// kept short: unrolled over a whole tile they came to 40 KB, and waiting for
// instructions was the largest stall.
//
// The queries are rotated by a kernel before (page_rotate_kernel): with a row
// block's rotation inside the attention, every unit began with 25 us of it.
//
// What bounds it: a half's tile is a chain of scores (512 cycles of MMAs), their
// load, 128 exponentials a thread (1024 cycles of the MUFU pipe if nobody else
// asks) and values (512); two halves in flight cover each other only in part,
// and a tile takes 4000 to 4200 cycles where the MMAs alone need 2048 and the
// exponentials as much: MMA and MUFU pipes 52 % busy, issue slots 37 %.
// Measured: 2048 tokens at the end of 32K, 32 heads on 8: 1.05 ms, 1.02 PFLOP/s.
// Tried and slower: 16 softmax warps with two threads to a row (1.12 ms against
// 1.08 then), scores by 64 tokens in turn (1.19 against 1.06), the halves taking
// turns at the exponentials (1.16 against 1.06).
#include "page.cuh"
#include "tc.cuh"

namespace salsc {
namespace {

constexpr int kThreads = 512;
constexpr int kRegisters = 128; // a thread, at launch: shared out anew by the roles
constexpr int kConvert = 128;   // threads of the converting warps
constexpr int kRing = 4;        // tiles whose scales are kept
constexpr float kUp = 7.f;        // log2 of the weight of the maximum that weights refer to
constexpr float kMost = 32768.f;  // sum of a tile's weights that the maximum must follow

// What the copying warp says of a tile, by group of 16 tokens.
struct alignas(16) TileScales {  // read by float4
  float ks[8], ve[8], ive[8];  // key scale; value scale f * 2^e: e, 2^-e
  uint32_t vf[8];              // f, twice in f16
  uint32_t loaded;             // groups that were loaded (bits)
  bool plain;                  // all f are 1
};

// A segment: a piece of one unit, this CTA's tiles of it.  Warp 13 writes them.
struct alignas(16) Segment {
  int n, t0;    // tiles (0: there are no more segments), first tile
  int p0, p1;   // positions of the unit's first and last row
  int lo;       // first token that any row sees
  int all_lo;   // first token that no row sees too late (window)
  int row;      // token row of the first row
  short u;      // KV head
  bool starts, whole;  // the unit's first tile is in the segment; all of them are
};
// An entry is read until its last tile's results are out. All readers say when they are done with
// it, and the copying warp waits for that before it writes the entry again: the softmax warps of
// the second half take part in no other barrier while units have one half only.
constexpr int kSegments = 8;
constexpr int kReaders = 13;  // warps: softmax 8, converting 4, MMA 1

struct Shared {
  Segment segments[kSegments];
  TileScales meta[kRing];
  uint32_t nan[2 * kRing][4];  // tokens whose values hold a NaN, where rows differ in what they see
  uint64_t bars[21 + 2 * kSegments];
  uint32_t tmem_base;
};

template <int D>
struct Many {
  static constexpr int kQHalf = 128 * D * 2;  // bytes
  static constexpr int kTileBytes = kPageTile * D * 2;
  static constexpr int kOffK = 2 * kQHalf;
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffCodes = kOffV + 2 * kTileBytes;  // of K, then of V
  static constexpr int kCodeBytes = kPageTile * D;
  static constexpr int kOffShared = kOffCodes + 2 * kCodeBytes;
  static constexpr int kSmem = kOffShared + (int)sizeof(Shared);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static constexpr int kTmem = 512;
  static constexpr int kColO = 256;
};

// 16 e4m3 codes -> 16 f16 in two chunks.
__device__ __forceinline__ void widen16(const uint4& c, uint32_t (&w)[8]) {
  const uint32_t x[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
        : "r"(x[i]));
}

// 32 bytes, the size of a sector: rows are apart, a thread has one to itself.
__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *(const uint32_t*)&h;
}

// Queries of the sequences that this file's attention takes, rotated, as f16
// times a power of two for each row: qrot [n_tokens][Hq][d], exponents
// qexp [n_tokens][Hq].  A warp per token and kRotateHeads heads, whose rows it
// loads at once; lanes hold two (d = 64: one) pairs, whose cos and sin serve
// those heads.  Bound by memory: 2 bytes in, 2 out.  With a warp per token, four
// of its rows at a time, a prompt of 4096 tokens and 32 heads took 227 us in all,
// with this and page_merge_kernel's four rows a warp 216.
constexpr int kRotateWarps = 8, kRotateHeads = 8;
template <int D>
__global__ void __launch_bounds__(kRotateWarps * 32)
page_rotate_kernel(const __grid_constant__ PageStep s, const __grid_constant__ PageWork w,
                   const __nv_bfloat16* __restrict__ q, int64_t q_stride) {
  constexpr int kP = D / 64;  // pairs of a lane
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRotateWarps + (threadIdx.x >> 5), h0 = blockIdx.y * kRotateHeads;
  grid_dependency_wait();
  allow_dependent_launch();
  if (t >= s.n_tokens) return;
  // the last sequence whose first row is at or before t, by 32 tries at a time
  int b = s.offs ? 0 : min(t, s.B - 1), n = s.offs ? s.B : 1;
  while (n > 1) {
    const int step = (n + 31) / 32, k = b + lane * step;
    const bool at = k < b + n && (s.offs[k] <= t);
    const int hit = max(__popc(__ballot_sync(0xffffffffu, at)) - 1, 0);
    n = min(step, n - hit * step);
    b += hit * step;
  }
  const PageSeq sq = page_seq<false>(s, b);
  const int64_t rows = (int64_t)sq.m * s.G;
  if (rows < w.min_rows || rows > w.max_rows || t < sq.row0 || t >= sq.row0 + sq.m) return;
  const int pos = sq.n - sq.m + (t - sq.row0);
  const __nv_bfloat16* src = q + (int64_t)t * q_stride + kP * lane;
  uint32_t xa[kRotateHeads], xb[kRotateHeads];  // d = 64: one element each
#pragma unroll
  for (int j = 0; j < kRotateHeads; ++j) {
    const int h = min(h0 + j, s.Hq - 1);
    if constexpr (kP == 2) {
      xa[j] = *(const uint32_t*)(src + h * D);
      xb[j] = *(const uint32_t*)(src + h * D + D / 2);
    } else {
      xa[j] = *(const uint16_t*)(src + h * D);
      xb[j] = *(const uint16_t*)(src + h * D + D / 2);
    }
  }
  float c[kP], sn[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    c[i] = 1.f, sn[i] = 0.f;
    if (s.rotate && pos >= 0) page_cs(pos, s.turns[kP * lane + i], c[i], sn[i]);
  }
  __half* dst = (__half*)w.qrot + (int64_t)t * s.Hq * D + kP * lane;
#pragma unroll
  for (int j = 0; j < kRotateHeads; ++j) {
    const int h = h0 + j;
    float x[kP], y[kP], am = 0.f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const float a = __uint_as_float(i ? xa[j] & 0xFFFF0000u : xa[j] << 16);
      const float b2 = __uint_as_float(i ? xb[j] & 0xFFFF0000u : xb[j] << 16);
      x[i] = a * c[i] - b2 * sn[i], y[i] = b2 * c[i] + a * sn[i];
      // an infinity becomes NaN: scores of -inf alone would leave a row that sees nothing
      x[i] += x[i] - x[i], y[i] += y[i] - y[i];
      am = fmaxf(am, fmaxf(fabsf(x[i]), fabsf(y[i])));
    }
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(am));
    // power of two that brings the row's largest element into [2^7, 2^8)
    int ex = (int)(__float_as_uint(am) >> 23) - 127 - 7;
    ex = max(ex, -119);
    const float mul = __uint_as_float((uint32_t)(127 - ex) << 23);
    if (h < s.Hq) {
      if constexpr (kP == 2) {
        *(uint32_t*)(dst + h * D) = half2_bits(x[0] * mul, x[1] * mul);
        *(uint32_t*)(dst + h * D + D / 2) = half2_bits(y[0] * mul, y[1] * mul);
      } else {
        dst[h * D] = __float2half_rn(x[0] * mul);
        dst[h * D + D / 2] = __float2half_rn(y[0] * mul);
      }
      if (lane == 0) w.qexp[(int64_t)t * s.Hq + h] = (int8_t)ex;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
page_many_kernel(const __grid_constant__ PageStep s, const __grid_constant__ PageWork w,
                 const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const float* __restrict__ k_scales,
                 const float* __restrict__ v_scales, __nv_bfloat16* __restrict__ out) {
  using C = Many<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared& sh = *(Shared*)(smem + C::kOffShared);
  auto& meta = sh.meta;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sm0 = tc::smem_u32(smem);
  const uint32_t bar0 = tc::smem_u32(sh.bars);
  auto kfull = [&](int i) { return bar0 + 8u * i; };
  auto kfree = [&](int i) { return bar0 + 8u * (2 + i); };
  auto vfull = [&](int i) { return bar0 + 8u * (4 + i); };
  auto vfree = [&](int i) { return bar0 + 8u * (6 + i); };
  auto sready = [&](int h) { return bar0 + 8u * (8 + h); };
  auto pready = [&](int h) { return bar0 + 8u * (10 + h); };
  auto odone = [&](int h) { return bar0 + 8u * (12 + h); };

  const uint32_t qfull = bar0 + 8u * 14, qfree = bar0 + 8u * 15;
  auto cfull = [&](int v) { return bar0 + 8u * (16 + v); };  // codes of K, of V
  auto cfree = [&](int v) { return bar0 + 8u * (18 + v); };
  auto segfull = [&](int i) { return bar0 + 8u * (20 + i % kSegments); };
  const uint32_t drained = bar0 + 8u * (20 + 2 * kSegments);
  auto segfree = [&](int i) { return bar0 + 8u * (20 + kSegments + i % kSegments); };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(kfull(i), kConvert);
      tc::mbar_init(kfree(i), 1);
      tc::mbar_init(vfull(i), kConvert);
      tc::mbar_init(vfree(i), 1);
      tc::mbar_init(sready(i), 2);  // the scores, and the issuer for what it has waited for
      tc::mbar_init(pready(i), 128);
      tc::mbar_init(odone(i), 1);
      tc::mbar_init(cfull(i), 1);
      tc::mbar_init(cfree(i), kConvert);
    }
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qfree, 1);
    tc::mbar_init(drained, 1);
    for (int i = 0; i < kSegments; ++i) {
      tc::mbar_init(segfull(i), 1);
      tc::mbar_init(segfree(i), kReaders);
    }
    tc::mbar_fence_init();
  }
  if (warp == 13 && lane < 3) tc::tma_prefetch_desc(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
  if (warp == 12) tc::tmem_alloc(tc::smem_u32(&sh.tmem_base), C::kTmem);
  if (tid < 2 * kRing * 4) sh.nan[tid / 4][tid % 4] = 0;
  // page_rotate_kernel, launched right before, has waited for all that came before
  // it, so only its own output is waited for: where queries are copied and where
  // their exponents are read, and by all at the end (a kernel that waits for this
  // one counts on it).  What is read earlier comes past L1.
  if (tid == 0) w.info[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  allow_dependent_launch();  // (a kernel that uses tensor memory must not come first to it)
  const uint32_t tmem = sh.tmem_base;
  bool dead = false;  // a wait gave up: skip the others, so that the kernel ends
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead && !tc::mbar_wait(bar, parity, s.flags)) dead = true;
  };
  const int tb2 = w.tb / 2;  // new tokens of a half

  {
    int it = 0;  // tiles so far
    auto segment = [&](int i) -> const Segment& {
      wait(segfull(i), (i / kSegments) & 1);
      return sh.segments[i % kSegments];
    };
    auto gone = [&] { return (bool)__any_sync(0xffffffffu, dead); };  // a lane gave up: the warp stops
    auto read = [&](int i) {  // the warp is done with the entry
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(segfree(i));
    };
    auto writable = [&](int i) -> Segment& {
      wait(segfree(i), ((i / kSegments) & 1) ^ 1);
      return sh.segments[i % kSegments];
    };
    static_assert(200 * 256 + 64 * 128 + 48 * 128 == kRegisters * kThreads, "registers");
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      // ------------------------------------------------ MMA issuer
      // All lanes run it, so that the compiler sees that descriptors and addresses
      // are the warp's and keeps them in uniform registers; one lane issues.
      if (warp == 12) {
        const uint32_t lead = tc::elect_one();
        constexpr uint32_t id_s = tc::idesc_f16_f32(128, kPageTile, false);
        constexpr uint32_t id_o = tc::idesc_f16_f32(128, D, true);
        int cnt[2] = {0, 0};
        auto scores = [&](int h, int i) {
          const uint64_t qa = tc::sdesc_kmajor_sw128(sm0 + (uint32_t)h * C::kQHalf);
          const uint64_t ka = tc::sdesc_kmajor_sw128(sm0 + C::kOffK + (uint32_t)(i & 1) * C::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
            tc::mma_lead(lead, tmem + h * 128, qa + off, ka + off, id_s, kk > 0);
          }
          tc::commit_lead(lead, sready(h));
          if (lead) tc::mbar_arrive(sready(h));
        };
        auto values = [&](int h, int i, bool first) {
          const uint64_t va =
              tc::sdesc_mnmajor_sw128(sm0 + C::kOffV + (uint32_t)(i & 1) * C::kTileBytes, 16384, 1024);
          wait(pready(h), cnt[h]++ & 1);
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < kPageTile / 16; ++kk)
            tc::mma_ts_lead(lead, tmem + C::kColO + h * D, tmem + h * 128 + kk * 8, va + (kk * 2048 >> 4), id_o,
                            !first || kk > 0);
          tc::commit_lead(lead, odone(h));
        };
        for (int seg = 0;; ++seg) {
          const Segment& sg = segment(seg);
          const int n = gone() ? 0 : __shfl_sync(0xffffffffu, sg.n, 0);
          if (n == 0) break;
          const bool two = __shfl_sync(0xffffffffu, sg.p1 - sg.p0, 0) >= tb2;
          read(seg);
          wait(qfull, seg & 1);
          wait(kfull(it & 1), (it >> 1) & 1);
          tc::fence_after_sync();
          scores(0, it);
          if (two) scores(1, it);
          tc::commit_lead(lead, kfree(it & 1));
          if (n == 1) tc::commit_lead(lead, qfree);
          for (int i = 0; i < n; ++i, ++it) {
            wait(vfull(it & 1), (it >> 1) & 1);
            if (i + 1 < n) wait(kfull((it + 1) & 1), ((it + 1) >> 1) & 1);
            values(0, it, i == 0);
            if (i + 1 < n) scores(0, it + 1);
            if (two) values(1, it, i == 0);
            tc::commit_lead(lead, vfree(it & 1));
            if (i + 1 < n) {
              if (two) scores(1, it + 1);
              tc::commit_lead(lead, kfree((it + 1) & 1));
              if (i + 2 == n) tc::commit_lead(lead, qfree);
            }
          }
        }
        if (gone()) {  // the MMAs in flight end before tensor memory is given back
          tc::commit_lead(lead, drained);
          tc::mbar_wait(drained, 0, s.flags);
        }
      }
      // ------------------------------------------------ pages to shared memory
      if (warp == 13) {
        PageCursor cur(s, w);
        int64_t total, x1;
        const bool any = page_begin(cur, total, x1);
        int nk = 0, nv = 0, nq = 0;  // copies of K, V and queries
        for (int seg = 0; !gone(); ++seg) {
          const int n = any ? cur.upto(x1) : 0;
          Segment& sg = writable(seg);
          if (gone()) break;
          if (n <= 0) {
            if (lane == 0) {
              sg.n = 0;
              tc::mbar_arrive(segfull(seg));
            }
            break;
          }
          const int t0 = cur.blk.tile0(cur.k) + cur.tile;
          const int p0 = cur.blk.pos0(cur.k), hi = cur.blk.pos1(cur.k), lo = cur.blk.lo(cur.k);
          if (lane == 0) {
            sg.n = n, sg.t0 = t0, sg.p0 = p0, sg.p1 = hi, sg.lo = lo;
            sg.all_lo = s.window ? (hi - p0 < s.window ? max(hi - s.window + 1, 0) : INT32_MAX) : 0;
            sg.row = cur.row0 + cur.k * w.tb;
            sg.u = (short)cur.u;
            sg.starts = cur.tile == 0;
            sg.whole = cur.whole(n);
            tc::mbar_arrive(segfull(seg));
            if (cur.tile == 0 && n < cur.tiles)  // others go on with the unit
              w.info[blockIdx.x] = make_int4(cur.row0 + cur.k * w.tb, cur.u, (hi - p0 + 1) * s.G,
                                             (int)share_of_tile(cur.last(), total, gridDim.x));
          }
          // lane i: the page that holds group i % 8 of a tile, or -1; a page is copied
          // whole if a row sees any of it
          auto look = [&](int i) {
            const int64_t first = (int64_t)(t0 + i) * kPageTile + ((lane & 7) * 16 & -s.T);
            return i < n && first <= hi && first + s.T > lo ? page_of<true>(s, cur.b, (int)(first / s.T)) : -1;
          };
          int pg = look(0), big = kNoScale;
          float ks = 0.f, vs = 0.f;
          auto scales = [&] {
            ks = vs = 0.f;
            if (pg >= 0) {
              ks = __ldcg(k_scales + (size_t)pg * s.U + cur.u);
              vs = __ldcg(v_scales + (size_t)pg * s.U + cur.u);
            }
          };
          scales();
          for (int i = 0; i < n; ++i, ++it) {
            const int pg_next = look(i + 1);
            const uint32_t loaded = __ballot_sync(0xffffffffu, pg >= 0) & 0xFFu;
            const uint32_t bytes = (uint32_t)__popc(loaded) * 16 * D;
            // a page's first group copies it (a tile holds whole pages)
            const bool first = lane < 8 && (lane * 16) % s.T == 0 && pg >= 0;
            const int src = (pg * s.U + cur.u) * s.T;
            const uint32_t dst = sm0 + C::kOffCodes + lane * 16 * D;
            big = max(big, __reduce_max_sync(0xffffffffu, scale_exponent(vs)));
            const ValueScale v = value_scale(vs, big);
            const bool plain = __all_sync(0xffffffffu, pg < 0 || v.f == 1.f);
            wait(cfree(0), (it & 1) ^ 1);
            if (gone()) break;
            if (lane == 0) {
              TileScales& mt = meta[it & (kRing - 1)];
              mt.loaded = loaded;
              mt.plain = plain;
            }
            if (lane < 8) {
              TileScales& mt = meta[it & (kRing - 1)];
              mt.ks[lane] = key_scale(ks);
              mt.ve[lane] = v.e;
              mt.ive[lane] = v.down;
              mt.vf[lane] = half2_bits(v.f, v.f);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_expect_tx(cfull(0), bytes);
            __syncwarp();
            if (first) tc::tma_load_2d(dst, &kmap, 0, src, cfull(0));
            ++nk;
            if (i == 0) {
              if (seg > 0)
                wait(qfree, (seg - 1) & 1);
              else
                grid_dependency_wait();
              if (gone()) break;
              if (lane == 0) {
                // whole boxes count, what lies behind the last row included
                tc::mbar_expect_tx(qfull, (uint32_t)(2 * tb2 * s.G * D * 2));
                for (int j = 0; j < 2 * (D / 64); ++j)
                  tc::tma_load_3d(sm0 + j * 16384, &qmap, j % (D / 64) * 64, cur.u * s.G,
                                  cur.row0 + cur.k * w.tb + j / (D / 64) * tb2, qfull);
              }
              __syncwarp();
              ++nq;
            }
            wait(cfree(1), (it & 1) ^ 1);
            if (gone()) break;
            if (lane == 0) tc::mbar_expect_tx(cfull(1), bytes);
            __syncwarp();
            if (first) tc::tma_load_2d(dst + C::kCodeBytes, &vmap, 0, src, cfull(1));
            ++nv;
            pg = pg_next;
            scales();
          }
          if (gone()) break;
          if (!cur.next_unit()) {
            Segment& end = writable(seg + 1);
            if (lane == 0 && !dead) {
              end.n = 0;
              tc::mbar_arrive(segfull(seg + 1));
            }
            break;
          }
        }
        if (gone()) {  // the copies in flight land before the block ends
          if (nk) tc::mbar_wait(cfull(0), (nk - 1) & 1, s.flags);
          if (nv) tc::mbar_wait(cfull(1), (nv - 1) & 1, s.flags);
          if (nq) tc::mbar_wait(qfull, (nq - 1) & 1, s.flags);
        }
      }
      __syncwarp();
    } else if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
      // ------------------------------------------------ cache tiles
      // A pass is 32 rows by 64 codes: a warp's lanes hold 16 codes each of 8
      // rows, and eight lanes that access shared memory together those of rows
      // p and p ^ 5: the swizzles then send them to all banks, both for reading
      // (rows that differ in bit 2) and for writing (in bit 0).
      constexpr int kWarpC = 8;  // the first of these warps
      const int ct = tid - kWarpC * 32;
      constexpr int kHalves = D / 64;
      constexpr int kBatch = 4;  // passes whose codes are read together
      const int row = (warp - kWarpC) * 8 + ((lane >> 3) ^ ((lane >> 2 & 1) * 5)), col = lane & 3;
      // this thread's chunk of codes of a pass, and its two chunks of f16
      const uint32_t in0 = C::kOffCodes + row * D + ((col ^ (D == 128 ? row & 7 : row >> 1 & 3)) << 4);
      const uint32_t in1 = in0 ^ 64;  // d = 128: of the second half of the row
      const uint32_t out0 = row * 128 + (((2 * col) ^ (row & 7)) << 4), out1 = out0 ^ 16;
      auto put = [&](uint32_t off, const uint32_t (&x)[8]) {
        *(uint4*)(smem + off + out0) = make_uint4(x[0], x[1], x[2], x[3]);
        *(uint4*)(smem + off + out1) = make_uint4(x[4], x[5], x[6], x[7]);
      };
      // a tile that all rows see whole and whose f are 1
      auto convert = [&](uint32_t in, uint32_t out) {
#pragma unroll 1
        for (int a = 0; a < kHalves; ++a) {
          uint4 c[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            c[k] = *(const uint4*)(smem + in + (k % kHalves ? in1 : in0) + k / kHalves * 32 * D);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            uint32_t x[8];
            widen16(c[k], x);
            put(out + k % kHalves * 16384 + k / kHalves * 4096, x);
          }
          in += kBatch / kHalves * 32 * D;
          out += kBatch / kHalves * 4096;
        }
      };
      // any tile
      auto convert_any = [&](uint32_t in, uint32_t out, bool full, int64_t tile0, int lo, int p1, bool values,
                             const TileScales& mt, uint32_t* nan) {
#pragma unroll 1
        for (int r0 = 0; r0 < kPageTile; r0 += 32) {
          const int rr = r0 + row;
          uint4 c[kHalves];
          bool bad = false;
#pragma unroll
          for (int k = 0; k < kHalves; ++k) {
            c[k] = *(const uint4*)(smem + in + (k ? in1 : in0) + r0 * D);
            bad |= has_nan(c[k].x) || has_nan(c[k].y) || has_nan(c[k].z) || has_nan(c[k].w);
          }
          uint32_t f = mt.vf[rr >> 4];
          if (!full) {
            // Rows differ in what they see.  A NaN would not be hidden by a
            // weight of zero, nor would a factor that is not finite: such a token's
            // values become zeros, and the NaN is handed to the rows that see it by
            // their weights.
            bad |= values && (f & 0x7C00u) == 0x7C00u;
            const int64_t tok = tile0 + rr;
            const bool none = tok < lo || tok > p1 || !((mt.loaded >> (rr >> 4)) & 1u);
            const uint32_t any = __ballot_sync(0xffffffffu, bad && !none) >> (lane & 28) & 15u;  // the row's lanes
            if (none || (values && any)) {
#pragma unroll
              for (int k = 0; k < kHalves; ++k) c[k] = make_uint4(0, 0, 0, 0);
              f = 0x3C003C00u;  // 1
            }
            if (values && any && col == 0) atomicOr(&nan[rr >> 5], 1u << (rr & 31));
          }
#pragma unroll
          for (int k = 0; k < kHalves; ++k) {
            uint32_t x[8];
            widen16(c[k], x);
            if (values) {
#pragma unroll
              for (int a = 0; a < 8; ++a) {
                const __half2 y = __hmul2(*(const __half2*)&x[a], *(const __half2*)&f);
                x[a] = *(const uint32_t*)&y;
              }
            }
            put(out + k * 16384 + r0 * 128, x);
          }
        }
      };
      for (int seg = 0;; ++seg) {
        const Segment& sg = segment(seg);
        const int n = gone() ? 0 : sg.n;
        if (n == 0) break;
        const int p0 = sg.p0, p1 = sg.p1, lo = sg.lo, all_lo = sg.all_lo;
        const int64_t first = (int64_t)sg.t0 * kPageTile;
        read(seg);
        for (int i = 0; i < n; ++i, ++it) {
          const int st = it & 1;
          const int64_t tile0 = first + (int64_t)i * kPageTile;
          const TileScales& mt = meta[it & (kRing - 1)];
          uint32_t(&nan)[4] = sh.nan[it & (2 * kRing - 1)];
          wait(cfull(0), it & 1);
          const bool full = tile0 >= all_lo && tile0 + kPageTile - 1 <= p0 && mt.loaded == 0xFFu;
          const bool plain = mt.plain;
          wait(kfree(st), ((it >> 1) & 1) ^ 1);
          // a later tile's; all have left the slot's last one, and none is there yet
          if (ct < 4) sh.nan[(it + 2) & (2 * kRing - 1)][ct] = 0;
          if (full)
            convert(0, C::kOffK + st * C::kTileBytes);
          else
            convert_any(0, C::kOffK + st * C::kTileBytes, false, tile0, lo, p1, false, mt, nan);
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(cfree(0));
          tc::mbar_arrive(kfull(st));
          wait(cfull(1), it & 1);
          wait(vfree(st), ((it >> 1) & 1) ^ 1);
          if (full && plain)
            convert(C::kCodeBytes, C::kOffV + st * C::kTileBytes);
          else
            convert_any(C::kCodeBytes, C::kOffV + st * C::kTileBytes, full, tile0, lo, p1, true, mt, nan);
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(cfree(1));
          tc::mbar_arrive(vfull(st));
        }
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
      // ------------------------------------------------ softmax
      const int h = warp >> 2, r = tid & 127;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t cs = lanes + h * 128, co = lanes + C::kColO + h * D;
      const int ri = r / s.G, rg = r - ri * s.G;  // token in the half, head in the group
      int cnt = 0;  // tiles of this half so far
      grid_dependency_wait();  // the exponents
      for (int seg = 0;; ++seg) {
        const Segment& sg = segment(seg);
        const int n = gone() ? 0 : sg.n;
        if (n == 0) break;
        const int p0 = sg.p0, p1 = sg.p1;
        const int ti = h * tb2 + ri;  // token in the block
        const bool live = ri < tb2 && p0 + ti <= p1;
        const int pos = live ? p0 + ti : -1;
        const int see_lo = s.window && live ? max(pos - s.window + 1, 0) : 0;
        if (h == 0 || p1 - p0 >= tb2) {
          float m = -INFINITY, l = 0.f;
          // softmax scale * log2(e) * the row's power of two
          float fac = s.scale * 1.4426950408889634f;
          if (live)
            fac *= __uint_as_float((uint32_t)(127 + w.qexp[(int64_t)(sg.row + ti) * s.Hq + sg.u * s.G + rg]) << 23);
          for (int i = 0; i < n; ++i, ++cnt) {
            const TileScales& mt = meta[(it + i) & (kRing - 1)];
            const int64_t tile0 = (int64_t)(sg.t0 + i) * kPageTile;
            wait(sready(h), cnt & 1);
            tc::fence_after_sync();
            // t = S * c + e by group of 16 tokens; where tokens are masked t itself takes
            // S's place
            const uint32_t loaded = mt.loaded;
            const bool masked = !(tile0 >= sg.all_lo && tile0 + kPageTile - 1 <= p0 && loaded == 0xFFu);
            if (masked) wait(vfull((it + i) & 1), ((it + i) >> 1) & 1);  // the NaN bits
            if (masked) {
              const int64_t top = min((int64_t)pos - tile0, (int64_t)kPageTile - 1);  // last token seen
              const int bot = (int)max(min((int64_t)see_lo - tile0, (int64_t)kPageTile), (int64_t)0);
#pragma unroll 1
              for (int c0 = 0; c0 < kPageTile; c0 += 32) {
                float y[32];
                tc::tmem_ld32(cs + c0, y);
                const int hi = (int)max(top - c0, (int64_t)-1), lo = bot - c0;
                uint32_t sees = hi < 0 ? 0u : 0xFFFFFFFFu >> (31 - min(hi, 31));
                if (lo > 0) sees &= lo > 31 ? 0u : 0xFFFFFFFFu << lo;
                const int g = c0 / 16;
                if (!((loaded >> g) & 1u)) sees &= 0xFFFF0000u;
                if (!((loaded >> (g + 1)) & 1u)) sees &= 0x0000FFFFu;
                const uint32_t nan = sh.nan[(it + i) & (2 * kRing - 1)][c0 / 32];
                const float ca = mt.ks[g] * fac, cb = mt.ks[g + 1] * fac, ea = mt.ve[g], eb = mt.ve[g + 1];
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float a = fmaf(y[j], j < 16 ? ca : cb, j < 16 ? ea : eb);
                  y[j] = (sees >> j) & 1u ? a : -INFINITY;
                }
                if (nan) {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if ((nan & sees) >> j & 1u) y[j] = __uint_as_float(0x7FC00000u);
                }
                tc::tmem_st16(cs + c0, *(const uint32_t(*)[16])y);
                tc::tmem_st16(cs + c0 + 16, *(const uint32_t(*)[16])(y + 16));
              }
              tc::tmem_st_wait();
            }
            float t[kPageTile];
#pragma unroll
            for (int c0 = 0; c0 < kPageTile; c0 += 32) tc::tmem_ld32(cs + c0, t + c0);
            tc::tmem_ld_wait();
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float c = masked ? 1.f : mt.ks[k] * fac, d = (masked ? 0.f : mt.ve[k]) - ref;
#pragma unroll
              for (int j = 16 * k; j < 16 * k + 16; j += 2) fma2(t[j], t[j + 1], c, d);
            }
            float lt;
            bool known = i > 0;  // m is worth a try
            for (bool last = false;; last = true) {
              if (known) {
                float total = 0.f;
                lt = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float sum0 = 0.f, sum1 = 0.f;
                  uint32_t pk[8];
#pragma unroll
                  for (int j = 0; j < 16; j += 2) {
                    const float a0 = ex2(t[16 * k + j]), a1 = ex2(t[16 * k + j + 1]);
                    add2(sum0, sum1, a0, a1);
                    pk[j / 2] = half2_bits(a0, a1);
                  }
                  sum0 += sum1;
                  total += sum0;
                  lt = fmaf(sum0, mt.ive[k], lt);
                  tc::tmem_st8(cs + 8 * k, pk);  // the weights take the scores' place
                }
                // (rows that do not exist may hold anything)
                if (last || !__any_sync(0xffffffffu, live && (!(total < kMost) || m == -INFINITY))) break;
              }
              // go by this tile's maximum
              known = true;
              float a[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) a[k] = fmaxf(t[16 * k], t[16 * k + 1]);
#pragma unroll
              for (int j = 2; j < 16; j += 2)
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] = max3(a[k], t[16 * k + j], t[16 * k + j + 1]);
              const float top = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
              const bool none = m == -INFINITY;
              const float by = top > kUp || (none && top > -INFINITY) ? top - kUp : 0.f;
              const float half = none ? 0.f : ex2(-0.5f * by), al = half * half;
              if (!none || top > -INFINITY) m = (none ? 0.f : m) + by;
              l = l * half * half;  // in two steps, as page_factor
#pragma unroll
              for (int j = 0; j < kPageTile; ++j) t[j] -= by;
              if (i > 0) {  // the sums so far (of this piece) follow
                wait(odone(h), (cnt - 1) & 1);
                tc::fence_after_sync();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                  uint32_t v[16];
                  tc::tmem_ld16(co + c0, v);
                  tc::tmem_ld_wait();
#pragma unroll
                  for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * al);
                  tc::tmem_st16(co + c0, v);
                }
              }
            }
            l += lt;
            tc::tmem_st_wait();
            tc::fence_before_sync();
            tc::mbar_arrive(pready(h));
          }

          // ---- the piece's result
          wait(odone(h), (cnt - 1) & 1);
          tc::fence_after_sync();
          const bool whole = sg.whole;
          const int slot = 2 * blockIdx.x + (sg.starts ? 1 : 0);
          const size_t prow = (size_t)slot * w.rows + ti * s.G + rg;
          const int64_t orow = (int64_t)(sg.row + ti) * s.Hq + sg.u * s.G + rg;
          if (live && !whole) w.ml[prow] = make_float2(m, l);
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const bool wide = ((uintptr_t)out & 31u) == 0;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float v[32];
            tc::tmem_ld32(co + c0, v);
            tc::tmem_ld_wait();
            if (live && whole) {
              uint32_t y[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const __nv_bfloat162 hb = __floats2bfloat162_rn(l == 0.f ? 0.f : v[2 * j] * inv,
                                                               l == 0.f ? 0.f : v[2 * j + 1] * inv);
                y[j] = *(const uint32_t*)&hb;
              }
              __nv_bfloat16* dst = out + orow * D + c0;
              if (wide) {
                store32(dst, y);
                store32(dst + 16, y + 8);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ((uint4*)dst)[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
              }
            } else if (live) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) store32(w.acc + prow * D + c0 + k, (const uint32_t*)v + k);
            }
          }
          tc::fence_before_sync();
        }
        it += n;
        read(seg);
      }
    }
  }
  __syncthreads();
  if (warp == 12) tc::tmem_dealloc(tmem, C::kTmem);
  grid_dependency_wait();
}

template <int D>
cudaError_t launch(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                   const void* kp, const void* vp, const float* ks, const float* vs, void* out,
                   cudaStream_t stream) {
  static int done[kMaxDevices];
  auto kern = page_many_kernel<D>;
  // The roles share out the registers that the block is launched with: a build
  // that gave it fewer than they add up to would wait for them for good.
  static const bool enough = [&] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs == kRegisters;
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  cudaError_t e = ensure_smem(kern, Many<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap qm, km, vm;
  const uint64_t rows = (uint64_t)s.n_pages * s.U * s.T;
  if (!make_tmap_f16_heads(&qm, w.qrot, s.n_tokens, s.Hq, D, w.tb / 2, s.G) ||
      !make_tmap_u8_rows(&km, kp, rows, D, s.T) || !make_tmap_u8_rows(&vm, vp, rows, D, s.T))
    return cudaErrorInvalidValue;
  // these two in this order, and nothing between them: page_many_kernel counts on
  // the rotation's wait for all earlier work
  e = launch_k(page_rotate_kernel<D>, dim3((unsigned)((s.n_tokens + kRotateWarps - 1) / kRotateWarps),
                    (unsigned)((s.Hq + kRotateHeads - 1) / kRotateHeads)),
               dim3(kRotateWarps * 32), 0, stream, true, s, w, (const __nv_bfloat16*)q, q_stride);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(kPageGrid), dim3(kThreads), Many<D>::kSmem, stream, true, s, w, qm, km, vm,
                  ks, vs, (__nv_bfloat16*)out);
}

}  // namespace

cudaError_t launch_page_many(const PageStep& s, const PageWork& w, const void* q, int64_t q_stride,
                             const void* k_pages, const void* v_pages, const float* k_scales,
                             const float* v_scales, void* out, cudaStream_t stream) {
  return s.d == 64 ? launch<64>(s, w, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, stream)
                   : launch<128>(s, w, q, q_stride, k_pages, v_pages, k_scales, v_scales, out, stream);
}

}  // namespace salsc
