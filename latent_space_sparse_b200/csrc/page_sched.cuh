// page_sched.cuh -- the paged attention's work list: which tiles of keys each
// block of query rows needs, and where the i-th tile of the step lies.
//
// A unit is (sequence, row block, KV head): a row block is `tb` consecutive
// new tokens with all the query heads of the KV head, and its tiles are the
// 128-token tiles that any of its rows sees (one tile at least, so that rows
// that see nothing have somebody to write their zeros).  Tiles are numbered
// in the order sequence, row block, KV head, tile; CTAs take contiguous
// ranges of equal length, so no sizes need to be known on the host.  A unit's
// tiles come after `over` places that stand for what a unit costs besides its
// tiles (queries, start and end of the pipeline, results).  All of
// it is integer arithmetic on a sequence's length and number of new tokens.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SALSC_HD __host__ __device__ __forceinline__
#else
#define SALSC_HD inline
#endif

namespace salsc {

constexpr int kPageTile = 128;  // tokens of a key tile

// x / m for 0 <= x, 0 < m < 2^32: a 32-bit division where x fits (a 64-bit one
// takes about four times as long on the GPU).
SALSC_HD int64_t div_small(int64_t x, int64_t m) {
  return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)m) : x / m;
}

// sum over i < n of floor((a*i + b) / m), for n, a, b >= 0, 0 < m < 2^32, by
// the Euclidean reduction of (a, m).
SALSC_HD int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t s = 0;
  while (n > 0) {
    const int64_t qa = div_small(a, m), qb = div_small(b, m);
    s += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const int64_t y = a * n + b;
    if (y < m) break;
    n = div_small(y, m);
    b = y - n * m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// One sequence's row blocks: n tokens in the cache, the last m of them new (m
// may exceed n), blocks of tb new tokens, window w (0: none), `over` places
// before a unit's tiles.
struct PageBlocks {
  int n, m, tb, w, over;

  SALSC_HD int count() const { return m / tb + (m % tb != 0); }
  // positions of the first and last row of block k (negative: no position)
  SALSC_HD int pos0(int k) const { return n - m + k * tb; }
  SALSC_HD int pos1(int k) const {
    const int left = m - k * tb;
    return n - m + k * tb + (tb < left ? tb : left) - 1;
  }
  // first token that block k sees, and its first tile
  SALSC_HD int lo(int k) const {
    const int64_t x = (int64_t)pos0(k) - w + 1;
    return w && x > 0 ? (int)x : 0;
  }
  SALSC_HD int tile0(int k) const { return lo(k) / kPageTile; }
  SALSC_HD int tiles(int k) const {
    const int p = pos1(k);
    return (p > 0 ? p / kPageTile : 0) - tile0(k) + 1;
  }
  // sum over blocks i < k of max(c + i*tb, 0) / 128
  SALSC_HD int64_t ramp(int64_t c, int64_t k) const {
    int64_t r0 = 0;
    if (c < 0) r0 = div_small(-c + tb - 1, tb);
    return r0 < k ? floor_sum(k - r0, kPageTile, tb, c + r0 * tb) : 0;
  }
  // places of blocks 0 .. k-1
  SALSC_HD int64_t before(int k) const {
    const int nb = count();
    if (k <= 0) return 0;
    if (nb == 1) return over + tiles(0);
    const int full = k < nb ? k : nb - 1;
    int64_t s = ramp((int64_t)n - m + tb - 1, full) + (int64_t)k * (over + 1);
    if (k == nb) s += (n > 1 ? n - 1 : 0) / kPageTile;
    if (w) s -= ramp((int64_t)n - m - w + 1, k);
    return s;
  }
};

}  // namespace salsc
