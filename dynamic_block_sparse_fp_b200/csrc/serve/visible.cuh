// visible.cuh -- which rows a CTA takes, and which keys they see.
//
// The query heads of one kv head are g consecutive packed [n, d] matrices, g n
// consecutive rows.  They are cut into tiles of ROWS consecutive rows of all those
// (so a single token's g heads share one tile and one pass over the keys), or of
// ROWS consecutive tokens of one head: a tile across two heads holds the last
// tokens of one and the first of the next, and sees the keys of both, but the last
// tile of each head may be nearly empty.  The cut with less work is taken, by the
// key positions that its tiles pass over.
#pragma once

#include "serve_internal.cuh"

namespace fps {

// Whether a sequence's tiles run across heads.
template <int ROWS>
__device__ __forceinline__ bool across_heads(const Problem &P, const Seq &q) {
  if (q.n < ROWS) return true;
  const int per = (q.n + ROWS - 1) / ROWS;
  const int less = P.g * per - int((static_cast<long long>(q.n) * P.g + ROWS - 1) / ROWS);
  if (less == 0) return false;
  // what a tile passes over (on average), and how much more the g - 1 tiles across
  // two heads do
  const long long one = P.window >= q.len ? q.len - q.n / 2 : min(q.len, P.window + ROWS);
  const long long two = min(static_cast<long long>(q.len), static_cast<long long>(P.window) + q.n);
  return less * one > (P.g - 1) * (two - one);
}

// Tiles of any one (sequence, kv head) at most: a sequence of n < ROWS tokens has
// (n g + ROWS - 1) / ROWS, which is g or less, a longer one g ceil(n / ROWS) or less.
template <int ROWS>
__host__ __device__ __forceinline__ int most_row_tiles(const Problem &P) {
  const int n = P.max_q_len;
  return n < ROWS ? (n * P.g + ROWS - 1) / ROWS : P.g * ((n + ROWS - 1) / ROWS);
}

struct RowTile {
  int first, rows;   // packed rows of the kv head's group: [first, first + rows)
  int t_lo, t_hi;    // its tokens lie in [t_lo, t_hi]
};

// Tile x of a sequence (rows = 0: it has no such tile).  Long sequences' tiles
// run from the last tokens (the most keys) to the first, the heads of a token
// range next to each other (they read the same keys).
template <int ROWS>
__device__ __forceinline__ RowTile row_tile(const Problem &P, const Seq &q, int x) {
  RowTile r = {0, 0, 0, 0};
  if (across_heads<ROWS>(P, q)) {
    const int total = q.n * P.g;
    r.first = x * ROWS;
    r.rows = min(ROWS, total - r.first);
    if (r.rows <= 0) return r;
    r.t_lo = r.first % q.n;
    r.t_hi = r.t_lo + r.rows - 1;
    if (r.t_hi >= q.n) r.t_lo = 0, r.t_hi = q.n - 1;  // (of two heads or more)
  } else {
    const int per = (q.n + ROWS - 1) / ROWS, j = per - 1 - x / P.g, h = x % P.g;
    if (j < 0) return r;
    r.t_lo = j * ROWS;
    r.rows = min(ROWS, q.n - r.t_lo);
    r.t_hi = r.t_lo + r.rows - 1;
    r.first = h * q.n + r.t_lo;
  }
  return r;
}

// Position of tile row r (a row past the tile's end: of its last row).
__device__ __forceinline__ int row_position(const Seq &q, const RowTile &rt, int r) {
  return q.len - q.n + (rt.first + min(r, rt.rows - 1)) % q.n;
}

// The 64-key tiles that some row of a tile sees: those of the sinks before the
// window's first, then the window's.
struct KeyTiles {
  int sinks, first, window;  // tiles: [0, sinks) and [first, first + window)
  __device__ __forceinline__ int count() const { return sinks + window; }
  __device__ __forceinline__ int key(int t) const {
    return 64 * (t < sinks ? t : first + t - sinks);
  }
};

__device__ __forceinline__ KeyTiles key_tiles(const Problem &P, const Seq &q, const RowTile &rt) {
  KeyTiles k = {0, 0, 0};
  const int p_lo = max(0, q.len - q.n + rt.t_lo), p_hi = q.len - q.n + rt.t_hi;
  if (p_hi < 0) return k;
  k.first = max(0, p_lo - P.window + 1) / 64;
  k.window = p_hi / 64 - k.first + 1;
  k.sinks = min((P.sinks + 63) / 64, k.first);
  return k;
}

// Bit c: the query at position pos sees key t0 + c.
__device__ __forceinline__ uint64_t below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ uint64_t seen_keys(const Problem &P, int pos, int t0) {
  const int low = pos - P.window + 1;  // the window's first key
  return below(pos + 1 - t0) & (~below(low - t0) | below(P.sinks - t0));
}

// Bit c: some row of a tile sees key t0 + c (their windows' union: the positions are
// consecutive).
__device__ __forceinline__ uint64_t used_keys(const Problem &P, const Seq &q, const RowTile &rt,
                                              int t0) {
  const int p_lo = max(0, q.len - q.n + rt.t_lo), p_hi = q.len - q.n + rt.t_hi;
  return below(p_hi + 1 - t0) & (~below(p_lo - P.window + 1 - t0) | below(P.sinks - t0));
}

// Bit c: key t0 + c lies in a page that does not exist.
__device__ __forceinline__ uint64_t missing_keys(const Problem &P, int s, const Seq &q, int t0) {
  uint64_t m = 0;
  for (int c = 0; c < 64 && t0 + c < q.len; c += 16)
    if (page_row(P, s, (t0 + c) >> P.shift, 0) < 0) m |= 0xffffull << c;
  return m;
}

}  // namespace fps
