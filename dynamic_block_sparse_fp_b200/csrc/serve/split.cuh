// split.cuh -- what the two tensor-core attention kernels share: how the work
// is cut into units, waits, tensor maps, and the kernel that joins the units.
#pragma once

#include <math.h>

#include <atomic>

#include "serve_internal.cuh"
#include "visible.cuh"

namespace fps {
namespace {

constexpr int BN = 64;  // keys per tile

struct Split {
  int on;        // units are found on the device (else one unit per item)
  int target;    // units of a kv head that run at a time
  int most;      // and that many items are cut into, beside their ends
  int min_tiles; // key tiles that a unit has at least
  int pairs, tiles;  // n_seqs * tiles, and row tiles per sequence
  int rows;      // rows of a partial result
  int cluster;   // CTAs that share an item (1 where units are found)
  int2 *plan;    // [pairs]: units, first partial
  float *part_o; // [partials][rows][d]
  float2 *part_ml;
};

// mbar_wait whose clock is read only after some thousand tries: a wait that
// memory or another warp answers soon costs its tries and nothing else.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         uint64_t limit_ns = 2000000000ull) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 1023u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) return false;
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
// The unit of a CTA: which item, which of its units.
struct Unit {
  int s, x;      // sequence and row tile
  int k, units;  // unit k of the item's units
  int part;      // where its partial result goes (units > 1)
  Seq seq;
};

__device__ __forceinline__ int pair_seq(const Split &sp, int pair) {
  return sp.tiles == 1 ? pair : pair / sp.tiles;
}

template <int ROWS>
__device__ __forceinline__ int tiles_of(const Problem &P, const Seq &q, int x) {
  const RowTile rt = row_tile<ROWS>(P, q, x);
  return rt.rows > 0 ? key_tiles(P, q, rt).count() : 0;
}
template <int ROWS>
__device__ __forceinline__ int pair_tiles(const Problem &P, const Split &sp, int pair) {
  const int s = pair_seq(sp, pair);
  return tiles_of<ROWS>(P, load_seq(P, s), pair - s * sp.tiles);
}

// The cut: each item's key tiles in units of `size` (each item one at least).
// Few items (twice as many fit): about one unit for each CTA that runs at a
// time, and not more, so that all of them start at once; the size grows until
// they fit.  Many items: `most` units, a few for each CTA that runs at a time, so
// that their uneven ends overlap.  Or nothing is cut, where that should take less
// time (stay_whole).
//
// find_unit finds unit blockIdx.x of the kv head.  Every CTA computes the same cut
// from the lengths.  Up to 32 items: every warp by itself, an item a
// lane.
__device__ __forceinline__ int first_size(const Split &sp, long long all, int units) {
  const unsigned most = unsigned(units);
  // (a 64-bit division takes half a microsecond)
  const long long size = all < (1ll << 31) ? (unsigned(all) + most - 1) / most
                                           : (all + most - 1) / most;
  return int(min(1ll << 30, max(static_cast<long long>(sp.min_tiles), size)));
}
__host__ __device__ __forceinline__ bool few_items(const Split &sp) {
  return 2 * sp.pairs <= sp.target;
}
__device__ __forceinline__ int units_of(int tiles, int size) {
  return max(1u, (unsigned(tiles) + size - 1) / unsigned(size));
}

// Whether all items should stay whole, by when the last would end, in tiles of one
// CTA: an item's own start and end take some 5, a unit's with its partial result 8,
// the joining 10; what does not run all at once ends half a unit or item apart.
// (4 chunks of 256 over 4000 tokens, 256 items of 63 tiles: 118 us in units of 21,
// 70 whole; 176 items of 77 tiles: 141 us in units of 13, 115 whole; one chunk of
// 128 over 4000, 32 items of 63: 33 us in units of 8, 62 whole.)
__device__ __forceinline__ bool stay_whole(const Split &sp, long long all, int longest, int size,
                                           bool few) {
  const float places = float(sp.target), n = float(sp.pairs), sum = float(all);
  const float whole = n <= places ? longest + 5.f
                                  : fmaxf(longest + 5.f, (sum + 5.f * n) / places + 0.5f * longest);
  const float cut = few ? size + 15.f
                        : (sum + 8.f * (n + sum / size)) / places + 0.5f * size + 10.f;
  return whole <= cut;
}

constexpr int SIZES = 8;  // that the search compares

struct FindUnit {  // shared memory of the search
  long long tiles[8];
  int longest[8];
  int scan[2][8];
  uint16_t units[SIZES][8];
  int unit[5];
};

template <int ROWS>
__device__ __forceinline__ bool find_unit_warp(const Problem &P, const Split &sp, Unit *out) {
  const int lane = threadIdx.x % 32;
  const bool item = lane < sp.pairs;
  const int s = pair_seq(sp, lane);
  Seq q = {0, 0, 0, false};
  if (item) q = load_seq(P, s);
  const int tiles = item ? tiles_of<ROWS>(P, q, lane - s * sp.tiles) : 0;
  long long all = tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  const bool few = few_items(sp);
  int size = first_size(sp, all, few ? sp.target : sp.most);
  int units = item ? units_of(tiles, size) : 0;
  while (few && __reduce_add_sync(0xffffffffu, units) > sp.target) {
    size += 1 + size / 8;
    units = item ? units_of(tiles, size) : 0;
  }
  if (stay_whole(sp, all, __reduce_max_sync(0xffffffffu, tiles), size, few)) units = item ? 1 : 0;
  const int parts = units > 1 ? units : 0;
  int u = units, t = parts;  // inclusive scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, u, o), b = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) u += a, t += b;
  }
  // cut items' units come first, whole items (shorter) after them all
  const int cut = __shfl_sync(0xffffffffu, t, 31);
  u = units > 1 ? t : cut + u - t;
  const int mine = blockIdx.x;
  const unsigned owner = __ballot_sync(0xffffffffu, mine >= u - units && mine < u);
  if (owner == 0u) return false;
  const int who = __ffs(owner) - 1;
  if (lane == who && threadIdx.x < 32 && mine == u - units && blockIdx.y == 0)
    sp.plan[who] = make_int2(units, t - parts);
  const int k = mine - __shfl_sync(0xffffffffu, u - units, who);
  out->s = pair_seq(sp, who), out->x = who - out->s * sp.tiles, out->k = k;
  out->seq.q0 = __shfl_sync(0xffffffffu, q.q0, who);
  out->seq.n = __shfl_sync(0xffffffffu, q.n, who);
  out->seq.len = __shfl_sync(0xffffffffu, q.len, who);
  out->seq.ok = __shfl_sync(0xffffffffu, int(q.ok), who) != 0;
  out->units = __shfl_sync(0xffffffffu, units, who);
  out->part = __shfl_sync(0xffffffffu, t - parts, who) + k;
  return true;
}

// More: each thread takes a run of consecutive items; two block scans (a warp's
// by shuffles, the warps' through shared memory).
template <int ROWS, int THREADS>
__device__ __forceinline__ bool find_unit(const Problem &P, const Split &sp, FindUnit &sm,
                                          Unit *out) {
  if (sp.pairs <= 32) return find_unit_warp<ROWS>(P, sp, out);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int WARPS = THREADS / 32;
  static_assert(WARPS <= 8, "FindUnit has room for 8 warps");
  const int per = (sp.pairs + THREADS - 1) / THREADS;
  const int p0 = threadIdx.x * per, p1 = min(sp.pairs, p0 + per);
  // (64 bits: sequences may share pages, so their lengths can add up to more
  // than a cache holds)
  long long all = 0;
  int longest = 0;
  for (int p = p0; p < p1; ++p) {
    const int n = pair_tiles<ROWS>(P, sp, p);
    all += n;
    longest = max(longest, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) sm.tiles[warp] = all, sm.longest[warp] = longest;
  if (threadIdx.x == 0) sm.unit[0] = -1;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) all += sm.tiles[w], longest = max(longest, sm.longest[w]);
  const bool few = few_items(sp);
  int size = first_size(sp, all, few ? sp.target : sp.most);
  if (few) {
    // the least of some sizes that fits; the last does for sure, as each item has
    // less than a unit too many
    const int more = first_size(sp, all, sp.target - sp.pairs) - size;
    auto nth = [&](int c) { return size + int((static_cast<long long>(more) * c) / (SIZES - 1)); };
    int units[SIZES] = {};
    for (int p = p0; p < p1; ++p) {
      const int n = pair_tiles<ROWS>(P, sp, p);
#pragma unroll
      for (int c = 0; c < SIZES; ++c) units[c] += units_of(n, nth(c));
    }
#pragma unroll
    for (int c = 0; c < SIZES; ++c) {
      units[c] = __reduce_add_sync(0xffffffffu, units[c]);
      if (lane == 0) sm.units[c][warp] = uint16_t(units[c]);  // (<= pairs + target)
    }
    __syncthreads();
    int best = SIZES - 1;
#pragma unroll
    for (int c = SIZES - 2; c >= 0; --c) {
      int sum = 0;
      for (int w = 0; w < WARPS; ++w) sum += sm.units[c][w];
      if (sum <= sp.target) best = c;
    }
    size = nth(best);
  }
  if (stay_whole(sp, all, longest, size, few)) size = max(longest, 1);
  int units = 0, parts = 0;
  for (int p = p0; p < p1; ++p) {
    const int n = units_of(pair_tiles<ROWS>(P, sp, p), size);
    units += n;
    parts += n > 1 ? n : 0;
  }
  // exclusive scans over the threads
  int su = units, st = parts;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, su, o), b = __shfl_up_sync(0xffffffffu, st, o);
    if (lane >= o) su += a, st += b;
  }
  if (lane == 31) sm.scan[0][warp] = su, sm.scan[1][warp] = st;
  __syncthreads();
  int u = su - units, t = st - parts, cut = 0;
  for (int w = 0; w < WARPS; ++w) {
    cut += sm.scan[1][w];
    if (w < warp) u += sm.scan[0][w], t += sm.scan[1][w];
  }
  // cut items' units come first, whole items (shorter) after them all
  u = cut + u - t;
  const int mine = blockIdx.x;
  if ((mine >= t && mine < t + parts) || (mine >= u && mine < u + units - parts)) {
    for (int p = p0; p < p1; ++p) {
      const int n = units_of(pair_tiles<ROWS>(P, sp, p), size);
      const int first = n > 1 ? t : u;
      if (mine >= first && mine < first + n) {
        sm.unit[0] = pair_seq(sp, p), sm.unit[1] = p - sm.unit[0] * sp.tiles;
        sm.unit[2] = mine - first, sm.unit[3] = n, sm.unit[4] = t + (mine - first);
        if (mine == first && blockIdx.y == 0) sp.plan[p] = make_int2(n, t);
        break;
      }
      (n > 1 ? t : u) += n;
    }
  }
  __syncthreads();
  out->s = sm.unit[0], out->x = sm.unit[1], out->k = sm.unit[2], out->units = sm.unit[3];
  out->part = sm.unit[4];
  if (out->s < 0) return false;
  out->seq = load_seq(P, out->s);
  return true;
}

// First key tile and number of key tiles of unit k of `units` of an item of n.
__device__ __forceinline__ void unit_tiles(int n, int k, int units, int *first, int *count) {
  const int each = units == 1 ? n : n / units, more = n - each * units;
  *first = k * each + min(k, more);
  *count = each + (k < more ? 1 : 0);
}

// First partial result of a kv head.  An item in n > 1 units has fewer than
// 2 tiles / size of them, and all tiles / size <= most: 2 most suffice.
__device__ __forceinline__ size_t first_part(const Split &sp, int kv) {
  return size_t(kv) * 2 * sp.most;
}

// Row (of the K and V tensor maps) of the first of the keys key .. of one page,
// or 0 where nothing may be read there: those keys are masked and zeroed.
template <bool COPIES>  // P.k and P.v may be copies by place
__device__ __forceinline__ int tile_row(const Problem &P, int s, int kv, int len, int key) {
  if (P.page == 0) return (s * P.hkv + kv) * len + key;
  if (key >= len) return 0;
  const long long row = COPIES ? held_row(P, s, key >> P.shift, kv)
                               : page_row(P, s, key >> P.shift, kv);
  return row < 0 ? 0 : int(row) + (key & (P.page - 1));
}

// Whether some row of a tile may not see all of the keys t0 .. t0 + 63.
__device__ __forceinline__ bool partial_tile(const Problem &P, const Seq &q, const RowTile &rt,
                                             int t0, int missing) {
  const int p_lo = q.len - q.n + rt.t_lo, p_hi = q.len - q.n + rt.t_hi;
  return missing != 0 || p_lo < t0 + BN - 1 ||
         (p_hi - P.window + 1 > t0 && P.sinks < t0 + BN);
}

// Bits of infinities' and NaNs' exponent fields carried into the signs' places.
__device__ __forceinline__ uint32_t odd16(uint32_t x) {
  return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// Adds to the rows' outputs (a lane's: bf16, or its unit's fp32 sums; neither: the
// lane has no row) the infinities and NaNs that were taken out of V, from the keys
// that each row sees.  Only tiles seen in part were cleaned, or (`all`) every tile
// of a unit with missing pages; a key of another tile would add what its product
// added already, an infinity to an infinity of its sign or a NaN to a NaN.  The
// warp finds a tile's keys with such values together; a lane then takes those that
// its row sees, eight columns at a time, until all of them are NaN.  (Each row by
// itself, element for element over all keys of its unit, took 3.1 ms where this
// takes 76 us: a chunk of 200 tokens over 12001, 8 heads over 2, with one infinity;
// with NaNs only 13.8 ms, 96 us; 56 us without.)
template <int HD>
__device__ __forceinline__ void add_odd_values(const Problem &P, const Seq &seq, const RowTile &rt,
                                               int s, int kv, const KeyTiles &kt, int first_tile,
                                               int ntile, int pos, bool all, __nv_bfloat16 *out,
                                               float *part) {
  const int lane = threadIdx.x % 32;
  auto value_row = [&](int key) {
    const long long row = P.page == 0
                              ? (static_cast<long long>(s) * P.hkv + kv) * seq.len + key
                              : held_row(P, s, key >> P.shift, kv) + (key & (P.page - 1));
    return reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.v) + row * HD);
  };
  auto is_odd = [](uint4 w) { return (odd16(w.x) | odd16(w.y) | odd16(w.z) | odd16(w.w)) != 0u; };
#pragma unroll 1
  for (int t = first_tile; t < first_tile + ntile; ++t) {
    const int t0 = kt.key(t);
    if (!all && !partial_tile(P, seq, rt, t0, 0)) continue;
    const uint64_t there =
        below(seq.len - t0) & ~(P.page == 0 ? 0ull : missing_keys(P, s, seq, t0));
    uint64_t keys = 0;  // that hold such values
#pragma unroll 1
    for (int n = 0; n < 64; n += 32) {
      bool odd = false;
      if (there >> (n + lane) & 1) {
        const uint4 *v = value_row(t0 + n + lane);
#pragma unroll 8
        for (int c = 0; c < HD / 8; ++c) odd |= is_odd(v[c]);
      }
      keys |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, odd)) << n;
    }
    if (!out && !part) continue;
    keys &= seen_keys(P, pos, t0);
#pragma unroll 1
    for (int c = 0; keys != 0 && c < HD; c += 8) {
      float x[8];
      bool open = false, changed = false;  // open: something in x is not yet NaN
      if (out) {
        const uint4 w = *reinterpret_cast<const uint4 *>(out + c);
        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = __uint_as_float(i % 2 ? y[i / 2] & 0xffff0000u : y[i / 2] << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = part[c + i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) open |= x[i] == x[i];
#pragma unroll 1
      for (uint64_t left = keys; open && left; left &= left - 1) {
        const uint4 w = value_row(t0 + __ffsll(static_cast<long long>(left)) - 1)[c / 8];
        if (!is_odd(w)) continue;
        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
        open = false, changed = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t v = i % 2 ? y[i / 2] & 0xffff0000u : y[i / 2] << 16;
          if ((v & 0x7f800000u) == 0x7f800000u) x[i] += __uint_as_float(v);
          open |= x[i] == x[i];
        }
      }
      if (!changed) continue;
      if (out) {
        *reinterpret_cast<uint4 *>(out + c) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                       pack_bf16(x[6], x[7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[c + i] = x[i];
      }
    }
  }
}

// Joins the units of an item: with M the largest m, O = sum 2^(m_u - M) O_u and
// l = sum 2^(m_u - M) l_u in a fixed order.  W warps take a row together, unit u
// by warp u % W, and their sums are added in the warps' order.  Launched early
// (programmatic dependent launch): it waits for the partial results.
constexpr int JOIN_WARPS = 8;

template <int HD, int ROWS, int W>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
    join_kernel(const __grid_constant__ Problem P, const __grid_constant__ Split sp,
                __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
  __shared__ float2 ml_w[JOIN_WARPS];
  __shared__ float o_w[JOIN_WARPS][HD];
  const int pair = blockIdx.x, kv = blockIdx.y;
  const int s = pair_seq(sp, pair);
  const Seq seq = load_seq(P, s);
  const RowTile rt = row_tile<ROWS>(P, seq, pair - s * sp.tiles);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int V = HD / 32, ROWS_AT = JOIN_WARPS / W;  // columns of a lane; rows at a time
  const int first = blockIdx.z * ROWS_AT + warp / W, w = warp % W;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 plan = sp.plan[pair];
  if (plan.x <= 1) return;
  const size_t base = first_part(sp, kv) + plan.y;
  // (the same number of rounds for every warp of the block)
  for (int r0 = blockIdx.z * ROWS_AT; r0 < rt.rows; r0 += gridDim.z * ROWS_AT) {
    const int r = first + r0 - blockIdx.z * ROWS_AT;
    const bool row = r < rt.rows;
    float big = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (row) {
      for (int u = lane; u < plan.x; u += 32)
        big = fmaxf(big, sp.part_ml[(base + u) * sp.rows + r].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      if (big == -INFINITY) big = 0.f;  // no key at all: every weight below is 0
#pragma unroll 4
      for (int u = w; u < plan.x; u += W) {
        const size_t at = (base + u) * sp.rows + r;
        const float2 ml = sp.part_ml[at];
        const float f = ex2(ml.x - big);
        l = fmaf(f, ml.y, l);
        const float *o = sp.part_o + at * HD + lane * V;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 x = *reinterpret_cast<const float2 *>(o + i);
          acc[i] = fmaf(f, x.x, acc[i]);
          acc[i + 1] = fmaf(f, x.y, acc[i + 1]);
        }
      }
    }
    if (W > 1) {
      __syncthreads();  // (the last round's sums have been read)
#pragma unroll
      for (int i = 0; i < V; ++i) o_w[warp][lane * V + i] = acc[i];
      if (lane == 0) ml_w[warp] = make_float2(big, l);
      __syncthreads();
      if (w != 0) continue;
#pragma unroll
      for (int x = 1; x < W; ++x) {
        l += ml_w[warp + x].y;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += o_w[warp + x][lane * V + i];
      }
    }
    if (!row) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = size_t(seq.q0) * P.hq + size_t(kv) * P.g * seq.n + rt.first + r;
    uint32_t *dst = reinterpret_cast<uint32_t *>(out + at * HD + lane * V);
#pragma unroll
    for (int i = 0; i < V; i += 2) dst[i / 2] = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
    if (lse && lane == 0)
      lse[at] = l == 0.f ? -INFINITY : (big + log2f(l)) * 0.6931471805599453f;
  }
}

template <int HD, int ROWS, int W>
cudaError_t launch_join(const Problem &P, const Split &sp, __nv_bfloat16 *out, float *lse,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // one round of rows for each CTA, more where that would make very many CTAs
  // (most of them of items that were not cut)
  const int rounds = (sp.rows + JOIN_WARPS / W - 1) / (JOIN_WARPS / W);
  const long long few = 1024 / (static_cast<long long>(sp.pairs) * P.hkv) + 1;
  cfg.gridDim = dim3(sp.pairs, P.hkv, unsigned(rounds < few ? rounds : few));
  cfg.blockDim = dim3(32 * JOIN_WARPS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<HD, ROWS, W>, P, sp, out, lse);
}

// Runs `f` once for each device (kernel attributes; all of it again if two
// threads come first at the same time, which does no harm).
template <class F>
cudaError_t once_per_device(std::atomic<bool> (&done)[64], F f) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  if ((e = f()) == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// 2-D tensor map over [rows x d] with a box of [box_rows x box_d].
inline bool encode_map(CUtensorMap *map, const void *ptr, uint64_t rows, int d, int box_d,
                uint32_t box_rows, bool codes, CUtensorMapSwizzle swizzle) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cuuint64_t(d), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(d) * (codes ? 1 : 2)};
  const cuuint32_t box[2] = {cuuint32_t(box_d), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the host knows of the cut (the lengths are on the device).  Nothing is cut
// where no item can have more than `least` tiles, nor beyond kMaxPairs row tiles, where
// every CTA's search for its unit would cost more than the cut gains: so many items
// fill the machine, unless most of them are short or empty (max_q_len is the longest
// sequence's: one long chunk among single tokens counts as many).  Then a long item is
// walked by one CTA, at some 1500 cycles for each 64 keys of a chunk's kernel.
constexpr int kMaxPairs = 1024, kSms = 148;

// Longest list of key tiles that an item can have.
inline long long most_tiles(const Problem &P) {
  const long long all = (static_cast<long long>(P.max_pages) * P.page + BN - 1) / BN;
  const long long seen = (static_cast<long long>(P.window) + P.max_q_len + BN - 1) / BN + 1 +
                         (static_cast<long long>(P.sinks) + BN - 1) / BN;
  return P.window > 0 && seen < all ? seen : all;
}

template <int ROWS>
Split make_split(const Problem &P, int least, int min_tiles, int at_a_time) {
  Split sp = {};
  sp.cluster = 1;
  sp.tiles = most_row_tiles<ROWS>(P);
  const long long pairs = static_cast<long long>(P.n_seqs) * sp.tiles;
  if (P.page == 0 || pairs > kMaxPairs || most_tiles(P) <= least) return sp;
  sp.on = 1;
  sp.pairs = int(pairs);
  sp.min_tiles = min_tiles;
  sp.target = at_a_time > P.hkv ? at_a_time / P.hkv : 1;
  sp.most = 2 * sp.target;
  const long long rows = static_cast<long long>(P.max_q_len) * P.g;
  sp.rows = rows < ROWS ? int(rows) : ROWS;
  return sp;
}

// A CTA for each unit that there can be.  (Those without one delay the others: 600
// more of them took 9 us of 117, a chunk of 700 tokens over 65536, window 4096.)
inline dim3 grid_of(const Problem &P, const Split &sp) {
  if (!sp.on) return dim3(sp.tiles * sp.cluster, P.hkv, P.n_seqs);
  return dim3(few_items(sp) ? sp.target : sp.pairs + sp.most, P.hkv, 1);
}

inline size_t carve(const Problem &P, Split *sp, void *ws) {
  Carver c{static_cast<char *>(ws), 0};
  const size_t parts = size_t(P.hkv) * 2 * sp->most;
  sp->plan = c.take<int2>(sp->pairs);
  sp->part_o = c.take<float>(parts * sp->rows * P.d);
  sp->part_ml = c.take<float2>(parts * sp->rows);
  return c.off;
}

}  // namespace
}  // namespace fps
