// attn_serve_tc.cu -- bf16 queries against visible keys on the sm_100a tensor
// cores (tcgen05 + TMEM + TMA): fp_window_attn and fp_paged_attn, for long
// prompts and chunks of more than 64 packed rows.
//
// One pass over a row's visible keys with a running maximum m (in base-2
// exponents) and sum l:  p_j = 2^(s_j scale log2(e) - m),  l = sum p_j,
// O = sum p_j v_j,  out = O / l.  The work is cut into items of one tile of at
// most 128 packed query rows of one kv head (visible.cuh) and its list of
// 64-key tiles; an item whose list is long against the machine's share of the
// whole is cut again, into units of consecutive key tiles, whose (m, l, O) a
// second kernel joins in a fixed order.
//
// One CTA handles one unit and two CTAs share an SM, so one's softmax overlaps
// the other's MMAs and loads:
//   warps 0-3  softmax + epilogue: thread r owns row r = TMEM lane r (warps
//              without rows take no part);
//   warp 4     TMA producer: Q's second half once, K and V through rings of 3;
//   warp 5     MMA issuer (one thread): S = Q K^T (128 x 64), O += P V;
//   warps 6-7  clean V of what hidden keys may hold (below).
// TMEM (256 columns): S [0,64) fp32 | P [64,96) bf16 pairs | Q d 0..63 [96,128)
// bf16 pairs | O [128,128+d) fp32.  K and V tiles are 64-d halves of 64 keys x
// 128 B in the 128-byte swizzle; K is the K-major B operand of S, V the MN-major
// B operand of P V.
//
// A hidden key's weight is zero, but 0 x NaN would still spoil the product with
// V.  So in a tile that some row does not see in full, values of keys nobody may
// read (past the sequence, missing pages) are zeroed in shared memory, and so
// are infinities and NaNs of the others, which the epilogue then adds back to
// the rows that do see them.  Two warps of their own do that as V arrives; done
// by the softmax warps it made such a tile take twice as long (3000 against 1500
// cycles, 5 of 19 tiles with a window of 1024).
//
// 8-bit caches come here as bf16 copies of the pages that are read (kv_cache.cu):
// converting tiles as they are loaded, by four more warps, took 390 us where
// 175 us are enough (2048 new tokens, 32 heads over 2, window 4096), since every
// row tile converts its keys again.
//
// Every wait is bounded (2 s); on expiry the kernel records FP_ERR_TIMEOUT,
// raises a CTA-wide abort flag, drains its outstanding loads and frees TMEM
// before returning.
#include <math.h>

#include <algorithm>

#include "split.cuh"

namespace fps {
namespace {

constexpr int BM = 128;  // query rows per tile
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t S_COL = 0, P_COL = BN, Q0_COL = BN + BN / 2, O_COL = 2 * BN;
// Items of up to LEAST key tiles stay whole, units have MIN_TILES at least (one
// chunk of 128 tokens over 1000, 16 tiles: 21 us whole, 25 in two units).
constexpr int LEAST = 20, MIN_TILES = 8;

template <int HD>
struct Cfg {
  static constexpr int NK = 3, NV = 3;
  static constexpr int LAG = 2;                // V(i - LAG) is loaded after K(i)
  static constexpr uint32_t HALF = BN * 128;   // [64 keys x 64 d] bf16
  static constexpr uint32_t TILE = HALF * (HD / 64);
};
constexpr int THREADS = 256, TMA_WARP = 4, MMA_WARP = 5, CLEAN_WARP = 6, CLEANERS = 64;

template <int HD>
struct Smem {
  using C = Cfg<HD>;
  uint8_t q[BM * 128];  // Q, d 64..127 (d 0..63 lives in TMEM; d = 64: on its way there)
  uint8_t k[C::NK][C::TILE];
  uint8_t v[C::NV][C::TILE];
  uint64_t bar[22];
  __device__ uint64_t *bar_q() { return &bar[0]; }     // Q is in shared memory
  __device__ uint64_t *q_tmem() { return &bar[1]; }    // and its first half in TMEM
  __device__ uint64_t *s_full() { return &bar[2]; }
  __device__ uint64_t *s_free() { return &bar[3]; }
  __device__ uint64_t *p_full() { return &bar[4]; }
  __device__ uint64_t *p_empty() { return &bar[5]; }
  __device__ uint64_t *o_full() { return &bar[6]; }
  __device__ uint64_t *k_full() { return &bar[7]; }    // [3]
  __device__ uint64_t *k_empty() { return &bar[10]; }
  __device__ uint64_t *v_full() { return &bar[13]; }
  __device__ uint64_t *v_empty() { return &bar[16]; }
  __device__ uint64_t *v_part() { return &bar[19]; }   // V of a tile seen in part, not yet clean
  uint32_t tmem_base;
  int abort_flag, poison, missing;
  FindUnit find;
  int rows[64];  // the producer's
};

__device__ __forceinline__ bool bit(uint64_t m, int c) {
  return (c < 32 ? uint32_t(m) >> c : uint32_t(m >> 32) >> (c - 32)) & 1u;
}

// bar.sync that tells every thread whether some thread's x was true.
__device__ __forceinline__ bool named_barrier_or(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(x)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// The maximum of one row of S over a 64-key tile (raw scores).
__device__ __forceinline__ float tile_max(const uint32_t (&u)[BN]) {
  float mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
  for (int c = 0; c < BN; c += 2)
    mx[(c / 2) % 8] = max3f(mx[(c / 2) % 8], __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
  return max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// p = 2^(s * sl2 - base) for one row of S, packed to bf16 pairs, and its sum in
// 4 two-lane chains.
__device__ __forceinline__ void tile_exp(const uint32_t (&u)[BN], float sl2, float base,
                                         float2 (&acc)[4], uint32_t (&pk)[BN / 2]) {
  const float2 sc = make_float2(sl2, sl2), nm = make_float2(-base, -base);
#pragma unroll
  for (int i = 0; i < BN; i += 2) {
    const float2 x = ffma2(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), sc, nm);
    float2 p;
    p.x = ex2(x.x);
    p.y = ex2(x.y);
    acc[(i / 2) % 4] = fadd2(acc[(i / 2) % 4], p);
    // bf16 weights: the tensor core's operand type, half a step of 2^-8 each,
    // as much as the output's own rounding; the sum keeps the fp32 weights
    pk[i / 2] = pack_bf16(p.x, p.y);
  }
}

// One S tile of one row: read out of TMEM (then released), hidden keys' scores
// made -infinity (weight 0), exponentials against the running maximum first, and
// again only if some row of the warp needs a new one: its first tile with a
// key, or a weight above 2^8 (which a tile sum of at most 2^8 rules out; until
// then p <= 256 is as exact, and 1/l uses the same m).
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint64_t *s_free, uint64_t seen,
                                             float sl2, float m, float &muse, float &alpha,
                                             uint32_t (&pk)[BN / 2], float &ps) {
  uint32_t u[BN];
  float2 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
  tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&u[0]));
  tmem_ld32(s_addr + 32u, *reinterpret_cast<uint32_t(*)[32]>(&u[32]));
  tc_wait_ld();
  // S is in registers: the next S may overwrite the TMEM buffer
  tc_fence_before();
  mbar_arrive(s_free);
  if (__any_sync(0xffffffffu, seen != ~0ull)) {
#pragma unroll
    for (int c = 0; c < BN; ++c) u[c] = bit(seen, c) ? u[c] : 0xff800000u;
  }
  const bool first = m == -INFINITY;
  if (!first) tile_exp(u, sl2, m, acc, pk);
  muse = m;
  ps = ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
       ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
  const bool need = first || !(ps <= 256.f);  // (a NaN sum too)
  if (__any_sync(0xffffffffu, need)) {
    const float tmax = tile_max(u) * sl2;
    if (need && (tmax > m + 8.0f || first)) muse = fmaxf(m, tmax);
  }
  if (__any_sync(0xffffffffu, first || muse != m)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
    // (no key so far, or only scores of -infinity: their weights are 0)
    tile_exp(u, sl2, muse == -INFINITY ? 0.f : muse, acc, pk);
    ps = ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
         ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
  }
  alpha = muse != m ? ex2(m - muse) : 1.f;  // 0 on the first tile
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 2)
    attn_serve_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ Problem P, const __grid_constant__ Split sp,
                      const __nv_bfloat16 *__restrict__ qg, __nv_bfloat16 *__restrict__ out,
                      float *__restrict__ lse, int *status) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // the 128-B swizzled tiles need 1024-B alignment and there is no slack to
  // realign: refuse (before touching shared memory) if it is missing
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) report(status, FP_ERR_UNSUPPORTED);
    return;
  }
  auto &sm = *reinterpret_cast<Smem<HD> *>(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kv = blockIdx.y;

  // ------------------------------------------------------------- the unit --
  Unit un = {int(blockIdx.z), int(blockIdx.x), 0, 1, 0, {}};
  if (sp.on) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!find_unit<BM, THREADS>(P, sp, sm.find, &un)) return;
  } else {
    un.seq = load_seq(P, un.s);
  }
  const Seq seq = un.seq;
  if (!seq.ok) {
    if (threadIdx.x == 0 && un.x == 0 && kv == 0) report(status, FP_ERR_DEVICE_CHECK);
    return;
  }
  const RowTile rt = row_tile<BM>(P, seq, un.x);
  if (rt.rows <= 0) return;
  const KeyTiles kt = key_tiles(P, seq, rt);
  int first_tile, ntile;
  unit_tiles(kt.count(), un.k, un.units, &first_tile, &ntile);
  const int nact = (rt.rows + 31) / 32;  // softmax warps with rows
  const int box = P.page == 0 ? BN : min(P.page, BN), nbox = BN / box;
  // first packed row of the tile
  const size_t row0 = size_t(seq.q0) * P.hq + size_t(kv) * P.g * seq.n + rt.first;
  volatile int *abort_flag = &sm.abort_flag;
  auto fail = [&](int code) {
    report(status, code);
    *abort_flag = 1;
  };
  // The others wait for the barriers (2) and for each other's scan of the pages
  // (3: who finds one of the unit's pages missing says so, an error where some row
  // would see one of its keys); the producer asks for the outcome (5) when the first
  // loads are on their way.
  auto begin = [&]() -> int {
    int missing = 0;
    const int id = warp < 4 ? threadIdx.x : threadIdx.x - 32;
    if (P.page != 0)
      for (int e = id; e < ntile * nbox; e += THREADS - 32) {
        const int t0 = kt.key(first_tile + e / nbox), c = e % nbox * box, key = t0 + c;
        if (key < seq.len && page_row(P, un.s, key >> P.shift, kv) < 0) {
          missing = 1;
          if (used_keys(P, seq, rt, t0) >> c & below(box)) report(status, FP_ERR_DEVICE_CHECK);
        }
      }
    named_barrier_sync(2, THREADS);
    if (missing) sm.missing = 1;
    tc_fence_before();
    named_barrier_sync(3, THREADS - 32);
    tc_fence_after();
    asm volatile("bar.arrive 5, %0;" ::"n"(THREADS) : "memory");
    return sm.missing;
  };

  // 2 warpgroups of 128 registers a thread, dealt out as 208 + 48 = 2 x 128 (each
  // role's code is compiled for its own share)
  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (warp < nact) {
      // -------------------------------------------------------- softmax --
      const int r = threadIdx.x;  // row in the tile, TMEM lane
      const bool row_exists = r < rt.rows;
      const float sl2 = 1.4426950408889634f / sqrtf(float(HD));  // scale * log2(e)
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      const int missing = begin();
      const uint32_t lane_base = sm.tmem_base + (uint32_t(warp * 32) << 16);
      {
        // the first 64 d of this row's query -> TMEM (A operand of Q K^T);
        // 32-bit column c holds d 2c (low half) and 2c + 1
        if (!__all_sync(0xffffffffu, bar_wait(sm.bar_q(), 0, abort_flag))) ok = false;
        uint32_t qw[32];
        const uint8_t *src = (HD == 128 ? sm.v[2] : sm.q) + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 w = *reinterpret_cast<const uint4 *>(src + ((c ^ (r & 7)) << 4));
          qw[4 * c] = w.x;
          qw[4 * c + 1] = w.y;
          qw[4 * c + 2] = w.z;
          qw[4 * c + 3] = w.w;
        }
        tmem_st32(lane_base + Q0_COL, qw);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(sm.q_tmem());
      }
      const int pos = row_position(seq, rt, r);
      for (int t = 0; ok && t < ntile; ++t) {
        const int t0 = kt.key(first_tile + t);
        uint64_t seen = ~0ull;
        if (partial_tile(P, seq, rt, t0, missing)) {
          seen = seen_keys(P, pos, t0);
          if (missing) seen &= ~missing_keys(P, un.s, seq, t0);
        }
        // waits are made warp-uniform: tcgen05.ld/st below are .sync.aligned
        if (!__all_sync(0xffffffffu, bar_wait(sm.s_full(), t & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float muse, alpha, ps;
        uint32_t pk[BN / 2];
        softmax_tile(lane_base + S_COL, sm.s_free(), seen, sl2, m, muse, alpha, pk, ps);
        l = l * alpha + ps;
        // P(t) overwrites P(t-1), and O may be rescaled: both need P(t-1) V(t-1)
        // finished (for t = 0 the wait is on the phase before the first and
        // returns at once)
        if (!__all_sync(0xffffffffu, bar_wait(sm.p_empty(), (t & 1) ^ 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // O is rescaled (rarely: lazy) by the whole warp if any of its rows'
        // max grew
        if (__any_sync(0xffffffffu, t > 0 && alpha != 1.f)) {
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {
            uint32_t u[32];
            tmem_ld32(lane_base + O_COL + uint32_t(c0), u);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
            tmem_st32(lane_base + O_COL + uint32_t(c0), u);
          }
        }
        tmem_st32(lane_base + P_COL, pk);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(sm.p_full());
        m = muse;
      }
      // ---------------------------------------------------------- epilogue --
      if (ok && ntile > 0 && !__all_sync(0xffffffffu, bar_wait(sm.o_full(), 0, abort_flag)))
        ok = false;
      if (!ok) fail(FP_ERR_TIMEOUT);
      named_barrier_sync(1, 32 * nact + CLEANERS);
      const bool poison = *static_cast<volatile int *>(&sm.poison) != 0;
      tc_fence_after();
      const bool good = ok && ntile > 0;
      const bool whole = un.units == 1;
      const float inv = !good || l == 0.f ? 0.f : 1.f / l;
      const size_t prow0 = whole ? 0 : (first_part(sp, kv) + un.part) * sp.rows;
      // Each warp lays its rows out in the rings (all tiles are used up) and stores
      // them row by row: 32 threads with a row each would touch 32 lines a store.
      uint8_t *stage = sm.k[0] + warp * 32 * HD * (whole ? 2 : 4);
      const int lg = (HD == 128 ? 4 : 3) + (whole ? 0 : 1);  // 2^lg chunks of 16 bytes a row
#pragma unroll
      for (int c0 = 0; c0 < HD; c0 += 32) {
        uint32_t u[32];
        if (good) {
          tmem_ld32(lane_base + O_COL + uint32_t(c0), u);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(u[i + 0]) * inv, __uint_as_float(u[i + 1]) * inv);
            w.y = pack_bf16(__uint_as_float(u[i + 2]) * inv, __uint_as_float(u[i + 3]) * inv);
            w.z = pack_bf16(__uint_as_float(u[i + 4]) * inv, __uint_as_float(u[i + 5]) * inv);
            w.w = pack_bf16(__uint_as_float(u[i + 6]) * inv, __uint_as_float(u[i + 7]) * inv);
            const int c = (c0 + i) / 8;
            *reinterpret_cast<uint4 *>(stage + lane * HD * 2 + ((c ^ (lane & 7)) << 4)) = w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const int c = (c0 + i) / 4;
            *reinterpret_cast<uint4 *>(stage + lane * HD * 4 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
          }
        }
      }
      __syncwarp();
      {
        const int c = lane & ((1 << lg) - 1), rows = rt.rows - 32 * warp;
        uint8_t *dst = (whole ? reinterpret_cast<uint8_t *>(out + row0 * HD)
                              : reinterpret_cast<uint8_t *>(sp.part_o + prow0 * HD)) +
                       (size_t(32 * warp) << (lg + 4)) + c * 16;
#pragma unroll 4
        for (int x = lane >> lg; x < min(32, rows); x += 32 >> lg)
          *reinterpret_cast<uint4 *>(dst + (size_t(x) << (lg + 4))) =
              *reinterpret_cast<const uint4 *>(stage + (x << (lg + 4)) + ((c ^ (x & 7)) << 4));
      }
      __syncwarp();
      if (poison && good)
        add_odd_values<HD>(P, seq, rt, un.s, kv, kt, first_tile, ntile, pos, missing != 0,
                           row_exists && whole ? out + (row0 + r) * HD : nullptr,
                           row_exists && !whole ? sp.part_o + (prow0 + r) * HD : nullptr);
      if (row_exists) {
        if (!whole)
          sp.part_ml[prow0 + r] = make_float2(m, l);
        else if (lse)
          lse[row0 + r] = !good || l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    } else {
      begin();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == TMA_WARP) {
      // ----------------------------------------------------- TMA producer --
      if (lane < 22)
        mbar_init(&sm.bar[lane], lane == 1 || lane == 3 || lane == 4 ? 32 * nact : 1);
      if (lane == 0) {
        sm.abort_flag = 0;
        sm.poison = 0;
        sm.missing = 0;
      }
      mbar_fence_init();
      __syncwarp();
      asm volatile("bar.arrive 2, %0;" ::"n"(THREADS) : "memory");
      // Q once (its first half passes through V's last slot on its way to TMEM), then
      // K(i) and V(i - LAG) in turn, by one thread.
      // It has a few hundred cycles per tile, so the rows that the boxes of the
      // tiles start at come from a ring in shared memory, which the whole warp
      // fills 16 at a time, a batch ahead of the loads.
      const int nb = 31 - __clz(nbox), total = ntile << nb;
      auto fill = [&](int first) {
        const int c = first + lane;
        if (lane < 16 && c < total)
          sm.rows[c % 64] = tile_row<true>(P, un.s, kv, seq.len,
                                     kt.key(first_tile + (c >> nb)) + (c & (nbox - 1)) * box);
      };
      if (lane == 0) {
        mbar_arrive_expect_tx(sm.bar_q(), BM * HD * 2);
        if (HD == 128) {
          tma_load_2d(sm.v[2], &tm_q, sm.bar_q(), 0, int(row0));
          tma_load_2d(sm.q, &tm_q, sm.bar_q(), 64, int(row0));
        } else {
          tma_load_2d(sm.q, &tm_q, sm.bar_q(), 0, int(row0));
        }
      }
      fill(0);
      __syncwarp();
      int issued_k = 0, slot_k = 0, slot_v = 0;
      // slot s of V, 4 bits each: loaded, onto v_part, parity of that load's phase;
      // and the parities of v_part's next phases
      uint32_t last_v = 0, parts = 0;
      uint32_t par_k = 1, par_v = 1;
      // one tile into a slot of K or V
      auto load = [&](const CUtensorMap *map, int t, int &slot, uint32_t &par, int n,
                      uint64_t *full, uint64_t *empty, uint8_t *dst) -> bool {
        if (!bar_wait(&empty[slot], par, abort_flag)) return false;
        mbar_arrive_expect_tx(&full[slot], C::TILE);
        for (int j = 0; j < nbox; ++j) {
          const int row = sm.rows[((t << nb) + j) % 64];
#pragma unroll
          for (int h = 0; h < HD / 64; ++h)
            tma_load_2d(dst + slot * C::TILE + h * C::HALF + j * box * 128, map, &full[slot],
                        64 * h, row);
        }
        if (++slot == n) slot = 0, par ^= 1;
        return true;
      };
      bool began = false;
      int missing = 0;
      for (int i = 0; ntile > 0 && i < ntile + C::LAG; ++i) {
        int go = 1;
        if (i == C::LAG) {  // (V's first tile: is it seen in part?)
          named_barrier_sync(5, THREADS);
          began = true;
          missing = sm.missing;
        }
        if (lane == 0) {
          if (*abort_flag) go = 0;
          if (go && i < ntile) {
            go = load(&tm_k, i, slot_k, par_k, C::NK, sm.k_full(), sm.k_empty(), sm.k[0]);
            issued_k += go;
          }
          if (go && i >= C::LAG) {
            const bool part =
                partial_tile(P, seq, rt, kt.key(first_tile + i - C::LAG), missing);
            const int sl = slot_v;
            // (Q's first half has left the slot)
            if (HD == 128 && i == C::LAG + 2) go = bar_wait(sm.q_tmem(), 0, abort_flag);
            go = go && load(&tm_v, i - C::LAG, slot_v, par_v, C::NV,
                            part ? sm.v_part() : sm.v_full(), sm.v_empty(), sm.v[0]);
            if (go) {
              const uint32_t phase = part ? parts >> sl & 1 : (i - C::LAG) / C::NV & 1;
              last_v = (last_v & ~(15u << 4 * sl)) |
                       (1u | (part ? 2u : 0u) | phase << 2) << 4 * sl;
              if (part) parts ^= 1u << sl;
            }
          }
          if (!go) fail(FP_ERR_TIMEOUT);
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        // the first tile of a batch is under way: fill the batch after the next
        // (of the ring's four, the one before this is still read by V)
        if (i == 0) fill(16);
        if (((i << nb) & 15) == 0) fill((i << nb) + 32);
        __syncwarp();
      }
      __syncwarp();
      if (!began) named_barrier_sync(5, THREADS);
      if (lane == 0 && *abort_flag) {
        // drain: wait (bounded) for the loads still in flight, the last load of
        // each slot
        volatile int never = 0;
        bar_wait(sm.bar_q(), 0, &never, 100000000ull);
        for (int t = max(0, issued_k - C::NK); t < issued_k; ++t)
          bar_wait(&sm.k_full()[t % C::NK], (t / C::NK) & 1, &never, 100000000ull);
        for (int s = 0; s < C::NV; ++s)
          if (last_v >> 4 * s & 1)
            bar_wait(last_v >> 4 * s & 2 ? &sm.v_part()[s] : &sm.v_full()[s], last_v >> (4 * s + 2) & 1,
                     &never, 100000000ull);
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      // ------------------------------------------------------- MMA issuer --
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
      }
      __syncwarp();
      tmem_alloc(&sm.tmem_base, TMEM_COLS);
      tmem_relinquish();
      begin();
      const uint32_t tmem = sm.tmem_base;
      if (lane == 0 && ntile > 0) {
        constexpr uint32_t idesc_s = umma_idesc_bf16(BM, BN, 0);
        constexpr uint32_t idesc_o = umma_idesc_bf16(BM, HD, 1);
        const uint32_t q_addr = smem_u32(sm.q);
        bool ok = bar_wait(sm.bar_q(), 0, abort_flag) && bar_wait(sm.q_tmem(), 0, abort_flag);
        auto issue_pv = [&](int u) -> bool {
          const int sv = u % C::NV;
          if (!bar_wait(sm.p_full(), u & 1, abort_flag)) return false;
          if (!bar_wait(&sm.v_full()[sv], (u / C::NV) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint32_t v_addr = smem_u32(sm.v[sv]);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            // A = P(u) [128 lanes x 64 keys] in TMEM: 16 keys = 8 columns;
            // B = V [64 keys x d]: MN-major, 64-d halves HALF apart, 16 keys =
            // 16 rows of 128 B
            const uint64_t bd = umma_desc_sw128(v_addr + kk * 16 * 128, C::HALF, 1024);
            tc_mma_ts(tmem + O_COL, tmem + P_COL + uint32_t(kk * 8), bd, idesc_o,
                      (u > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&sm.v_empty()[sv]);
          tc_commit(sm.p_empty());
          return true;
        };
        for (int t = 0; ok && t < ntile; ++t) {
          const int s = t % C::NK;
          // S(t) overwrites S(t-1): the softmax must have read it out
          if (!bar_wait(&sm.k_full()[s], (t / C::NK) & 1, abort_flag) ||
              !bar_wait(sm.s_free(), (t & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t k_addr = smem_u32(sm.k[s]);
          // d 0..63: A = Q from TMEM (16 d = 8 columns); d 64..127: A = Q's second
          // half in shared memory (16 d = 32 B inside a 64-d half)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ts(tmem + S_COL, tmem + Q0_COL + uint32_t(kk * 8),
                      umma_desc_sw128(k_addr + kk * 32, 16, 1024), idesc_s, kk > 0 ? 1u : 0u);
          if (HD == 128) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ss(tmem + S_COL, umma_desc_sw128(q_addr + kk * 32, 16, 1024),
                        umma_desc_sw128(k_addr + C::HALF + kk * 32, 16, 1024), idesc_s, 1u);
          }
          tc_commit(sm.s_full());
          tc_commit(&sm.k_empty()[s]);
          if (t >= 1 && !issue_pv(t - 1)) {
            ok = false;
            break;
          }
        }
        if (ok && !issue_pv(ntile - 1)) ok = false;
        if (ok) tc_commit(sm.o_full());
        if (!ok) fail(FP_ERR_TIMEOUT);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------- V of hidden keys --
      const int missing = begin();
      const int id = threadIdx.x - 32 * CLEAN_WARP;
      uint32_t parity = 0;  // bit i: of slot i's next tile seen in part
      for (int t = 0; t < ntile; ++t) {
        const int t0 = kt.key(first_tile + t);
        if (!partial_tile(P, seq, rt, t0, missing)) continue;
        const uint64_t gone =
            (missing ? missing_keys(P, un.s, seq, t0) : 0ull) | ~below(seq.len - t0);
        // (a barrier and a parity for each slot: a slot's next such tile comes only
        // after this one has been used, while v_full's phases pass unseen here)
        const int sv = t % C::NV;
        const bool there = bar_wait(&sm.v_part()[sv], parity >> sv & 1, abort_flag);
        parity ^= 1u << sv;
        if (!there) fail(FP_ERR_TIMEOUT);
        if (named_barrier_or(4, CLEANERS, !there)) break;  // (both warps, or neither)
        uint4 *vt = reinterpret_cast<uint4 *>(sm.v[sv]);
        if (gone)
          for (int e = id; e < int(C::TILE / 16); e += CLEANERS)
            if (gone >> (e / 8 % BN) & 1) vt[e] = make_uint4(0u, 0u, 0u, 0u);
        // an exponent field of all ones carries into the sign's place
        auto sum = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
        auto clean = [&](uint32_t x) { return x & ~((sum(x) >> 15 & 0x00010001u) * 0xffffu); };
#pragma unroll 1
        for (int e0 = id; e0 < int(C::TILE / 16); e0 += 4 * CLEANERS) {
          uint4 w[4];
          uint32_t odd = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = vt[e0 + e * CLEANERS];
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= sum(w[e].x) | sum(w[e].y) | sum(w[e].z) | sum(w[e].w);
          if (odd & 0x80008000u) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              vt[e0 + e * CLEANERS] =
                  make_uint4(clean(w[e].x), clean(w[e].y), clean(w[e].z), clean(w[e].w));
            sm.poison = 1;
          }
        }
        fence_async_smem();
        named_barrier_sync(4, CLEANERS);
        if (id == 0) mbar_arrive(&sm.v_full()[sv]);
      }
      __syncwarp();
      // (what was found is there before the epilogue looks)
      asm volatile("bar.arrive 1, %0;" ::"r"(32 * nact + CLEANERS) : "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(sm.tmem_base, TMEM_COLS);
  }
}

template <int HD>
cudaError_t run(const Problem &P, const Split &sp, const void *q, void *out, float *lse,
                cudaStream_t st) {
  auto *kernel = attn_serve_kernel<HD>;
  // two CTAs (and no third, which TMEM has no room for) share an SM
  constexpr int bytes = int(sizeof(Smem<HD>) > 80 * 1024 ? sizeof(Smem<HD>) : 80 * 1024);
  static_assert(2 * (bytes + 1024) <= 233472, "two CTAs must fit in one SM");
  static std::atomic<bool> set[64];
  cudaError_t e = once_per_device(set, [&] {
    cudaError_t r =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (r != cudaSuccess) return r;
    // the roles' register shares need exactly what the launch hands out
    cudaFuncAttributes a;
    if ((r = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return r;
    return a.numRegs == 128 ? cudaSuccess : cudaErrorInvalidConfiguration;
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  const uint64_t kv_rows = P.page == 0 ? uint64_t(P.n_seqs) * P.hkv * P.max_q_len
                           : P.by_place ? uint64_t(P.n_seqs) * P.max_pages * P.hkv * P.page
                                        : uint64_t(P.n_pages) * P.hkv * P.page;
  const uint32_t box = P.page == 0 || P.page > BN ? BN : P.page;
  const CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_map(&mq, q, uint64_t(P.total_q) * P.hq, HD, 64, BM, false, swizzle) ||
      !encode_map(&mk, P.k, kv_rows, HD, 64, box, false, swizzle) ||
      !encode_map(&mv, P.v, kv_rows, HD, 64, box, false, swizzle))
    return cudaErrorInvalidValue;
  __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(out);
  kernel<<<grid_of(P, sp), THREADS, bytes, st>>>(mq, mk, mv, P, sp,
                                                static_cast<const __nv_bfloat16 *>(q), ob, lse,
                                                serve_status_ptr());
  if ((e = cudaGetLastError()) != cudaSuccess || !sp.on) return e;
  return launch_join<HD, BM, 1>(P, sp, ob, lse, st);
}

// Fewer than twice as many items as run at a time are cut finer, into 3.5 units for
// each place (3 chunks of up to 512 tokens over up to 32768, 48 items for 37 places:
// 500 us, with 2 units a place 590); more items end as unevenly without that, and a
// CTA with nothing to do costs some time too (7 over 16000, 112 items: 490 us, 466
// with 2; 2 of 2000 tokens over 9000, 126: 392, 372).  Nor does it pay to have units
// of less than 32 tiles.
Split tc_split(const Problem &P) {
  Split sp = make_split<BM>(P, LEAST, MIN_TILES, 2 * kSms);
  if (sp.pairs < 2 * sp.target) {
    const long long most = std::min(most_tiles(P), 1ll << 30) * sp.pairs / 32;
    sp.most = int(std::min(std::max<long long>(most, sp.target), 7ll * sp.target / 2));
  }
  return sp;
}

// The copies of an 8-bit cache's pages: by their place in the table, or by their
// number where the cache has fewer pages than the table has places.
long long copied_pages(const Problem &P) {
  return std::min<long long>(P.n_pages, static_cast<long long>(P.n_seqs) * P.max_pages);
}

// Workspace: the units' partial results, and the copies.
size_t carve_serve(const Problem &P, bool narrow, Split *sp, void **k, void **v, void *ws) {
  Carver c{static_cast<char *>(ws), sp->on ? carve(P, sp, ws) : 0};
  const size_t cache = narrow ? size_t(copied_pages(P)) * P.hkv * P.page * P.d : 0;
  *k = c.take<__nv_bfloat16>(cache);
  *v = c.take<__nv_bfloat16>(cache);
  return c.off;
}

}  // namespace

size_t attn_serve_ws_bytes(const Problem &P, bool narrow) {
  Split sp = tc_split(P);
  void *k, *v;
  return carve_serve(P, narrow, &sp, &k, &v, nullptr);
}

cudaError_t launch_attn_serve(const Problem &P, bool narrow, const void *q, void *out, float *lse,
                              void *ws, cudaStream_t st) {
  Split sp = tc_split(P);
  Problem W = P;
  void *k, *v;
  carve_serve(P, narrow, &sp, &k, &v, ws);
  if (narrow) {
    W.by_place = copied_pages(P) < P.n_pages;
    const cudaError_t e = launch_kv_widen(P, W.by_place, k, v, st);
    if (e != cudaSuccess) return e;
    W.k = k;
    W.v = v;
    W.k_exps = W.v_exps = nullptr;
  }
  return P.d == 64 ? run<64>(W, sp, q, out, lse, st) : run<128>(W, sp, q, out, lse, st);
}

}  // namespace fps
