// attn_few.cu -- bf16 attention of few query rows (at most 64 for each sequence
// and kv head: single tokens, or a handful) over a paged cache.
//
// With so few rows every key and value is used once and read once: DRAM is the
// bound, and the work is to keep it busy.  The tcgen05 kernel (attn_serve_tc.cu)
// pads the rows to 128 and takes a chain of TMEM round trips for each 64 keys;
// here four independent warps hold their rows' queries and outputs in registers
// and run 16-row warp MMAs (mma.sync m16n8k16) straight on the tiles that TMA
// puts into a shared-memory ring.  They meet only at the end, where their
// (m, l, O) are joined.
//
// One CTA handles one unit (split.cuh): consecutive 64-key tiles of one item.
// Two CTAs share an SM (8-bit caches: three; of 8 rows, four).  Of a tile, warp w takes row group
// w % R (of 16) and the keys [16 R (w / R), + 16 R), in chunks of 16.  The warps
// refill the ring in turn.  (A fifth warp for that would leave one SM quarter with
// two warps of every CTA, whose registers fit three times in some SMs only: of 384
// units for 444 places 36 waited for another's end.  Warp 0 alone would be the
// slowest of the four: 142 us in place of 127 for 64 ragged sequences, 120 now.)
//   S^T [16 keys x 8 rows] += K [16 x 16 d] Q^T: A = K, B = Q in registers;
//   O^T [16 d x 8 rows] += V^T [16 d x 16 keys] P^T: A = V, B = P, which is S^T's
//   accumulator with its 8 x 8 quarters transposed (movmatrix).
// bf16: A by ldmatrix (V transposed).  e4m3: a pair of codes becomes a pair of
// fp16 numbers by one conversion, exact (e4m3's values lie within fp16's); Q is
// brought to fp16 by a power of two for each row, K's exponents go into the
// scores' fp32 factor and V's into the weights' exponents, so no instruction is
// spent on a code but its half of a conversion (shifts and masks to bf16, and
// products with the scales, took 205 us where this takes 120: 64 ragged
// sequences of up to 8192 tokens, 32 heads over 8).
#include <math.h>

#include <algorithm>

#include "split.cuh"

namespace fps {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;

template <int HD, bool NARROW, int RG>
struct Ring {
  static constexpr int ROW = HD * (NARROW ? 1 : 2);  // bytes of a vector
  static constexpr int TILE = BN * ROW;              // of 64
  // some 190 KB in flight or in use for each SM
  static constexpr int CTAS = !NARROW ? 2 : RG > 0 ? 3 : 4, KB = 192 / CTAS;
  static constexpr int SLOTS = KB * 1024 / (2 * TILE) < 8 ? KB * 1024 / (2 * TILE) : 8;
};

template <int HD, bool NARROW, int RG>
struct FewSmem {
  using G = Ring<HD, NARROW, RG>;
  union {
    uint8_t ring[G::SLOTS][2][G::TILE];  // K and V tiles
    struct {                             // at the end:
      float o[WARPS][RG == 0 ? 8 : 16][HD + 4];       // the warps' results
      float all_o[RG == 0 ? 8 : 16 * RG][HD + 4];     // and the CTA's
      float2 all_ml[RG == 0 ? 8 : 16 * RG];
    };
  };
  uint8_t exps[G::SLOTS][2][BN];
  float2 ml[WARPS][16];
  uint64_t full[G::SLOTS], empty[G::SLOTS];
  FindUnit find;
  int abort_flag;
  int poison;  // bit 0: V held an infinity or a NaN; bit 1: and pages are missing
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of CTA `rank`'s copy of this CTA's shared memory at `addr`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ int ld_cluster(uint32_t a) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
               : "=f"(x.x), "=f"(x.y)
               : "r"(a)
               : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(a)
               : "memory");
  return x;
}

// c += a b: bf16, or fp16 operands
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Two codes as fp16 numbers; two fp32 numbers rounded to fp16.
__device__ __forceinline__ uint32_t codes16(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float power(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// RG: row groups of 16 (0: one of 8)
template <int HD, bool NARROW, int RG>
__global__ void __launch_bounds__(THREADS, Ring<HD, NARROW, RG>::CTAS)
    attn_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Problem P,
                    const __grid_constant__ Split sp, const __nv_bfloat16 *__restrict__ qg,
                    __nv_bfloat16 *__restrict__ out, float *__restrict__ lse, int *status) {
  using G = Ring<HD, NARROW, RG>;
  constexpr int R = RG == 0 ? 1 : RG, NB = RG == 0 ? 1 : 2;  // NB: groups of 8 rows of a warp
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // the swizzled tiles need 1024-B alignment: refuse if it is missing
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) report(status, FP_ERR_UNSUPPORTED);
    return;
  }
  auto &sm = *reinterpret_cast<FewSmem<HD, NARROW, RG> *>(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kv = blockIdx.y;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // ------------------------------------------------------------- the unit --
  const int crank = blockIdx.x % sp.cluster;  // of the CTAs that share an item
  Unit un = {int(blockIdx.z), int(blockIdx.x) / sp.cluster, 0, 1, 0, {}};
  if (sp.on) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!find_unit<64, THREADS>(P, sp, sm.find, &un)) return;
  } else {
    un.seq = load_seq(P, un.s);
  }
  const Seq seq = un.seq;
  if (!seq.ok) {
    if (threadIdx.x == 0 && un.x == 0 && kv == 0 && crank == 0) report(status, FP_ERR_DEVICE_CHECK);
    return;
  }
  const RowTile rt = row_tile<64>(P, seq, un.x);
  if (rt.rows <= 0) return;
  const KeyTiles kt = key_tiles(P, seq, rt);
  const int n_all = kt.count();
  int unit_first, unit_count, first_tile, ntile;
  unit_tiles(n_all, un.k, un.units, &unit_first, &unit_count);
  unit_tiles(unit_count, crank, sp.cluster, &first_tile, &ntile);
  first_tile += unit_first;
  const int box = min(P.page, BN), nbox = BN / box;
  const size_t row0 = size_t(seq.q0) * P.hq + size_t(kv) * P.g * seq.n + rt.first;

  volatile int *abort_flag = &sm.abort_flag;
  auto fail = [&](int code) {
    report(status, code);
    *abort_flag = 1;
  };

  // ------------------------------------------------------------ the ring --
  // A lane copies one box (consecutive keys of one page, 64 at most) of K and V;
  // the slot's barrier expects all boxes.
  const int nb = 31 - __clz(nbox);
  auto box_row = [&](int t, int j) {
    return tile_row<false>(P, un.s, kv, seq.len, kt.key(first_tile + t) + j * box);
  };
  auto expect = [&](int slot) {
    mbar_arrive_expect_tx(&sm.full[slot], 2 * G::TILE + (NARROW ? 2 * BN : 0));
  };
  auto copy_box = [&](int slot, int j, int row) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const CUtensorMap *map = w ? &tm_v : &tm_k;
      if constexpr (NARROW) {
        tma_load_2d(sm.ring[slot][w] + j * box * HD, map, &sm.full[slot], 0, row);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1], %2, [%3];" ::"r"(smem_u32(sm.exps[slot][w] + j * box)),
            "l"((w ? P.v_exps : P.k_exps) + row), "r"(box), "r"(smem_u32(&sm.full[slot]))
            : "memory");
      } else {
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
          tma_load_2d(sm.ring[slot][w] + h * (BN * 128) + j * box * 128, map, &sm.full[slot],
                      64 * h, row);
      }
    }
  };
  const int begun = min(ntile, G::SLOTS);
  if (warp == 0) {
    // the first tiles, as soon as there are barriers (8 tiles of 4 boxes at most)
    const int row = lane < begun << nb ? box_row(lane >> nb, lane & (nbox - 1)) : 0;
    if (lane == 0) {
      for (int i = 0; i < G::SLOTS; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], WARPS);
      }
      sm.abort_flag = 0;
      sm.poison = 0;
      mbar_fence_init();
      for (int i = 0; i < begun; ++i) expect(i);
    }
    __syncwarp();
    if (lane < begun << nb) copy_box(lane >> nb, lane & (nbox - 1), row);
    __syncwarp();
  }
  // At tile t > 0 warp t % 4 refills the slot of tile t - 1 with tile t - 1 + SLOTS;
  // the rows of its next turn are looked up at the last.
  int turn = warp == 0 ? WARPS : warp;
  auto look_up = [&]() {
    const int t = turn - 1 + G::SLOTS;
    return lane < nbox && t < ntile ? box_row(t, lane) : 0;
  };
  int next_row = look_up();

  const int rg = warp % R, ks = warp / R;     // row group, key subset
  const int i8 = lane / 4, j4 = lane % 4;     // accumulator row, column pair
  // Which key of 8 stands at row i8 of S^T (and so at column i8 of V^T).  In 8
  // bits with d = 128 a quarter warp's 16-byte loads take two keys; 0 and 4 (1
  // and 5, ..) lie in different banks, neighbours do not.
  constexpr bool MIXED = NARROW && HD == 128;
  auto key_of = [](int i) { return MIXED ? (i >> 1) + (i & 1) * 4 : i; };
  const float scale2 = 1.4426950408889634f / sqrtf(float(HD));  // scale * log2(e)
  uint32_t qf[NB][HD / 16][2];
  // Factor of the scores of the lane's rows 8 b + 2 j4 + e.  8 bits: times 2^-14, so
  // that a sum (at most 2^31) times it is finite for every query.  (The product of the
  // row's power and the key's may not be: 0 x infinity for a sum of 0.)
  float factor[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = rg * 16 + 8 * b + i8;
    const bool in = r < rt.rows;
    const __nv_bfloat16 *src = qg + (row0 + r) * HD;
    factor[b][0] = factor[b][1] = scale2;
    if constexpr (!NARROW) {
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[b][k][e] =
              in ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 8 * e + 2 * j4)) : 0u;
    } else {
      uint2 w[HD / 16];
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        // step 4 h + w takes the d = 64 h + 16 j4 + 4 w + {0, 1 | 2, 3}
        const int d = 64 * (k / 4) + 16 * j4 + 4 * (k % 4);
        w[k] = in ? __ldg(reinterpret_cast<const uint2 *>(src + d)) : make_uint2(0u, 0u);
        big = max(max(max(big, w[k].x & 0x7fffu), (w[k].x >> 16) & 0x7fffu),
                  max(w[k].y & 0x7fffu, (w[k].y >> 16) & 0x7fffu));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
      // q 2^(14 - x) with 2^x the row's largest: bf16's 8 bits fit fp16's 11, and
      // what falls below fp16's smallest is below 2^-38 of the largest (of queries
      // below 2^-95, for which 2^(x - 28) scale2 would leave the normal range: 2^-133)
      const int x = max(int(big >> 7) - 127, -95);
      const float up = power(14 - x);
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        qf[b][k][0] = pack_f16(__uint_as_float(w[k].x << 16) * up,
                               __uint_as_float(w[k].x & 0xffff0000u) * up);
        qf[b][k][1] = pack_f16(__uint_as_float(w[k].y << 16) * up,
                               __uint_as_float(w[k].y & 0xffff0000u) * up);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        factor[b][e] = scale2 * power(__shfl_sync(0xffffffffu, x, 4 * (2 * j4 + e)) - 28);
    }
  }
  // pages of this unit that do not exist (their keys are hidden; that is an error
  // where some row would see one)
  int missing = 0;
  for (int e = threadIdx.x; e < ntile * nbox; e += THREADS) {
    const int t0 = kt.key(first_tile + e / nbox), c = e % nbox * box, key = t0 + c;
    if (key < seq.len && page_row(P, un.s, key >> P.shift, kv) < 0) {
      missing = 1;
      if (used_keys(P, seq, rt, t0) >> c & below(box)) report(status, FP_ERR_DEVICE_CHECK);
    }
  }
  missing = __syncthreads_or(missing);
  int pos[NB][2];
  float o[NB][HD / 16][4], m[NB][2], l[NB][2];
  // 8 bits: weights times their values' scales are 2^(t - mt), t a score plus the
  // value's exponent, with a running maximum mt of their own
  float mt[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[b][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      pos[b][e] = row_position(seq, rt, rg * 16 + 8 * b + 2 * j4 + e);
      m[b][e] = mt[b][e] = -INFINITY;
      l[b][e] = 0.f;
    }
  }
  bool bad = false, ok = true;
  int slot = 0;
  uint32_t par = 0;
  // ldmatrix: this lane's row of the matrices (of 8 keys) and its chunk's place
  const int lrow = lane % 8, lm = lane / 8;

  for (int t = 0; t < ntile; ++t) {
    const int t0 = kt.key(first_tile + t);
    const bool part = partial_tile(P, seq, rt, t0, missing);
    uint64_t seen[NB][2], gone = 0;
    if (part) {
      if (missing) gone = missing_keys(P, un.s, seq, t0);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) seen[b][e] = seen_keys(P, pos[b][e], t0) & ~gone;
      gone |= ~used_keys(P, seq, rt, t0);
    }
    if (!__all_sync(0xffffffffu, bar_wait(&sm.full[slot], par, abort_flag))) {
      ok = false;
      break;
    }
    if (t == turn) {
      if (t - 1 + G::SLOTS < ntile) {
        // the slot of the tile before this is free when all warps are done with it
        const int last = slot == 0 ? G::SLOTS - 1 : slot - 1;
        if (!__all_sync(0xffffffffu,
                        bar_wait(&sm.empty[last], (t - 1) / G::SLOTS & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) expect(last);
        __syncwarp();
        if (lane < nbox) copy_box(last, lane, next_row);
      }
      turn += WARPS;
      next_row = look_up();
    }
    const uint32_t kbase = smem_u32(sm.ring[slot][0]), vbase = smem_u32(sm.ring[slot][1]);
#pragma unroll 1
    for (int c = 0; c < R; ++c) {
      const int kb = (ks * R + c) * 16;  // first key of the chunk
      // ---------------------------------------------------------- S^T --
      // (two sums, of the even and the odd steps: shorter chains)
      float s[NB][2][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][0][e] = s[b][1][e] = 0.f;
      const int key0 = kb + key_of(i8);  // the lane's keys: key0 and key0 + 8
      if constexpr (NARROW) {
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) {
          uint32_t w[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int key = key0 + 8 * n;
            const int ch = HD == 128 ? (j4 + 4 * h) ^ (key & 7) : j4 ^ ((key >> 1) & 3);
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[n][0]), "=r"(w[n][1]), "=r"(w[n][2]), "=r"(w[n][3])
                         : "r"(kbase + key * HD + ch * 16)
                         : "memory");
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a[4] = {codes16(uint16_t(w[0][i])), codes16(uint16_t(w[1][i])),
                                   codes16(uint16_t(w[0][i] >> 16)),
                                   codes16(uint16_t(w[1][i] >> 16))};
#pragma unroll
            for (int b = 0; b < NB; ++b)
              mma16816<true>(s[b][i % 2], a, qf[b][4 * h + i][0], qf[b][4 * h + i][1]);
          }
        }
      } else {
        const uint32_t row = kbase + (kb + 8 * (lm & 1) + lrow) * 128;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          uint32_t a[4];
          ldmatrix4<false>(a, row + (k / 4) * (BN * 128) + ((2 * (k % 4) + (lm >> 1)) ^ lrow) * 16);
#pragma unroll
          for (int b = 0; b < NB; ++b) mma16816<false>(s[b][k % 2], a, qf[b][k][0], qf[b][k][1]);
        }
      }
      // ------------------------------------------------- scores, masks --
      float y[NB][4], ev[2];  // of keys n = 0, 1 and rows e = 0, 1: y[2 n + e]
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float kf = 1.f;
        if constexpr (NARROW) {
          const uint32_t bk = sm.exps[slot][0][key0 + 8 * n], bv = sm.exps[slot][1][key0 + 8 * n];
          kf = __uint_as_float(bk == 255u ? 0x7fc00000u : bk << 23);
          // (2^23 + bv) - (2^23 + 127)
          ev[n] = bv == 255u ? __uint_as_float(0x7fc00000u)
                             : __uint_as_float(0x4b000000u | bv) - 8388735.f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = (s[b][0][2 * n + e] + s[b][1][2 * n + e]) * factor[b][e];
            y[b][2 * n + e] = NARROW ? x * kf * 16384.f : x;
          }
      }
      if (part) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            y[b][x] = seen[b][x % 2] >> (key0 + 8 * (x / 2)) & 1 ? y[b][x] : -INFINITY;
      }
      // ------------------------------------ the rows' maxima (if they grow) --
      float top[NB][2], topt[NB][2];
      bool grow = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[b][e] = fmaxf(y[b][e], y[b][2 + e]);
          grow |= top[b][e] > m[b][e] + 8.f;
          if constexpr (NARROW) {
            topt[b][e] = fmaxf(y[b][e] + ev[0], y[b][2 + e] + ev[1]);
            grow |= topt[b][e] > mt[b][e] + 8.f;
          }
        }
      // m is moved only for a weight above 2^8, or for a row's first key (until
      // then weights are as exact, and 1 / l uses the same m)
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              top[b][e] = fmaxf(top[b][e], __shfl_xor_sync(0xffffffffu, top[b][e], x));
              if (NARROW)
                topt[b][e] = fmaxf(topt[b][e], __shfl_xor_sync(0xffffffffu, topt[b][e], x));
            }
            const float nm = top[b][e] > m[b][e] + 8.f ? top[b][e] : m[b][e];
            float down = nm != m[b][e] ? ex2(m[b][e] - nm) : 1.f;
            m[b][e] = nm;
            l[b][e] *= down;
            if constexpr (NARROW) {
              const float nt = topt[b][e] > mt[b][e] + 8.f ? topt[b][e] : mt[b][e];
              down = nt != mt[b][e] ? ex2(mt[b][e] - nt) : 1.f;
              mt[b][e] = nt;
            }
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) o[b][i][e] *= down, o[b][i][2 + e] *= down;
          }
      }
      // ----------------------------------------------------------- weights --
      uint32_t pf[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = m[b][e] == -INFINITY ? 0.f : m[b][e];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            p[2 * n + e] = ex2(y[b][2 * n + e] - base);
            l[b][e] += p[2 * n + e];
          }
          if constexpr (NARROW) {
            // fp16 weights, 64 at the running maximum (at most 2^14): half a step
            // of 2^-11 each, or of 2^-31 of the maximum where they are small
            const float baset = (mt[b][e] == -INFINITY ? 0.f : mt[b][e]) - 6.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
              // (a hidden key's exponent may be NaN: its weight stays 0)
              p[2 * n + e] = y[b][2 * n + e] == -INFINITY ? 0.f
                                                         : ex2(y[b][2 * n + e] + ev[n] - baset);
          }
        }
        // bf16 weights: half a step of 2^-8 each, as much as the output's own
        // rounding; the sums keep the fp32 weights
#pragma unroll
        for (int n = 0; n < 2; ++n)
          pf[b][n] = transposed(NARROW ? pack_f16(p[2 * n], p[2 * n + 1])
                                       : pack_bf16(p[2 * n], p[2 * n + 1]));
      }
      // ------------------------------------------------------- V^T P^T --
      // the halves of A's words whose keys no row sees become 0 (whatever stands
      // there, a code of NaN too: its weight of 0 would not hide it)
      uint32_t keep0 = ~0u, keep1 = ~0u;
      if (part) {
        const uint32_t g16 = uint32_t(gone >> kb);
        const int e0 = key_of(2 * j4), e1 = key_of(2 * j4 + 1);
        keep0 = (g16 >> e0 & 1 ? 0u : 0xffffu) | (g16 >> e1 & 1 ? 0u : 0xffff0000u);
        keep1 = (g16 >> (e0 + 8) & 1 ? 0u : 0xffffu) | (g16 >> (e1 + 8) & 1 ? 0u : 0xffff0000u);
      }
      if constexpr (NARROW) {
        const int key = kb + 8 * (lm & 1) + key_of(lrow);
#pragma unroll
        for (int cc = 0; cc < HD / 32; ++cc) {
          uint32_t r[4];
          const int c16 = 2 * cc + (lm >> 1);
          const int ch = HD == 128 ? c16 ^ (key & 7) : c16 ^ ((key >> 1) & 3);
          ldmatrix4<true>(r, vbase + key * HD + ch * 16);
          // a word holds the codes of d, d + 1 of two keys: even d are A's rows
          // 0-7, odd d its rows 8-15
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = __byte_perm(r[2 * i] & keep0, 0, 0x3120),
                           z = __byte_perm(r[2 * i + 1] & keep1, 0, 0x3120);
            const uint32_t a[4] = {codes16(uint16_t(x)), codes16(uint16_t(x >> 16)),
                                   codes16(uint16_t(z)), codes16(uint16_t(z >> 16))};
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816<true>(o[b][2 * cc + i], a, pf[b][0], pf[b][1]);
          }
        }
      } else {
        const uint32_t row = vbase + (kb + 8 * (lm >> 1) + lrow) * 128;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
          uint32_t a[4];
          ldmatrix4<true>(a, row + (c / 4) * (BN * 128) + ((2 * (c % 4) + (lm & 1)) ^ lrow) * 16);
          if (part) {
            // and so do the others' infinities and NaNs, which are added back to
            // the rows that see them
            a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = odd16(a[e]);
              bad |= x != 0u;
              a[e] &= ~((x >> 15) * 0xffffu);
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) mma16816<false>(o[b][c], a, pf[b][0], pf[b][1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[slot]);
    if (++slot == G::SLOTS) slot = 0, par ^= 1;
  }
  if (!ok) fail(FP_ERR_TIMEOUT);
  if (lane == 0 && *abort_flag) {
    // drain: wait (bounded) for this warp's loads that may be in flight, its last
    // two turns' (a third would need more than 8 slots) and the first tiles
    volatile int never = 0;
    for (int k = 1; k <= 2; ++k) {
      const int t = turn - k * WARPS - 1 + G::SLOTS;
      if (turn - k * WARPS > 0 && t < ntile)
        bar_wait(&sm.full[t % G::SLOTS], (t / G::SLOTS) & 1, &never, 100000000ull);
    }
    if (warp == 0)
      for (int t = 0; t < begun; ++t) bar_wait(&sm.full[t], 0, &never, 100000000ull);
  }
  __syncwarp();

  // ------------------------------------------------- the warps' results --
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], x);
  if (__any_sync(0xffffffffu, bad) && lane == 0) sm.poison = missing ? 3 : 1;
  __syncthreads();  // the ring is no longer read
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * b + 2 * j4 + e;
      if (i8 == 0) sm.ml[warp][r] = make_float2(m[b][e], l[b][e]);
      if constexpr (NARROW) {
        // O to the weights' own reference: 2^(mt - m - 6), in two factors (it may
        // lie outside fp32 where the product does not)
        const float base = m[b][e] == -INFINITY ? 0.f : m[b][e];
        const float f = ex2(0.5f * (mt[b][e] == -INFINITY ? 0.f : mt[b][e] - base - 6.f));
#pragma unroll
        for (int c = 0; c < HD / 16; ++c)
          *reinterpret_cast<float2 *>(&sm.o[warp][r][16 * c + 2 * i8]) =
              make_float2(o[b][c][e] * f * f, o[b][c][2 + e] * f * f);
      } else {
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
          sm.o[warp][r][16 * c + i8] = o[b][c][e];
          sm.o[warp][r][16 * c + 8 + i8] = o[b][c][2 + e];
        }
      }
    }
  __syncthreads();
  const bool whole = un.units == 1;
  const size_t part0 = whole ? 0 : (first_part(sp, kv) + un.part) * sp.rows;
  ok = ok && !*abort_flag;
  // one row's result at 4 columns: out and lse
  auto store = [&](int r, int d, float big, float l, float4 x) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(out + (row0 + r) * HD + d) =
        make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (lse && d == 0)
      lse[row0 + r] = l == 0.f ? -INFINITY : (big + log2f(l)) * 0.6931471805599453f;
  };
  for (int e = threadIdx.x; e < rt.rows * (HD / 4); e += THREADS) {
    const int r = e / (HD / 4), d = e % (HD / 4) * 4;
    float big = -INFINITY;
#pragma unroll
    for (int k = 0; k < WARPS / R; ++k) big = fmaxf(big, sm.ml[k * R + r / 16][r % 16].x);
    const float base = big == -INFINITY ? 0.f : big;
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < WARPS / R; ++k) {
      const int w = k * R + r / 16;
      const float2 ml = sm.ml[w][r % 16];
      const float f = ex2(ml.x - base);
      const float4 y = *reinterpret_cast<const float4 *>(&sm.o[w][r % 16][d]);
      l = fmaf(f, ml.y, l);
      x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
    }
    if (!ok) l = 0.f, x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!whole) {
      // the unit's partial result, whose maximum is -infinity where the row sees none
      // of its keys: any number in its place would be taken for a score when the
      // units are joined
      *reinterpret_cast<float4 *>(sp.part_o + (part0 + r) * HD + d) = x;
      if (d == 0) sp.part_ml[part0 + r] = make_float2(big, l);
    } else if (sp.cluster == 1) {
      store(r, d, big, l, x);
    } else {
      *reinterpret_cast<float4 *>(&sm.all_o[r][d]) = x;
      if (d == 0) sm.all_ml[r] = make_float2(big, l);
    }
  }
  int poison = sm.poison;
  int r_first = 0, r_step = 1;  // the rows that this CTA writes
  if (sp.cluster > 1) {
    // the CTAs that share the unit join their rows through each other's shared
    // memory, rows dealt out in turn, pieces in the CTAs' order
    cluster_sync();
    r_first = crank, r_step = sp.cluster;
    if (!NARROW)
      for (int c = 0; c < sp.cluster; ++c)
        poison |= ld_cluster(cluster_addr(smem_u32(&sm.poison), c));
    const int mine = rt.rows > crank ? (rt.rows - crank + sp.cluster - 1) / sp.cluster : 0;
    for (int e = threadIdx.x; e < mine * (HD / 4); e += THREADS) {
      const int r = crank + e / (HD / 4) * sp.cluster, d = e % (HD / 4) * 4;
      float big = -INFINITY, l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int c0 = 0; c0 < sp.cluster; c0 += 8) {
        float2 ml[8];
        float4 y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int from = c0 + c < sp.cluster ? c0 + c : 0;
          ml[c] = ld_cluster2(cluster_addr(smem_u32(&sm.all_ml[r]), from));
          y[c] = ld_cluster4(cluster_addr(smem_u32(&sm.all_o[r][d]), from));
          if (c0 + c >= sp.cluster) ml[c] = make_float2(-INFINITY, 0.f);
        }
        float top = big;
#pragma unroll
        for (int c = 0; c < 8; ++c) top = fmaxf(top, ml[c].x);
        const float base = top == -INFINITY ? 0.f : top, old = ex2(big - base);
        big = top;
        l *= old;
        x.x *= old, x.y *= old, x.z *= old, x.w *= old;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float f = ex2(ml[c].x - base);
          if (c0 + c >= sp.cluster) continue;
          l = fmaf(f, ml[c].y, l);
          x.x = fmaf(f, y[c].x, x.x), x.y = fmaf(f, y[c].y, x.y);
          x.z = fmaf(f, y[c].z, x.z), x.w = fmaf(f, y[c].w, x.w);
        }
      }
      store(r, d, big, l, x);
    }
    cluster_sync();  // nobody leaves while its shared memory is read
  }
  if (!NARROW && poison) {
    __syncthreads();  // the rows are written
    // (a lane a row: at most 64 rows, whole warps)
    static_assert(THREADS >= 64, "a thread for each row");
    const int r = r_first + threadIdx.x * r_step;
    const bool row = r < rt.rows;
    add_odd_values<HD>(P, seq, rt, un.s, kv, kt, unit_first, unit_count,
                       row_position(seq, rt, r), (poison & 2) != 0,
                       row && whole ? out + (row0 + r) * HD : nullptr,
                       row && !whole ? sp.part_o + (part0 + r) * HD : nullptr);
  }
}

template <int HD, bool NARROW, int RG>
cudaError_t run(const Problem &P, const Split &sp, const void *q, void *out, float *lse,
                cudaStream_t st) {
  auto *kernel = attn_few_kernel<HD, NARROW, RG>;
  constexpr int bytes = int(sizeof(FewSmem<HD, NARROW, RG>));
  static_assert(Ring<HD, NARROW, RG>::CTAS * (bytes + 1024) <= 233472, "the SM holds them");
  static std::atomic<bool> set[64];
  cudaError_t e = once_per_device(set, [&] {
    const cudaError_t r =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const uint64_t rows = uint64_t(P.n_pages) * P.hkv * P.page;
  const uint32_t box = P.page > BN ? BN : P.page;
  const CUtensorMapSwizzle swizzle =
      NARROW && HD == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_map(&mk, P.k, rows, HD, NARROW ? HD : 64, box, NARROW, swizzle) ||
      !encode_map(&mv, P.v, rows, HD, NARROW ? HD : 64, box, NARROW, swizzle))
    return cudaErrorInvalidValue;
  const dim3 grid = grid_of(P, sp);
  __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(out);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = sp.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sp.cluster > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, P, sp, static_cast<const __nv_bfloat16 *>(q), ob,
                         lse, serve_status_ptr());
  if (e != cudaSuccess || !sp.on) return e;
  return launch_join<HD, 64, 8>(P, sp, ob, lse, st);
}

template <int HD, bool NARROW>
cudaError_t run_rows(const Problem &P, const Split &sp, const void *q, void *out, float *lse,
                     cudaStream_t st) {
  const int rows = P.max_q_len * P.g;
  if (rows <= 8) return run<HD, NARROW, 0>(P, sp, q, out, lse, st);
  if (rows <= 16) return run<HD, NARROW, 1>(P, sp, q, out, lse, st);
  if (rows <= 32) return run<HD, NARROW, 2>(P, sp, q, out, lse, st);
  return run<HD, NARROW, 4>(P, sp, q, out, lse, st);
}

// How the CTAs share the work.  Where the items are few and short, a cluster of
// 16, 8, 4 or 2 takes an item and joins its parts through shared memory.  Items
// that are too long for that, or too many, are cut into units for the whole
// machine, which a second kernel joins (some 4 us).  Measured in us, cluster against
// units: 8 items (of 32 heads over 8) of 141 tiles 13.7, 14.7, of 250 tiles 19.3,
// 17.1; 128 items of 32 tiles 26.4, 29.4, of 63 tiles 44.0, 46.6; 2 items, whose
// clusters use 32 SMs, of 250 tiles 20.3, 15.8.
Split few_split(const Problem &P, bool narrow) {
  // (clusters that run at a time: 14, 33, 71, 148, as the occupancy call says)
  static const int sizes[4] = {16, 8, 4, 2}, fit[4] = {8, 32, 64, 128};
  const long long items = static_cast<long long>(P.n_seqs) * P.hkv * most_row_tiles<64>(P);
  for (int i = 0; i < 4; ++i)
    if (items <= fit[i]) {
      // tiles for each CTA: 8 to 16, by how much of the machine the clusters use
      const int each = std::min(16, std::max(8, int(items) * sizes[i] / 10));
      if (most_tiles(P) <= each * sizes[i]) {
        Split sp = {};
        sp.cluster = sizes[i];
        sp.tiles = most_row_tiles<64>(P);
        return sp;
      }
    }
  const int ctas = !narrow ? 2 : P.max_q_len * P.g > 8 ? 3 : 4;
  return make_split<64>(P, 4, 4, ctas * kSms);
}

}  // namespace

bool attn_few_takes(const Problem &P) {
  return P.page != 0 && static_cast<long long>(P.max_q_len) * P.g <= 64;
}

size_t attn_few_ws_bytes(const Problem &P, bool narrow) {
  Split sp = few_split(P, narrow);
  return sp.on ? carve(P, &sp, nullptr) : 0;
}

cudaError_t launch_attn_few(const Problem &P, bool narrow, const void *q, void *out, float *lse,
                            void *ws, cudaStream_t st) {
  Split sp = few_split(P, narrow);
  if (sp.on) carve(P, &sp, ws);
  if (P.d == 64)
    return narrow ? run_rows<64, true>(P, sp, q, out, lse, st)
                  : run_rows<64, false>(P, sp, q, out, lse, st);
  return narrow ? run_rows<128, true>(P, sp, q, out, lse, st)
                : run_rows<128, false>(P, sp, q, out, lse, st);
}

}  // namespace fps
