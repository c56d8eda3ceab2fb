// attn_rows.cu -- attention of packed query rows over visible keys on the CUDA
// cores, fp32 products and sums throughout (the fp32 path of fp_window_attn and
// fp_paged_attn).
//
// out_i = sum_j p_ij v_j / sum_j p_ij with p_ij = exp(s_ij - m_i), one pass over
// the visible 64-key tiles with a running maximum m and sum (online softmax).
// A CTA takes 64 query rows that share a kv head (16, where 64 would leave SMs
// without work); 16 threads share 4 (2) rows and hold 4 scores and d/16 outputs of
// each, so a product reads 8 (6) vectors of 4 numbers from shared memory for 64
// (32) multiply-adds.  The next tile of K and V is copied in while one is used.
// Bound by that shared-memory traffic and the FMA pipe; there is no split over the
// keys (a debug path).  1024 tokens, 2 heads, d 64, window 256: 41 us with 64 rows,
// 23 with 16.
#include <math.h>

#include <type_traits>

#include "split.cuh"

namespace fps {
namespace {

constexpr int KEYS = 64;

template <int D, int ROWS>
struct RowsSmem {
  float q[ROWS][D + 4];
  float k[2][KEYS][D + 4];
  float v[2][KEYS][D + 4];
  float p[ROWS][KEYS + 4];
};

__device__ __forceinline__ float4 load4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }

// 4 elements at column c of the 8-bit key (or value) vector at row `row`.
__device__ __forceinline__ float4 vector4(const void *base, const uint8_t *exps, long long row,
                                          int d, int c) {
  return e4m3_values(
      *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(base) + row * d + c),
      exps[row]);
}

// 16 bytes into shared memory, behind the thread's back; zeros where there is
// nothing to read.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// threads of a CTA of ROWS rows: 16 for each 4 rows, or 2
constexpr int threads_of(int rows) { return rows == 64 ? 256 : 8 * rows; }

template <class C, int D, int ROWS>
__global__ void __launch_bounds__(threads_of(ROWS))
    attn_rows_kernel(const Problem P, const float *__restrict__ q, float *__restrict__ out,
                     float *__restrict__ lse, int *status) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  constexpr int THREADS = threads_of(ROWS), R = ROWS * 16 / THREADS;  // R: rows of a thread
  auto &sm = *reinterpret_cast<RowsSmem<D, ROWS> *>(smem_raw);
  const int s = blockIdx.z, kv = blockIdx.y;
  const Seq seq = load_seq(P, s);
  if (!seq.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && kv == 0) report(status, FP_ERR_DEVICE_CHECK);
    return;
  }
  const RowTile rt = row_tile<ROWS>(P, seq, int(blockIdx.x));
  if (rt.rows <= 0) return;
  const KeyTiles kt = key_tiles(P, seq, rt);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const float scale = 1.f / sqrtf(float(D));

  // packed row of tile row 0 (the group's rows are consecutive)
  const size_t row0 = size_t(seq.q0) * P.hq + size_t(kv) * P.g * seq.n + rt.first;
  for (int e = threadIdx.x; e < ROWS * D / 4; e += THREADS) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const float4 x =
        r < rt.rows ? load4(q + (row0 + r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    sm.q[r][c] = x.x * scale, sm.q[r][c + 1] = x.y * scale;
    sm.q[r][c + 2] = x.z * scale, sm.q[r][c + 3] = x.w * scale;
  }
  int pos[R];
  float m[R], l[R], acc[R][D / 16];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    pos[i] = row_position(seq, rt, ty * R + i);
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
  }
  const long long row_s = (static_cast<long long>(s) * P.hkv + kv) * seq.len;
  // Copies a tile in; false if one of its pages does not exist.  A key at or past
  // the sequence's end, or in such a page, comes as zeros and is seen by nobody.
  auto load = [&](int t, int stage) -> bool {
    const int t0 = kt.key(t), c = threadIdx.x % (D / 4) * 4;
    bool there = true;
#pragma unroll 4
    for (int r = threadIdx.x / (D / 4); r < KEYS; r += THREADS / (D / 4)) {
      const int key = t0 + r;
      long long row = -1;
      if (key < seq.len) {
        if (P.page == 0) {
          row = row_s + key;
        } else {
          row = page_row(P, s, key >> P.shift, kv);
          if (row >= 0)
            row += (key & (P.page - 1));
          else
            there = false;
        }
      }
      float *dk = &sm.k[stage][r][c], *dv = &sm.v[stage][r][c];
      if constexpr (sizeof(C) == 1) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        store4(dk, row < 0 ? zero : vector4(P.k, P.k_exps, row, D, c));
        store4(dv, row < 0 ? zero : vector4(P.v, P.v_exps, row, D, c));
      } else {
        const size_t at = row < 0 ? 0 : size_t(row) * D + c;
        copy16(dk, static_cast<const float *>(P.k) + at, row >= 0);
        copy16(dv, static_cast<const float *>(P.v) + at, row >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return there;
  };
  const int tiles = kt.count();
  bool next_there = tiles > 0 && load(0, 0);
  for (int t = 0; t < tiles; ++t) {
    const int t0 = kt.key(t), stage = t % 2;
    const bool mine = next_there;
    if (t + 1 < tiles) {
      next_there = load(t + 1, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    const bool there = __syncthreads_and(mine);
    float sc[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 a[R], b[4];
#pragma unroll
      for (int i = 0; i < R; ++i) a[i] = load4(&sm.q[ty * R + i][c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = load4(&sm.k[stage][tx + 16 * j][c]);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][j] = fmaf(a[i].x, b[j].x, sc[i][j]);
          sc[i][j] = fmaf(a[i].y, b[j].y, sc[i][j]);
          sc[i][j] = fmaf(a[i].z, b[j].z, sc[i][j]);
          sc[i][j] = fmaf(a[i].w, b[j].w, sc[i][j]);
        }
    }
    uint64_t hidden_pages = 0;
    if (!there) {
      hidden_pages = missing_keys(P, s, seq, t0);
      if (threadIdx.x == 0 && (hidden_pages & used_keys(P, seq, rt, t0)))
        report(status, FP_ERR_DEVICE_CHECK);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint64_t seen = seen_keys(P, pos[i], t0) & ~hidden_pages;
      float tmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (seen >> (tx + 16 * j) & 1) tmax = fmaxf(tmax, sc[i][j]);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
      const float mnew = fmaxf(m[i], tmax);
      const float base = mnew == -INFINITY ? 0.f : mnew;
      const float alpha = expf(m[i] - base);
      float ps = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // a hidden key's weight is marked by -1: its value must not be touched
        const bool in = seen >> (tx + 16 * j) & 1;
        const float p = in ? expf(sc[i][j] - base) : -1.f;
        if (in) ps += p;
        sm.p[ty * R + i][tx + 16 * j] = p;
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
      l[i] = l[i] * alpha + ps;
      m[i] = mnew;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[i][c] *= alpha;
    }
    __syncwarp();  // a row's 16 threads are in one warp
    // (in a tile seen in part, what belongs to a hidden key is computed and thrown
    // away: a weight of 0 would not hide a NaN)
    auto product = [&](auto part) {
#pragma unroll 4
      for (int j = 0; j < KEYS; j += 4) {
        float4 p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = load4(&sm.p[ty * R + i][j]);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          float4 b[D / 64];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) b[c] = load4(&sm.v[stage][j + jj][c * 64 + tx * 4]);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
            const bool keep = !decltype(part)::value || !(w < 0.f);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const float y[4] = {b[c].x, b[c].y, b[c].z, b[c].w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float z = fmaf(w, y[x], acc[i][4 * c + x]);
                acc[i][4 * c + x] = keep ? z : acc[i][4 * c + x];
              }
            }
          }
        }
      }
    };
    if (partial_tile(P, seq, rt, t0, !there))
      product(std::true_type());
    else
      product(std::false_type());
    __syncthreads();  // the tile is used up
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ty * R + i;
    if (r >= rt.rows) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(out + (row0 + r) * D + c * 64 + tx * 4,
             make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                         acc[i][4 * c + 3] * inv));
    if (lse && tx == 0) lse[row0 + r] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
}

template <class C, int D, int ROWS>
cudaError_t run_rows(const Problem &P, const float *q, float *out, float *lse, cudaStream_t st) {
  const size_t smem = sizeof(RowsSmem<D, ROWS>);
  static std::atomic<bool> set[64];
  const cudaError_t e = once_per_device(set, [&] {
    return cudaFuncSetAttribute(attn_rows_kernel<C, D, ROWS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  });
  if (e != cudaSuccess) return e;
  attn_rows_kernel<C, D, ROWS>
      <<<dim3(most_row_tiles<ROWS>(P), P.hkv, P.n_seqs), threads_of(ROWS), smem, st>>>(
          P, q, out, lse, serve_status_ptr());
  return cudaGetLastError();
}

template <class C, int D>
cudaError_t run(const Problem &P, const float *q, float *out, float *lse, cudaStream_t st) {
  const long long tiles = static_cast<long long>(most_row_tiles<64>(P)) * P.hkv * P.n_seqs;
  return tiles < 2 * 148 ? run_rows<C, D, 16>(P, q, out, lse, st)
                         : run_rows<C, D, 64>(P, q, out, lse, st);
}

}  // namespace

cudaError_t launch_attn_rows(const Problem &P, bool narrow, const float *q, float *out,
                             float *lse, cudaStream_t st) {
  if (P.d == 64)
    return narrow ? run<uint8_t, 64>(P, q, out, lse, st) : run<float, 64>(P, q, out, lse, st);
  return narrow ? run<uint8_t, 128>(P, q, out, lse, st) : run<float, 128>(P, q, out, lse, st);
}

}  // namespace fps
