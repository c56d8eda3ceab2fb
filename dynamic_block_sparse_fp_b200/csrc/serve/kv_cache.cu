// kv_cache.cu -- fp_kv_write and fp_kv_read: new tokens' keys and values into the
// slots of a paged cache, in 8 bits where the cache is, and back; and the bf16
// copies of 8-bit pages that chunks of new tokens attend to.
//
// One vector (d elements of one token and head of K or V) is handled by a group of
// neighbouring lanes, 8 elements each (of an 8-bit cache 16, which a read takes as 8
// of each half, so that its stores are without gaps: 131072 tokens 143 us with 16 in
// a row, 132 so).  The 8-bit scale of a vector needs its largest magnitude: an
// exchange among those lanes.  Every thread has AHEAD vectors in hand, whose page
// numbers and elements are all asked for before the first is used.
// Bound by DRAM: each element is read once and written once.  Measured (8 kv heads,
// d 128): 32768 tokens into 8 bits 37 us (5.5 TB/s), 131072 out of 8 bits 132 us
// (6.1 TB/s); 32768 of bf16 in 47 us, out 49 us (5.7 and 5.5 TB/s), of fp32 88 and 90
// (6.1 and 6.0).
#include "serve_internal.cuh"

namespace fps {
namespace {

constexpr int THREADS = 256;

// 8 elements of one lane: as they come, and as fp32.
template <class T>
struct alignas(16) Raw {
  uint4 w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw<T> load8(const T *p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
  return r;
}
template <class T>
__device__ __forceinline__ void store8(T *p, const Raw<T> &r) {
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
}
__device__ __forceinline__ void floats(const Raw<float> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.w[i].x);
    x[4 * i + 1] = __uint_as_float(r.w[i].y);
    x[4 * i + 2] = __uint_as_float(r.w[i].z);
    x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void floats(const Raw<__nv_bfloat16> &r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ Raw<float> raw(const float4 &a, const float4 &b, float) {
  Raw<float> r;
  r.w[0] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z),
                      __float_as_uint(a.w));
  r.w[1] = make_uint4(__float_as_uint(b.x), __float_as_uint(b.y), __float_as_uint(b.z),
                      __float_as_uint(b.w));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ Raw<__nv_bfloat16> raw(const float4 &a, const float4 &b,
                                                  __nv_bfloat16) {
  Raw<__nv_bfloat16> r;
  r.w[0] = make_uint4(bf16_pair(a.x, a.y), bf16_pair(a.z, a.w), bf16_pair(b.x, b.y),
                      bf16_pair(b.z, b.w));
  return r;
}
template <class T>
__device__ __forceinline__ Raw<T> zeros() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
  return r;
}

// Two fp32 to e4m3, rounded to nearest even (|x| <= 448 here); y is the high byte.
__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// The exponent byte of a vector whose largest magnitude has these fp32 bits:
// e + 127 for the smallest e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(e + 8);
// 255 for an infinity or a NaN (whose bits, sign cleared, are the largest).
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = int(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return uint32_t(b < 1 ? 1 : b);
}

constexpr int AHEAD = 4;
// (a vector on its way into 8 bits takes twice the registers; 32768 tokens, against 2
// a thread: 9 % longer with 4, 29 % with 8)
template <class C>
constexpr int write_ahead() {
  return sizeof(C) == 1 ? 2 : AHEAD;
}

// The vectors of one sequence's new tokens, i = head * n + token.
struct Vectors {
  const Problem &P;
  const Seq q;
  const int s, total;
  const uint32_t magic;
  int *status;
  __device__ Vectors(const Problem &P_, const Seq &q_, int s_, int *status_)
      : P(P_), q(q_), s(s_), total(q_.n * P_.hkv), magic(q_.n > 0 ? 0xffffffffu / q_.n : 0u),
        status(status_) {}
  // Row of vector i in the cache; -1: it has none.
  __device__ __forceinline__ long long slot(int i) const {
    // i / n: the quotient by the rounded-down reciprocal is 1 too small at most
    int h = __umulhi(uint32_t(i), magic), t = i - h * q.n;
    if (t >= q.n) ++h, t -= q.n;
    const int pos = q.len - q.n + t;
    if (pos < 0) return -1;
    const long long row = page_row(P, s, pos >> P.shift, h);
    if (row < 0) {
      report(status, FP_ERR_DEVICE_CHECK);
      return -1;
    }
    return row + (pos & (P.page - 1));
  }
};

template <class T, class C, int D>
__global__ void __launch_bounds__(THREADS)
    kv_write_kernel(const __grid_constant__ Problem P, const T *__restrict__ k,
                    const T *__restrict__ v, int *status) {
  constexpr int E = sizeof(C) == 1 ? 16 : 8;  // elements of a lane
  constexpr int LANES = D / E, PER = THREADS / LANES, U = write_ahead<C>();
  const int s = blockIdx.y, lane = threadIdx.x % LANES;
  const Vectors vec(P, load_seq(P, s), s, status);
  if (!vec.q.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report(status, FP_ERR_DEVICE_CHECK);
    return;
  }
  const bool is_v = blockIdx.z != 0;
  const T *src = (is_v ? v : k) + size_t(vec.q.q0) * P.hkv * D;
  C *dst = static_cast<C *>(const_cast<void *>(is_v ? P.v : P.k));
  uint8_t *exps = const_cast<uint8_t *>(is_v ? P.v_exps : P.k_exps);
  for (int i0 = blockIdx.x * (PER * U); i0 < vec.total; i0 += gridDim.x * (PER * U)) {
    Raw<T> r[U][E / 8];
    long long slot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * PER + threadIdx.x / LANES;
      slot[u] = -1;
#pragma unroll
      for (int e = 0; e < E / 8; ++e) r[u][e] = zeros<T>();
      if (i < vec.total) {
        slot[u] = vec.slot(i);
#pragma unroll
        for (int e = 0; e < E / 8; ++e) r[u][e] = load8(src + size_t(i) * D + lane * E + 8 * e);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (sizeof(C) == 1) {
        float x[2][8];
        uint32_t amax = 0, c[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          floats(r[u][e], x[e]);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(x[e][j]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const uint32_t byte = exponent_byte(amax);
        // 2^-e: exact, and so is the product but for what rounds to zero anyway
        const float inv = __uint_as_float((254u - (byte == 255u ? 127u : byte)) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float *y = &x[j / 2][4 * (j % 2)];
          c[j] = e4m3_pair(y[0] * inv, y[1] * inv) | e4m3_pair(y[2] * inv, y[3] * inv) << 16;
          if (byte == 255u) c[j] = 0u;  // NaN by its exponent alone
        }
        if (slot[u] >= 0) {
          *reinterpret_cast<uint4 *>(dst + slot[u] * D + lane * E) =
              make_uint4(c[0], c[1], c[2], c[3]);
          if (lane == 0) exps[slot[u]] = uint8_t(byte);
        }
      } else {
        if (slot[u] >= 0) store8(reinterpret_cast<T *>(dst) + slot[u] * D + lane * E, r[u][0]);
      }
    }
  }
}

template <class T, class C, int D>
__global__ void __launch_bounds__(THREADS)
    kv_read_kernel(const __grid_constant__ Problem P, T *__restrict__ k, T *__restrict__ v,
                   int *status) {
  constexpr int E = sizeof(C) == 1 ? 16 : 8;
  constexpr int LANES = D / E, PER = THREADS / LANES;
  const int s = blockIdx.y, lane = threadIdx.x % LANES;
  const Vectors vec(P, load_seq(P, s), s, status);
  if (!vec.q.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report(status, FP_ERR_DEVICE_CHECK);
    return;
  }
  const bool is_v = blockIdx.z != 0;
  T *dst = (is_v ? v : k) + size_t(vec.q.q0) * P.hkv * D;
  const C *src = static_cast<const C *>(is_v ? P.v : P.k);
  const uint8_t *exps = is_v ? P.v_exps : P.k_exps;
  for (int i0 = blockIdx.x * (PER * AHEAD); i0 < vec.total; i0 += gridDim.x * (PER * AHEAD)) {
    long long slot[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u * PER + threadIdx.x / LANES;
      slot[u] = i < vec.total ? vec.slot(i) : -1;
    }
    if constexpr (sizeof(C) == 1) {
      uint4 c[AHEAD];
      uint32_t byte[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        c[u] = make_uint4(0u, 0u, 0u, 0u);
        byte[u] = 127u;
        if (slot[u] >= 0) {
          const C *from = src + slot[u] * D + lane * 8;
          const uint2 a = *reinterpret_cast<const uint2 *>(from);
          const uint2 b = *reinterpret_cast<const uint2 *>(from + D / 2);
          c[u] = make_uint4(a.x, a.y, b.x, b.y);
          byte[u] = exps[slot[u]];
        }
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * PER + threadIdx.x / LANES;
        if (i >= vec.total) continue;
        T *at = dst + size_t(i) * D + lane * 8;
        store8(at, raw(e4m3_values(c[u].x, byte[u]), e4m3_values(c[u].y, byte[u]), T()));
        store8(at + D / 2, raw(e4m3_values(c[u].z, byte[u]), e4m3_values(c[u].w, byte[u]), T()));
      }
    } else {
      Raw<T> r[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        r[u] = slot[u] >= 0 ? load8(reinterpret_cast<const T *>(src) + slot[u] * D + lane * E)
                            : zeros<T>();
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * PER + threadIdx.x / LANES;
        if (i < vec.total) store8(dst + size_t(i) * D + lane * E, r[u]);
      }
    }
  }
}

// The keys of a sequence that its new tokens see, as bf16 (16 codes a lane), at
// their place in the table or by their page's number.  By number, a page that two
// sequences share is written twice with the same numbers; a page that does not exist
// is not written.
template <int D>
__global__ void __launch_bounds__(THREADS)
    kv_widen_kernel(const Problem P, bool by_place, uint4 *__restrict__ k,
                    uint4 *__restrict__ v) {
  constexpr int LANES = D / 16, PER = THREADS / LANES;
  const int s = blockIdx.y, lane = threadIdx.x % LANES;
  const Seq q = load_seq(P, s);
  if (q.n == 0) return;
  // [0, sinks) and [first, len), the tiles' multiples of 64
  const int first = max(0, max(0, q.len - q.n) - P.window + 1) & ~63;
  const int sinks = min((P.sinks + 63) & ~63, first), keys = sinks + q.len - first;
  const bool is_v = blockIdx.z != 0;
  uint4 *dst = is_v ? v : k;
  const uint4 *src = static_cast<const uint4 *>(is_v ? P.v : P.k);
  const uint8_t *exps = is_v ? P.v_exps : P.k_exps;
  for (int i = blockIdx.x * PER + threadIdx.x / LANES; i < keys; i += gridDim.x * PER) {
    const int key = i < sinks ? i : first + i - sinks;
    const long long page = page_row(P, s, key >> P.shift, 0);
    if (page < 0) continue;
    const long long place = static_cast<long long>(s) * P.max_pages + (key >> P.shift);
    const long long first_row = by_place ? place * P.hkv * P.page : page;
    for (int h = 0; h < P.hkv; ++h) {
      const int in = h * P.page + (key & (P.page - 1));
      const long long row = page + in, to = first_row + in;
      const uint4 c = src[row * LANES + lane];
      const uint32_t byte = exps[row];
      const Raw<__nv_bfloat16> a = raw(e4m3_values(c.x, byte), e4m3_values(c.y, byte),
                                       __nv_bfloat16()),
                               b = raw(e4m3_values(c.z, byte), e4m3_values(c.w, byte),
                                       __nv_bfloat16());
      dst[(to * LANES + lane) * 2] = a.w[0];
      dst[(to * LANES + lane) * 2 + 1] = b.w[0];
    }
  }
}

// Blocks per sequence: enough for its vectors, and at most what the machine runs
// at a time a few times over.
template <class C>
dim3 grid_of(const Problem &P, int ahead) {
  const int elements = sizeof(C) == 1 ? 16 : 8;
  const long long vectors = static_cast<long long>(P.max_q_len) * P.hkv;
  const int per = THREADS / (P.d / elements) * ahead;
  long long x = (vectors + per - 1) / per;
  const long long most = (148ll * 32 + 2 * P.n_seqs - 1) / (2 * P.n_seqs);
  if (x > most) x = most;
  return dim3(unsigned(x), unsigned(P.n_seqs), 2);
}

template <class T, class C>
void write(const Problem &P, const void *k, const void *v, cudaStream_t st) {
  const T *kt = static_cast<const T *>(k), *vt = static_cast<const T *>(v);
  int *status = serve_status_ptr();
  const dim3 grid = grid_of<C>(P, write_ahead<C>());
  if (P.d == 64)
    kv_write_kernel<T, C, 64><<<grid, THREADS, 0, st>>>(P, kt, vt, status);
  else
    kv_write_kernel<T, C, 128><<<grid, THREADS, 0, st>>>(P, kt, vt, status);
}

template <class T, class C>
void read(const Problem &P, void *k, void *v, cudaStream_t st) {
  T *kt = static_cast<T *>(k), *vt = static_cast<T *>(v);
  int *status = serve_status_ptr();
  const dim3 grid = grid_of<C>(P, AHEAD);
  if (P.d == 64)
    kv_read_kernel<T, C, 64><<<grid, THREADS, 0, st>>>(P, kt, vt, status);
  else
    kv_read_kernel<T, C, 128><<<grid, THREADS, 0, st>>>(P, kt, vt, status);
}

}  // namespace

cudaError_t launch_kv_write(const Problem &P, int cache_dtype, int dtype, const void *k,
                            const void *v, cudaStream_t st) {
  if (cache_dtype == FP_BF16)
    write<__nv_bfloat16, __nv_bfloat16>(P, k, v, st);
  else if (cache_dtype == FP_F32)
    write<float, float>(P, k, v, st);
  else if (dtype == FP_BF16)
    write<__nv_bfloat16, uint8_t>(P, k, v, st);
  else
    write<float, uint8_t>(P, k, v, st);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const Problem &P, int cache_dtype, int dtype, void *k, void *v,
                           cudaStream_t st) {
  if (cache_dtype == FP_BF16)
    read<__nv_bfloat16, __nv_bfloat16>(P, k, v, st);
  else if (cache_dtype == FP_F32)
    read<float, float>(P, k, v, st);
  else if (dtype == FP_BF16)
    read<__nv_bfloat16, uint8_t>(P, k, v, st);
  else
    read<float, uint8_t>(P, k, v, st);
  return cudaGetLastError();
}

cudaError_t launch_kv_widen(const Problem &P, bool by_place, void *k, void *v, cudaStream_t st) {
  const long long keys = static_cast<long long>(P.max_pages) * P.page;
  const int per = THREADS / (P.d / 16);
  long long x = (keys + per - 1) / per;
  const long long most = (148ll * 16 + 2 * P.n_seqs - 1) / (2 * P.n_seqs);
  const dim3 grid(unsigned(x > most ? most : x), unsigned(P.n_seqs), 2);
  uint4 *kt = static_cast<uint4 *>(k), *vt = static_cast<uint4 *>(v);
  if (P.d == 64)
    kv_widen_kernel<64><<<grid, THREADS, 0, st>>>(P, by_place, kt, vt);
  else
    kv_widen_kernel<128><<<grid, THREADS, 0, st>>>(P, by_place, kt, vt);
  return cudaGetLastError();
}

}  // namespace fps
