// serve_internal.cuh -- shared declarations of the CUDA implementation of
// fp_serve.h (libfp_serve.so).  The device helpers (mbarriers, TMA, tcgen05)
// are those of fp_internal.cuh.
#pragma once

#include "../../../include/fp_serve.h"
#include "../fp_internal.cuh"

#include <cuda_fp16.h>

namespace fps {

using namespace fpi;

// Where keys and values come from, and who asks: a paged cache with a batch of
// sequences, or (page == 0) contiguous [n_seqs, hkv, max_q_len, d] tensors in
// which every sequence is max_q_len tokens long and all of them are new.
struct Problem {
  int n_seqs, hq, hkv, g, d;
  int n_pages, page, shift, max_pages, max_q_len, total_q;  // page == 1 << shift
  // The pages' vectors lie at [sequence, index in its row of the table], not at the
  // pages' numbers (copies of what a batch reads).
  int by_place;
  int window;  // > 0 (no window: a number above every length)
  int sinks;
  const int32_t *table, *kv_lens, *q_offsets;
  const void *k, *v;
  const uint8_t *k_exps, *v_exps;
};

// One sequence's new tokens: packed rows h * n + t (+ the sequence's base) and
// positions len - n + t.  ok = false: its description failed a check.
struct Seq {
  int q0, n, len;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const Problem &P, int s) {
  Seq x;
  if (P.page == 0) {
    x.q0 = s * P.max_q_len;
    x.n = x.len = P.max_q_len;
    x.ok = true;
    return x;
  }
  x.len = P.kv_lens[s];
  if (P.q_offsets) {
    x.q0 = P.q_offsets[s];
    const int q1 = P.q_offsets[s + 1];
    x.ok = x.q0 >= 0 && q1 >= x.q0 && q1 <= P.total_q && q1 - x.q0 <= P.max_q_len;
    x.n = x.ok ? q1 - x.q0 : 0;
  } else {
    x.q0 = s * P.max_q_len;
    x.n = P.max_q_len;
    x.ok = true;
  }
  if (x.len < 0 || x.len > P.max_pages * P.page) x.ok = false;
  if (!x.ok) x.n = x.len = 0;
  return x;
}

// Row of (page, kv head, slot 0) in the cache's [n_pages * hkv * page, d], or -1
// for a page that does not exist.
__device__ __forceinline__ long long page_row(const Problem &P, int s, int index, int kv) {
  const int id = P.table[size_t(s) * P.max_pages + index];
  if (id < 0 || id >= P.n_pages) return -1;
  return (static_cast<long long>(id) * P.hkv + kv) * P.page;
}
// The same where P.k and P.v may be copies by place.
__device__ __forceinline__ long long held_row(const Problem &P, int s, int index, int kv) {
  const long long row = page_row(P, s, index, kv);
  if (!P.by_place || row < 0) return row;
  return ((static_cast<long long>(s) * P.max_pages + index) * P.hkv + kv) * P.page;
}

// The 4 codes of a word times 2^(byte - 127), exact (NaN for byte 255).
__device__ __forceinline__ float4 e4m3_values(uint32_t w, uint32_t byte) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)),
               b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  const float scale = __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

int *serve_status_ptr();  // this library's per-device status word

cudaError_t launch_kv_write(const Problem &P, int cache_dtype, int dtype, const void *k,
                            const void *v, cudaStream_t st);
cudaError_t launch_kv_read(const Problem &P, int cache_dtype, int dtype, void *k, void *v,
                           cudaStream_t st);
// bf16 copies of the 8-bit vectors that a batch reads, by place or by page number.
cudaError_t launch_kv_widen(const Problem &P, bool by_place, void *k, void *v, cudaStream_t st);
// fp32 queries: CUDA-core attention over fp32 or (narrow) 8-bit vectors.
cudaError_t launch_attn_rows(const Problem &P, bool narrow, const float *q, float *out,
                             float *lse, cudaStream_t st);
// bf16 queries: tensor-core attention over bf16 or (narrow) 8-bit vectors.
bool attn_few_takes(const Problem &P);  // few enough rows for the first
size_t attn_few_ws_bytes(const Problem &P, bool narrow);
cudaError_t launch_attn_few(const Problem &P, bool narrow, const void *q, void *out, float *lse,
                            void *ws, cudaStream_t st);
size_t attn_serve_ws_bytes(const Problem &P, bool narrow);
cudaError_t launch_attn_serve(const Problem &P, bool narrow, const void *q, void *out, float *lse,
                              void *ws, cudaStream_t st);

}  // namespace fps
