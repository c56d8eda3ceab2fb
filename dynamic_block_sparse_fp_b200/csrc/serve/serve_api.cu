// serve_api.cu -- the extern "C" entry points of include/fp_serve.h: argument
// validation (on the host, before any launch) and dispatch.
#include <limits.h>

#include <atomic>
#include <mutex>

#include "serve_internal.cuh"

#define FP_API extern "C" __attribute__((visibility("default")))

namespace fpi {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  // a function-local static is initialised once, under the C++ runtime's lock
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult qr;
    void *p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) !=
            cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

}  // namespace fpi

namespace fps {

__device__ int g_serve_status;  // first device-side error since the last read

int *serve_status_ptr() {
  static int *ptrs[64] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_serve_status) == cudaSuccess) ptrs[dev] = static_cast<int *>(p);
  }
  return ptrs[dev];
}

namespace {

constexpr long long kRows = 1ll << 31;   // row coordinates fit in int32
constexpr int kTokens = 1 << 30;         // positions, with room for differences
constexpr int kGrid = 65535;             // grid.y and grid.z

fp_status check_device() {
  static std::atomic<int> cc[64];  // compute capability major, 0 = not yet read
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP_ERR_CUDA;
  int major = cc[dev].load(std::memory_order_relaxed);
  if (major == 0) {
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
      return FP_ERR_CUDA;
    cc[dev].store(major, std::memory_order_relaxed);
  }
  return major == 10 ? FP_OK : FP_ERR_UNSUPPORTED;
}

fp_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FP_OK : FP_ERR_CUDA; }

bool al(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

void set_window(Problem *P, int window, int sinks) {
  P->window = window <= 0 || window > kTokens ? kTokens : window;
  P->sinks = sinks > kTokens ? kTokens : sinks;
}

// The cache and the batch; pointers too unless `sizes_only`.
fp_status check_batch(const fp_kv_cache *c, const fp_batch *b, int hq, bool sizes_only,
                      Problem *P) {
  if (!c || !b) return FP_ERR_NULL;
  if (c->dtype != FP_BF16 && c->dtype != FP_F32 && c->dtype != FP_E4M3) return FP_ERR_DTYPE;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > kGrid) return FP_ERR_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FP_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return FP_ERR_SHAPE;
  if (static_cast<long long>(c->n_pages) * c->n_kv_heads >= kRows / c->page_size)
    return FP_ERR_SHAPE;
  if (b->n_seqs < 1 || b->n_seqs > kGrid || b->max_pages < 1 || b->max_q_len < 1 ||
      b->total_q < 0 || b->total_q >= kTokens || b->max_q_len >= kTokens)
    return FP_ERR_SHAPE;
  if (static_cast<long long>(b->max_pages) * c->page_size >= kTokens) return FP_ERR_SHAPE;
  if (hq < 1 || hq % c->n_kv_heads != 0) return FP_ERR_SHAPE;
  if (static_cast<long long>(b->total_q) * hq >= kRows) return FP_ERR_SHAPE;
  // row tiles of a sequence are counted in int32
  if (static_cast<long long>(b->max_q_len) * hq >= kRows) return FP_ERR_SHAPE;
  if (!sizes_only) {
    if (!b->q_offsets && static_cast<long long>(b->n_seqs) * b->max_q_len != b->total_q)
      return FP_ERR_SHAPE;
    if (!c->k || !c->v || !b->page_table || !b->kv_lens) return FP_ERR_NULL;
    if (c->dtype == FP_E4M3 && (!c->k_exps || !c->v_exps)) return FP_ERR_NULL;
    if (!al(c->k, 16) || !al(c->v, 16) || !al(c->k_exps, 16) || !al(c->v_exps, 16) ||
        !al(b->page_table, 4) || !al(b->kv_lens, 4) || !al(b->q_offsets, 4))
      return FP_ERR_ALIGN;
  }
  *P = Problem{};
  P->n_seqs = b->n_seqs;
  P->hq = hq;
  P->hkv = c->n_kv_heads;
  P->g = hq / c->n_kv_heads;
  P->d = c->head_dim;
  P->n_pages = c->n_pages;
  P->page = c->page_size;
  P->shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  P->max_pages = b->max_pages;
  P->max_q_len = b->max_q_len;
  P->total_q = b->total_q;
  P->table = b->page_table;
  P->kv_lens = b->kv_lens;
  P->q_offsets = b->q_offsets;
  P->k = c->k;
  P->v = c->v;
  P->k_exps = c->k_exps;
  P->v_exps = c->v_exps;
  return FP_OK;
}

fp_status check_kv(const fp_kv_cache *c, const fp_batch *b, int dtype, const void *k,
                   const void *v, Problem *P) {
  fp_status s = check_batch(c, b, c ? c->n_kv_heads : 1, false, P);
  if (s != FP_OK) return s;
  if (dtype != FP_BF16 && dtype != FP_F32) return FP_ERR_DTYPE;
  if (c->dtype != FP_E4M3 && c->dtype != dtype) return FP_ERR_DTYPE;
  if (P->total_q == 0) return FP_OK;
  if (!k || !v) return FP_ERR_NULL;
  if (!al(k, 16) || !al(v, 16)) return FP_ERR_ALIGN;
  return check_device();
}

fp_status run_attn(const Problem &P, int dtype, bool narrow, const void *q, void *out, float *lse,
                   void *ws, fp_stream_t stream) {
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == FP_F32)
    return cuda_status(launch_attn_rows(P, narrow, static_cast<const float *>(q),
                                        static_cast<float *>(out), lse, st));
  return cuda_status(attn_few_takes(P) ? launch_attn_few(P, narrow, q, out, lse, ws, st)
                                       : launch_attn_serve(P, narrow, q, out, lse, ws, st));
}

}  // namespace
}  // namespace fps

using namespace fps;

FP_API fp_status fp_window_attn(const fp_shape *shape, int window, int sinks, const void *q,
                                const void *k, const void *v, void *out, float *lse,
                                fp_stream_t stream) {
  if (!shape) return FP_ERR_NULL;
  if (shape->dtype != FP_BF16 && shape->dtype != FP_F32) return FP_ERR_DTYPE;
  if (shape->batch < 1 || shape->batch > kGrid || shape->n_q_heads < 1 || shape->n_kv_heads < 1 ||
      shape->n_kv_heads > kGrid || shape->seq_len < 1)
    return FP_ERR_SHAPE;
  if (shape->n_q_heads % shape->n_kv_heads != 0) return FP_ERR_SHAPE;
  if (shape->block_size != 64 && shape->block_size != 128) return FP_ERR_SHAPE;
  if (shape->head_dim != 64 && shape->head_dim != 128) return FP_ERR_SHAPE;
  if ((static_cast<long long>(shape->seq_len) + shape->block_size - 1) / shape->block_size > 4096)
    return FP_ERR_SHAPE;
  // (two products: batch * heads alone stays below 2^47, the whole may not)
  const long long heads = static_cast<long long>(shape->batch) * shape->n_q_heads;
  if (heads >= kRows || heads * shape->seq_len >= kRows) return FP_ERR_SHAPE;
  if (sinks < 0) return FP_ERR_PARAM;
  if (!q || !k || !v || !out) return FP_ERR_NULL;
  if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(out, 16) || !al(lse, 4)) return FP_ERR_ALIGN;
  const fp_status s = check_device();
  if (s != FP_OK) return s;
  Problem P = {};
  P.n_seqs = shape->batch;
  P.hq = shape->n_q_heads;
  P.hkv = shape->n_kv_heads;
  P.g = shape->n_q_heads / shape->n_kv_heads;
  P.d = shape->head_dim;
  P.max_q_len = shape->seq_len;
  P.total_q = shape->batch * shape->seq_len;
  P.k = k;
  P.v = v;
  set_window(&P, window, sinks);
  return run_attn(P, shape->dtype, false, q, out, lse, nullptr, stream);
}

FP_API fp_status fp_kv_write(const fp_kv_cache *cache, const fp_batch *batch, fp_dtype dtype,
                             const void *k, const void *v, fp_stream_t stream) {
  Problem P;
  const fp_status s = check_kv(cache, batch, dtype, k, v, &P);
  if (s != FP_OK || P.total_q == 0) return s;
  return cuda_status(launch_kv_write(P, cache->dtype, dtype, k, v,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

FP_API fp_status fp_kv_read(const fp_kv_cache *cache, const fp_batch *batch, fp_dtype dtype,
                            void *k, void *v, fp_stream_t stream) {
  Problem P;
  const fp_status s = check_kv(cache, batch, dtype, k, v, &P);
  if (s != FP_OK || P.total_q == 0) return s;
  return cuda_status(launch_kv_read(P, cache->dtype, dtype, k, v,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

FP_API size_t fp_paged_attn_workspace(const fp_kv_cache *cache, const fp_batch *batch,
                                      int n_q_heads) {
  Problem P;
  if (check_batch(cache, batch, n_q_heads, true, &P) != FP_OK) return 0;
  if (cache->dtype == FP_F32) return 0;
  const bool narrow = cache->dtype == FP_E4M3;
  return attn_few_takes(P) ? attn_few_ws_bytes(P, narrow) : attn_serve_ws_bytes(P, narrow);
}

FP_API fp_status fp_paged_attn(const fp_kv_cache *cache, const fp_batch *batch, int n_q_heads,
                               fp_dtype dtype, int window, int sinks, const void *q, void *out,
                               float *lse, void *ws, size_t ws_bytes, fp_stream_t stream) {
  Problem P;
  fp_status s = check_batch(cache, batch, n_q_heads, false, &P);
  if (s != FP_OK) return s;
  if (dtype != FP_BF16 && dtype != FP_F32) return FP_ERR_DTYPE;
  if (cache->dtype != FP_E4M3 && cache->dtype != int(dtype)) return FP_ERR_DTYPE;
  if (sinks < 0) return FP_ERR_PARAM;
  if (P.total_q == 0) return FP_OK;
  if (!q || !out) return FP_ERR_NULL;
  if (!al(q, 16) || !al(out, 16) || !al(lse, 4)) return FP_ERR_ALIGN;
  const size_t need =
      dtype == FP_F32 ? 0 : fp_paged_attn_workspace(cache, batch, n_q_heads);
  if (need > 0 && (!ws || !al(ws, 256) || ws_bytes < need)) return FP_ERR_WORKSPACE;
  if ((s = check_device()) != FP_OK) return s;
  set_window(&P, window, sinks);
  return run_attn(P, dtype, cache->dtype == FP_E4M3, q, out, lse, ws, stream);
}

FP_API fp_status fp_serve_last_device_status(fp_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return FP_ERR_CUDA;
  int *p = serve_status_ptr();
  if (!p) return FP_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FP_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return FP_ERR_CUDA;
  return static_cast<fp_status>(v);
}
