// Host side of the paged KV cache's entry points (dlm.h): argument checks
// and launches.  They take no context; the device error word is one per
// device, compiled into the library.
#include <climits>
#include <mutex>

#include "kernels.h"

using namespace dlm;

// the error word, and where a check puts what it took from it
static __device__ int g_paged_err[2];

namespace {

// A CUDA error is returned, and not left behind for the caller's next CUDA call to find.
int cuda_problem(const char* where, cudaError_t e) {
  cudaGetLastError();
  return api_cuda_fail(where, e);
}

// One step, so that what a kernel of another stream records meanwhile is either
// taken or stays.
__global__ void take_error_kernel(int* err) { err[1] = atomicExch(err, 0); }

struct PagedDevice {
  int* err = nullptr;
  std::mutex check;   // err[1] is one check's at a time
  int num_sms = 0;
};
PagedDevice g_paged[kMaxDeviceOnce];
DeviceOnce g_paged_once;

// the current device's state in *out, looked up on first use; a DLM status
int paged_device(PagedDevice** out, int* device = nullptr) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess)
    return cuda_problem("paged: cudaGetDevice", e);
  if (dev < 0 || dev >= kMaxDeviceOnce) return api_fail(DLM_EINVAL, "paged: device index out of range");
  PagedDevice& d = g_paged[dev];
  const cudaError_t e = g_paged_once.get([&d, dev] {
    void* p = nullptr;
    const cudaError_t status = cudaGetSymbolAddress(&p, g_paged_err);
    if (status != cudaSuccess) return status;
    d.err = static_cast<int*>(p);
    return cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
  });
  if (e != cudaSuccess) return cuda_problem("paged: device set-up", e);
  *out = &d;
  if (device != nullptr) *device = dev;
  return DLM_OK;
}

// device memory of `device`?
bool on_device(const void* p, int device) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return (at.type == cudaMemoryTypeDevice && at.device == device) ||
         at.type == cudaMemoryTypeManaged;
}

// log2 of a page size, or -1
int page_shift(int page_size) {
  for (int s = 3; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
const char* const kUnaligned = "paged: an array is not aligned to its element type";

// the checks of a cache that need no device
const char* cache_problem(const dlm_paged_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return "paged: NULL cache";
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return "paged: the cache is not 16-byte aligned";
  if (c->dtype != DLM_BF16 && c->dtype != DLM_F32) return "paged: dtype must be DLM_F32 or DLM_BF16";
  if (c->head_dim != 64 && c->head_dim != 128 && !(c->dtype == DLM_F32 && c->head_dim == 32))
    return "paged: head_dim must be 64 or 128 (32 too for DLM_F32)";
  if (page_shift(c->page_size) < 0) return "paged: page_size must be 8, 16, 32, 64, 128 or 256";
  if (c->n_kv_heads < 1 || c->n_pages < 1) return "paged: need n_kv_heads and n_pages >= 1";
  if (c->n_kv_heads > 65536 || ((long long)c->n_pages + 1) * c->n_kv_heads > INT_MAX)
    return "paged: (n_pages + 1) * n_kv_heads exceeds 2^31 - 1";
  return nullptr;
}

const char* heads_problem(const dlm_paged_cache* c, int n_heads) {
  if (n_heads < 1 || n_heads % c->n_kv_heads != 0 || n_heads / c->n_kv_heads > 128)
    return "paged_attention: n_heads must be a multiple of n_kv_heads, at most 128 times it";
  return nullptr;
}

size_t work_of(const dlm_paged_cache* c, const PagedDevice* d) {
  return c->dtype == DLM_BF16 ? paged_attention_work(c->head_dim, d->num_sms)
                              : paged_attention_f32_work(c->head_dim, d->num_sms);
}

PagedKV kv_of(const dlm_paged_cache* c) {
  return PagedKV{c->k, c->v, c->n_pages, page_shift(c->page_size), c->n_kv_heads, c->head_dim,
                 c->dtype == DLM_BF16 ? 2 : 4};
}

// rows of `width` elements, `stride` apart: 16-byte pieces, no overlap, and a
// stride that a tensor map can hold (below 2^40 bytes)
const char* rows_problem(const void* p, int64_t stride, int64_t width, int esize) {
  if (!aligned(p, 16)) return "paged: rows are not 16-byte aligned";
  if (stride < width || stride >= (1ll << 40) / esize || stride * esize % 16 != 0)
    return "paged: a row stride must be a multiple of 16 bytes, at least the row and below 2^40 bytes";
  return nullptr;
}

}  // namespace

extern "C" {

int dlm_paged_resize(const int32_t* cur_lens, const int32_t* new_lens, int32_t* out_lens,
                     int batch, int32_t* block_table, int table_width, int page_size,
                     int32_t* free_pages, int n_pages, const int32_t* n_free_in,
                     int32_t* n_free_out, int32_t* cu_new, int64_t* slots, int max_new,
                     void* stream) {
  api_clear_error();
  if (!cur_lens || !new_lens || !out_lens || !block_table || !free_pages || !n_free_in ||
      !n_free_out || !cu_new || (max_new > 0 && !slots))
    return api_fail(DLM_EINVAL, "paged_resize: NULL pointer argument");
  if (batch < 1 || batch > kPagedMaxBatch || table_width < 1 || n_pages < 1 || max_new < 0 ||
      max_new > (1 << 30) || page_shift(page_size) < 0)
    return api_fail(DLM_EINVAL,
                    "paged_resize: need 1 <= batch <= 4096, table_width and n_pages >= 1, "
                    "0 <= max_new <= 2^30 and a page_size of 8, 16, 32, 64, 128 or 256");
  for (const void* p : {(const void*)cur_lens, (const void*)new_lens, (const void*)out_lens,
                        (const void*)block_table, (const void*)free_pages, (const void*)n_free_in,
                        (const void*)n_free_out, (const void*)cu_new})
    if (!aligned(p, 4)) return api_fail(DLM_EINVAL, kUnaligned);
  if (!aligned(slots, 8)) return api_fail(DLM_EINVAL, kUnaligned);
  PagedDevice* d = nullptr;
  int dev = 0;
  if (int rc = paged_device(&d, &dev)) return rc;
  for (const void* p : {(const void*)cur_lens, (const void*)new_lens, (const void*)out_lens,
                        (const void*)block_table, (const void*)free_pages, (const void*)n_free_in,
                        (const void*)n_free_out, (const void*)cu_new, (const void*)slots})
    if (p != nullptr && !on_device(p, dev))
      return api_fail(DLM_EINVAL, "paged_resize: a pointer is not memory of the current device");
  const PagedResize a{cur_lens, new_lens, out_lens, batch, block_table, table_width,
                      page_shift(page_size), free_pages, n_pages, n_free_in, n_free_out, cu_new,
                      slots, max_new, d->err};
  if (cudaError_t e = paged_resize(a, (cudaStream_t)stream); e != cudaSuccess)
    return cuda_problem("paged_resize launch", e);
  return DLM_OK;
}

int dlm_paged_kv_write(const dlm_paged_cache* cache, const void* k, const void* v,
                       int64_t k_stride, int64_t v_stride, const int64_t* slots, int n_tokens,
                       void* stream) {
  api_clear_error();
  if (const char* why = cache_problem(cache)) return api_fail(DLM_EINVAL, why);
  if (n_tokens < 0) return api_fail(DLM_EINVAL, "paged_kv_write: n_tokens < 0");
  if (n_tokens == 0) return DLM_OK;
  if (!k || !v || !slots) return api_fail(DLM_EINVAL, "paged_kv_write: NULL pointer argument");
  if (!aligned(slots, 8)) return api_fail(DLM_EINVAL, kUnaligned);
  const PagedKV c = kv_of(cache);
  const int64_t row = (int64_t)c.Hkv * c.Dh;
  if (const char* why = rows_problem(k, k_stride, row, c.esize))
    return api_fail(DLM_EINVAL, why);
  if (const char* why = rows_problem(v, v_stride, row, c.esize))
    return api_fail(DLM_EINVAL, why);
  PagedDevice* d = nullptr;
  int dev = 0;
  if (int rc = paged_device(&d, &dev)) return rc;
  for (const void* p : {k, v, (const void*)slots, (const void*)c.k, (const void*)c.v})
    if (!on_device(p, dev))
      return api_fail(DLM_EINVAL, "paged_kv_write: a pointer is not memory of the current device");
  cudaError_t e =
      paged_kv_write(c, k, v, k_stride, v_stride, slots, n_tokens, d->err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_problem("paged_kv_write launch", e);
  return DLM_OK;
}

int dlm_paged_attention_workspace(const dlm_paged_cache* cache, int n_heads, size_t* bytes) {
  api_clear_error();
  if (bytes == nullptr) return api_fail(DLM_EINVAL, "paged_attention_workspace: NULL pointer argument");
  if (const char* why = cache_problem(cache)) return api_fail(DLM_EINVAL, why);
  if (const char* why = heads_problem(cache, n_heads)) return api_fail(DLM_EINVAL, why);
  PagedDevice* d = nullptr;
  if (int rc = paged_device(&d)) return rc;
  *bytes = work_of(cache, d);
  return DLM_OK;
}

int dlm_paged_attention(const dlm_paged_cache* cache, const void* q, int64_t q_stride, void* o,
                        int64_t o_stride, float* lse, const int32_t* cu_q,
                        const int32_t* ctx_lens, const int32_t* block_table, int table_width,
                        int batch, int n_tokens, int n_heads, int mask_block, float scale,
                        void* workspace, size_t workspace_bytes, void* stream) {
  api_clear_error();
  if (const char* why = cache_problem(cache)) return api_fail(DLM_EINVAL, why);
  if (const char* why = heads_problem(cache, n_heads)) return api_fail(DLM_EINVAL, why);
  if (n_tokens < 0 || batch < 1 || batch > kPagedMaxBatch || table_width < 1 || mask_block < 0 ||
      !(scale >= 0.f) || !(scale <= 1e30f))
    return api_fail(DLM_EINVAL,
                    "paged_attention: need n_tokens >= 0, 1 <= batch <= 4096, table_width >= 1, "
                    "mask_block >= 0 and 0 <= scale <= 1e30");
  if (n_tokens == 0) return DLM_OK;
  if (!q || !o || !cu_q || !ctx_lens || !block_table || !workspace)
    return api_fail(DLM_EINVAL, "paged_attention: NULL pointer argument");
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(ctx_lens, 4) || !aligned(block_table, 4))
    return api_fail(DLM_EINVAL, kUnaligned);
  if (!aligned(workspace, 256))
    return api_fail(DLM_EINVAL, "paged_attention: the workspace is not 256-byte aligned");
  const PagedKV c = kv_of(cache);
  const int64_t row = (int64_t)n_heads * c.Dh;
  if (const char* why = rows_problem(q, q_stride, row, c.esize))
    return api_fail(DLM_EINVAL, why);
  if (const char* why = rows_problem(o, o_stride, row, c.esize))
    return api_fail(DLM_EINVAL, why);
  if ((long long)n_tokens * n_heads > INT_MAX)
    return api_fail(DLM_EINVAL, "paged_attention: n_tokens * n_heads exceeds 2^31 - 1");
  if (workspace_bytes < 4096)   // less than any cache needs
    return api_fail(DLM_EINVAL, "paged_attention: the workspace is too small");
  PagedDevice* d = nullptr;
  int dev = 0;
  if (int rc = paged_device(&d, &dev)) return rc;
  if (workspace_bytes < work_of(cache, d))
    return api_fail(DLM_EINVAL, "paged_attention: the workspace is too small");
  for (const void* p : {q, (const void*)o, (const void*)lse, (const void*)cu_q,
                        (const void*)ctx_lens, (const void*)block_table, (const void*)workspace,
                        (const void*)c.k, (const void*)c.v})
    if (p != nullptr && !on_device(p, dev))
      return api_fail(DLM_EINVAL, "paged_attention: a pointer is not memory of the current device");
  PagedAttn a{c, q, q_stride, o, o_stride, lse, cu_q, ctx_lens, block_table, table_width, batch,
              n_tokens, n_heads, mask_block,
              scale > 0.f ? scale : (float)(1.0 / sqrt((double)c.Dh)), workspace, d->err};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = c.esize == 2 ? paged_attention_tc(a, d->num_sms, st)
                                : paged_attention_f32(a, d->num_sms, st);
  if (e != cudaSuccess)
    return cuda_problem("paged_attention launch", e);
  return DLM_OK;
}

int dlm_paged_check(void* stream) {
  api_clear_error();
  PagedDevice* d = nullptr;
  int dev = 0;
  if (int rc = paged_device(&d, &dev)) return rc;
  // (to wait for a stream that is being captured would end the capture)
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &capture); e != cudaSuccess)
    return cuda_problem("paged_check: cudaStreamIsCapturing", e);
  if (capture != cudaStreamCaptureStatusNone)
    return api_fail(DLM_EINVAL, "paged_check: the stream is being captured");
  if (cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream); e != cudaSuccess)
    return cuda_problem("paged_check: cudaStreamSynchronize", e);
  // in the caller's stream: the legacy stream would wait for work that is not its
  int word = 0;
  cudaError_t e;
  {
    std::lock_guard<std::mutex> one(d->check);
    take_error_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(d->err);
    e = cudaGetLastError();
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(&word, d->err + 1, sizeof(int), cudaMemcpyDeviceToHost,
                          (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  }
  if (e != cudaSuccess) return cuda_problem("paged_check: take the error word", e);
  if (word == 0) return DLM_OK;
  return api_fail(word, word == DLM_ETIMEOUT ? "paged: device wait timed out"
                                             : "paged: device index check failed");
}

}  // extern "C"
