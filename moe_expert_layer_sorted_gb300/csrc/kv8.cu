// C entry points of the 8-bit key/value cache: argument checks, the handle and
// its workspace.
#include <new>

#include "kv8_internal.h"

using namespace moe;

namespace {

#include "kv_entry.h"

const char* check_desc(const moe_kv8_desc* d) {
  if (!d) return "desc is NULL";
  if (d->struct_size != sizeof(moe_kv8_desc)) return "struct_size is not sizeof(moe_kv8_desc)";
  if (d->dtype != MOE_KV_BF16 && d->dtype != MOE_KV_F16) return "dtype must be MOE_KV_BF16 or MOE_KV_F16";
  if (d->num_layers < 1) return "num_layers must be >= 1";
  if (d->kv_heads < 1 || d->kv_heads > 1024) return "kv_heads must be in 1..1024";
  if (d->head_dim != 64 && d->head_dim != 128) return "head_dim must be 64 or 128";
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)))
    return "page_size must be 16, 32, 64, 128 or 256";
  if (d->num_pages < 1 || d->num_pages > 0x7fffffff) return "num_pages must be in 1..2^31 - 1";
  if (d->reserved0 || d->reserved[0] || d->reserved[1]) return "reserved fields must be zero";
  return nullptr;
}

void set_sizes(Kv8* kv) {
  const moe_kv8_desc& d = kv->d;
  kv->block_bytes = d.head_dim == 64 ? Kv8Geom<64>::kBytes : Kv8Geom<128>::kBytes;
  kv->head_bytes = kv->block_bytes * (d.page_size / kKvBlock);
  kv->page_bytes = kv->head_bytes * d.kv_heads;
  kv->layer_bytes = kv->page_bytes * d.num_pages;
  kv->mass_layer = (int64_t)d.num_pages * d.kv_heads * d.page_size;
}

KvView view(const Kv8* kv, int layer) {
  const moe_kv8_desc& d = kv->d;
  KvView c;
  c.pages = static_cast<uint8_t*>(d.pages) + layer * kv->layer_bytes;
  c.bounds = nullptr;
  c.page_stride = kv->page_bytes;
  c.head_stride = kv->head_bytes;
  c.num_pages = d.num_pages;
  c.page_size = d.page_size;
  c.page_shift = 31 - __builtin_clz((unsigned)d.page_size);
  c.heads = d.kv_heads;
  return c;
}
float* mass_of(const Kv8* kv, int layer) { return kv->d.mass ? kv->d.mass + layer * kv->mass_layer : nullptr; }

void release(Kv8* kv) {
  if (kv->ws) cudaFree(kv->ws);
  if (kv->err_host) cudaFreeHost(const_cast<uint32_t*>(kv->err_host));
  if (kv->ev_done) cudaEventDestroy(kv->ev_done);
  delete kv;
}

}  // namespace

extern "C" moe_status moe_kv8_sizes(const moe_kv8_desc* desc, int64_t* pages, int64_t* mass) {
  return guarded([&]() -> moe_status {
    const char* why = check_desc(desc);
    if (why) return fail<Kv8>(nullptr, MOE_ERR_INVALID, why);
    Kv8 kv;
    kv.d = *desc;
    set_sizes(&kv);
    if (pages) *pages = kv.layer_bytes;
    if (mass) *mass = kv.mass_layer * 4;
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv8_create(const moe_kv8_desc* desc, moe_kv8_cache** out) {
  return guarded([&]() -> moe_status {
    if (!out) return fail<Kv8>(nullptr, MOE_ERR_INVALID, "out is NULL");
    *out = nullptr;
    const char* why = check_desc(desc);
    if (!why && !desc->pages) why = "pages is NULL";
    if (!why && (!aligned16(desc->pages) || !aligned16(desc->mass))) why = "pages and mass must be 16-byte aligned";
    if (why) return fail<Kv8>(nullptr, MOE_ERR_INVALID, why);
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || desc->device < 0 || desc->device >= ndev) {
      cudaGetLastError();
      return fail<Kv8>(nullptr, MOE_ERR_INVALID, "no such CUDA device");
    }
    DeviceScope ds(desc->device);
    if (!ds.ok) return fail<Kv8>(nullptr, MOE_ERR_CUDA, "cudaSetDevice failed");
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, desc->device);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, desc->device);
    if (major != 10 || minor != 3) return fail<Kv8>(nullptr, MOE_ERR_UNSUPPORTED, "the library targets sm_103a (GB300) only");
    Kv8* kv = new Kv8();
    kv->d = *desc;
    set_sizes(kv);
    cudaDeviceGetAttribute(&kv->sms, cudaDevAttrMultiProcessorCount, desc->device);
    cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&kv->ws), kv->workspace());
    if (e == cudaSuccess) e = cudaMemset(kv->counters(), 0, Kv8::kCounterBytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();  // the memset is done before any stream's first call
    void* word = nullptr;
    if (e == cudaSuccess) e = cudaHostAlloc(&word, 64, cudaHostAllocMapped);
    if (e == cudaSuccess) {
      kv->err_host = static_cast<volatile uint32_t*>(word);
      *kv->err_host = 0;
      e = cudaHostGetDevicePointer(reinterpret_cast<void**>(&kv->err_dev), word, 0);
    }
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&kv->ev_done, cudaEventDisableTiming);
    if (e != cudaSuccess) {
      cudaGetLastError();
      release(kv);
      return cuda_fail<Kv8>(nullptr, e, "key/value cache workspace");
    }
    *out = reinterpret_cast<moe_kv8_cache*>(kv);
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv8_destroy(moe_kv8_cache* h) {
  return guarded([&]() -> moe_status {
    Kv8* kv = reinterpret_cast<Kv8*>(h);
    if (!kv) return fail<Kv8>(nullptr, MOE_ERR_INVALID, "handle is NULL");
    if (kv->busy.exchange(1)) return MOE_ERR_STATE;  // another call is running: stays as it is
    DeviceScope ds(kv->d.device);
    if (kv->have_last && (kv->last_stream != kDefaultStream || cudaEventRecord(kv->ev_done, nullptr) == cudaSuccess))
      cudaEventSynchronize(kv->ev_done);
    const bool late = take_timeout(kv);
    release(kv);
    return late ? fail<Kv8>(nullptr, MOE_ERR_TIMEOUT, "a bounded wait of an attention gave up: the last results are suspect; the handle is gone")
                : MOE_OK;
  });
}

extern "C" moe_status moe_kv8_status(moe_kv8_cache* h) {
  return on_handle<Kv8>(h, [](Kv8*) { return MOE_OK; });
}

extern "C" moe_status moe_kv8_debug_fail_next_attention(moe_kv8_cache* h) {
  return on_handle<Kv8>(h, [](Kv8* kv) {
    kv->fail_next = true;
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv8_append(moe_kv8_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* k,
                                     const moe_kv_tensor* v, void* stream) {
  return on_handle<Kv8>(h, [&](Kv8* kv) -> moe_status {
    const char* why = check_batch(kv->d.num_layers, layer, batch);
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(k)) || (why = check_tensor(v))) return fail(kv, MOE_ERR_INVALID, why);
    const cudaError_t e =
        kv8_append(*kv, view(kv, layer), batch_of(batch), static_cast<const uint16_t*>(k->data), rows_of(k),
                   static_cast<const uint16_t*>(v->data), rows_of(v), mass_of(kv, layer), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv8_append");
  });
}

extern "C" moe_status moe_kv8_read(moe_kv8_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* k,
                                   const moe_kv_tensor* v, void* stream) {
  return on_handle<Kv8>(h, [&](Kv8* kv) -> moe_status {
    const char* why = check_batch(kv->d.num_layers, layer, batch);
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(k)) || (why = check_tensor(v))) return fail(kv, MOE_ERR_INVALID, why);
    const cudaError_t e = kv8_read(*kv, view(kv, layer), batch_of(batch), static_cast<uint16_t*>(k->data), rows_of(k),
                                   static_cast<uint16_t*>(v->data), rows_of(v), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv8_read");
  });
}

extern "C" moe_status moe_kv8_attention(moe_kv8_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* q,
                                        int q_heads, float scale, int causal, const moe_kv_tensor* out, float* lse,
                                        int weigh, void* stream) {
  return on_handle<Kv8>(h, [&](Kv8* kv) -> moe_status {
    const char* why = check_batch(kv->d.num_layers, layer, batch);
    if (!why && (q_heads < 1 || q_heads % kv->d.kv_heads)) why = "q_heads must be a positive multiple of kv_heads";
    if (!why && (causal != 0 && causal != 1)) why = "causal must be 0 or 1";
    if (!why && !(scale == scale && scale - scale == 0.0f)) why = "scale must be finite";
    if (!why && (weigh != 0 && weigh != 1)) why = "weigh must be 0 or 1";
    if (!why && weigh && !kv->d.mass) why = "the cache has no mass";
    if (!why && weigh && !lse) why = "weights are counted from lse: it must be given";
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(q)) || (why = check_tensor(out))) return fail(kv, MOE_ERR_INVALID, why);
    if (q->data == out->data) return fail(kv, MOE_ERR_INVALID, "q and out must not overlap");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const KvAttnArgs a{view(kv, layer), batch_of(batch), static_cast<const uint16_t*>(q->data),
                       static_cast<uint16_t*>(out->data), lse, rows_of(q), rows_of(out), q_heads, scale, causal, nullptr, 0};
    Order order;
    cudaError_t e = order_before(kv, s, order);
    if (e == cudaSuccess) e = kv8_attention(*kv, a, weigh ? mass_of(kv, layer) : nullptr, s);
    kv->fail_next = false;
    if (e == cudaSuccess) e = order_after(kv, s, order);
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv8_attention");
  });
}

extern "C" moe_status moe_kv8_evict(moe_kv8_cache* h, int layer, const moe_kv_batch* batch, int budget, int keep_first,
                                    int keep_last, int32_t* kept, void* stream) {
  return on_handle<Kv8>(h, [&](Kv8* kv) -> moe_status {
    const char* why = check_batch(kv->d.num_layers, layer, batch);
    if (!why && (budget < 1 || keep_first < 0 || keep_last < 0 || (int64_t)keep_first + keep_last > budget))
      why = "budget must be >= 1 and hold keep_first >= 0 and keep_last >= 0 tokens";
    if (!why && !kv->d.mass) why = "the cache has no mass";
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (budget > 1 << 30) return fail(kv, MOE_ERR_UNSUPPORTED, "budget above 2^30 tokens");
    if (batch->batch == 0) return MOE_OK;
    if (!kept) return fail(kv, MOE_ERR_INVALID, "kept is NULL");
    const Kv8EvictArgs a{view(kv, layer), batch_of(batch), mass_of(kv, layer), budget, keep_first, keep_last, kept};
    const cudaError_t e = kv8_evict(*kv, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv8_evict");
  });
}

extern "C" const char* moe_kv8_last_error(const moe_kv8_cache* kv) {
  return (kv ? reinterpret_cast<const Kv8*>(kv)->last_error : g_kv_error).c_str();
}
