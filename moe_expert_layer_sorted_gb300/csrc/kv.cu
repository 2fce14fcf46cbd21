// C entry points of the 4-bit key/value cache: argument checks, the handle and
// its workspace, the order of calls on different streams.
#include <new>

#include "kv_internal.h"

using namespace moe;

namespace {

thread_local std::string g_kv_error;

moe_status fail(Kv* kv, moe_status s, const char* msg) {
  (kv ? kv->last_error : g_kv_error) = msg;
  return s;
}
moe_status cuda_fail(Kv* kv, cudaError_t e, const char* what) {
  (kv ? kv->last_error : g_kv_error) = std::string(what) + ": " + cudaGetErrorString(e);
  return e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA;
}

struct DeviceScope {  // makes `dev` current for a call and restores the caller's device
  int prev = -1;
  bool ok = true;
  explicit DeviceScope(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
    else prev = -1;  // nothing to restore
  }
  ~DeviceScope() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

struct Busy {  // one call at a time per handle
  Kv* kv;
  bool ok;
  explicit Busy(Kv* k) : kv(k), ok(k->busy.exchange(1) == 0) {}
  ~Busy() {
    if (ok) kv->busy.store(0);
  }
};

bool aligned16(const void* p) { return !(reinterpret_cast<uintptr_t>(p) & 15); }

const char* check_desc(const moe_kv_desc* d) {
  if (!d) return "desc is NULL";
  if (d->struct_size != sizeof(moe_kv_desc)) return "struct_size is not sizeof(moe_kv_desc)";
  if (d->dtype != MOE_KV_BF16 && d->dtype != MOE_KV_F16) return "dtype must be MOE_KV_BF16 or MOE_KV_F16";
  if (d->num_layers < 1) return "num_layers must be >= 1";
  if (d->kv_heads < 1 || d->kv_heads > 1024) return "kv_heads must be in 1..1024";
  if (d->head_dim != 64 && d->head_dim != 128) return "head_dim must be 64 or 128";
  if ((d->group_size != 32 && d->group_size != 64 && d->group_size != 128) || d->group_size > d->head_dim)
    return "group_size must be 32, 64 or 128 and divide head_dim";
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)))
    return "page_size must be 16, 32, 64, 128 or 256";
  if (d->num_pages < 1 || d->num_pages > 0x7fffffff) return "num_pages must be in 1..2^31 - 1";
  if (d->reserved[0] || d->reserved[1]) return "reserved fields must be zero";
  return nullptr;
}

void set_sizes(Kv* kv) {
  const moe_kv_desc& d = kv->d;
  kv->block_bytes = kKvBlock * (d.head_dim + 8 * (d.head_dim / d.group_size));
  kv->head_bytes = kv->block_bytes * (d.page_size / kKvBlock);
  kv->page_bytes = kv->head_bytes * d.kv_heads;
  kv->layer_bytes = kv->page_bytes * d.num_pages;
  kv->bounds_layer = (int64_t)d.num_pages * d.kv_heads * 2 * d.head_dim;
}

const char* check_batch(const Kv* kv, int layer, const moe_kv_batch* b) {
  if (layer < 0 || layer >= kv->d.num_layers) return "bad layer";
  if (!b || b->struct_size != sizeof(moe_kv_batch)) return "batch is NULL or its struct_size is not sizeof(moe_kv_batch)";
  if (b->batch < 0 || b->max_new < 0) return "batch and max_new must be >= 0";
  if (b->table_pages < 1 || b->table_stride < b->table_pages) return "table_pages must be >= 1 and table_stride >= table_pages";
  if (b->rows < 0 || (!b->starts && b->rows != (int64_t)b->batch * b->max_new)) return "rows must be batch * max_new without starts";
  if (b->batch > 0 && (!b->table || !b->lens)) return "table or lens is NULL";
  return nullptr;
}

const char* check_tensor(const moe_kv_tensor* t) {
  if (!t || !t->data) return "a tensor is NULL";
  if (!aligned16(t->data)) return "tensors must be 16-byte aligned";
  if ((t->batch_stride | t->row_stride | t->head_stride) & 7) return "strides must be multiples of 8 elements";
  return nullptr;
}

bool empty(const moe_kv_batch* b) { return b->batch == 0 || b->max_new == 0 || b->rows == 0; }

KvView view(const Kv* kv, int layer) {
  const moe_kv_desc& d = kv->d;
  KvView c;
  c.pages = static_cast<uint8_t*>(d.pages) + layer * kv->layer_bytes;
  c.bounds = d.bounds ? static_cast<uint16_t*>(d.bounds) + layer * kv->bounds_layer : nullptr;
  c.page_stride = kv->page_bytes;
  c.head_stride = kv->head_bytes;
  c.num_pages = d.num_pages;
  c.page_size = d.page_size;
  c.page_shift = 31 - __builtin_clz((unsigned)d.page_size);
  c.heads = d.kv_heads;
  return c;
}
KvBatch batch_of(const moe_kv_batch* b) {
  return {b->table, b->lens, b->starts, b->table_stride, b->rows, b->batch, b->table_pages, b->max_new};
}
KvRows rows_of(const moe_kv_tensor* t) { return {t->batch_stride, t->row_stride, t->head_stride}; }

// Calls that share the workspace follow one another across streams; inside a
// capture the graph's own edges order its nodes.  A stream may be gone by the
// next call, so its work is recorded at once, but for the default stream, which
// stays and is never captured: that one is recorded when another stream follows.
struct Order {
  bool capturing = false;
  unsigned long long stream = 0;
};
cudaError_t order_before(Kv* kv, cudaStream_t s, Order& o) {
  cudaError_t e = stream_identity(s, o.capturing, o.stream);
  if (e != cudaSuccess || o.capturing || !kv->have_last || kv->last_stream == o.stream) return e;
  if (kv->last_stream == kDefaultStream && (e = cudaEventRecord(kv->ev_done, nullptr)) != cudaSuccess) return e;
  return cudaStreamWaitEvent(s, kv->ev_done, 0);
}
cudaError_t order_after(Kv* kv, cudaStream_t s, const Order& o) {
  if (o.capturing) return cudaSuccess;
  const cudaError_t e = o.stream != kDefaultStream ? cudaEventRecord(kv->ev_done, s) : cudaSuccess;
  if (e == cudaSuccess) {
    kv->last_stream = o.stream;
    kv->have_last = true;
  }
  return e;
}

void release(Kv* kv) {
  if (kv->ws) cudaFree(kv->ws);
  if (kv->err_host) cudaFreeHost(const_cast<uint32_t*>(kv->err_host));
  if (kv->ev_done) cudaEventDestroy(kv->ev_done);
  delete kv;
}

// Runs f with no C++ exception leaving the library.
template <typename F>
moe_status guarded(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return MOE_ERR_OOM;  // the only exceptions here are failed host allocations
  }
}

// Whether a kernel's bounded wait gave up since this was last asked (for every wait of a launch
// counts its own CTA's state alone, nothing on the device needs to be put right).
bool take_timeout(Kv* kv) {
  if (!*kv->err_host) return false;
  *kv->err_host = 0;
  return true;
}
constexpr char kTimeoutMsg[] =
    "a bounded wait of an attention gave up: results of the calls since the last one that was reported as done are suspect; "
    "this call did nothing";

// The frame of a call on a handle: one at a time, its device current, no timeout unreported.
template <typename F>
moe_status on_handle(moe_kv_cache* h, F&& f) noexcept {
  return guarded([&]() -> moe_status {
    Kv* kv = reinterpret_cast<Kv*>(h);
    if (!kv) return fail(nullptr, MOE_ERR_INVALID, "handle is NULL");
    Busy busy(kv);
    if (!busy.ok) return MOE_ERR_STATE;  // the text is the other thread's to write
    DeviceScope ds(kv->d.device);
    if (!ds.ok) return fail(kv, MOE_ERR_CUDA, "cudaSetDevice failed");
    if (take_timeout(kv)) return fail(kv, MOE_ERR_TIMEOUT, kTimeoutMsg);
    return f(kv);
  });
}

}  // namespace

extern "C" moe_status moe_kv_sizes(const moe_kv_desc* desc, int64_t* pages, int64_t* bounds) {
  return guarded([&]() -> moe_status {
    const char* why = check_desc(desc);
    if (why) return fail(nullptr, MOE_ERR_INVALID, why);
    Kv kv;
    kv.d = *desc;
    set_sizes(&kv);
    if (pages) *pages = kv.layer_bytes;
    if (bounds) *bounds = kv.bounds_layer * 2;
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv_create(const moe_kv_desc* desc, moe_kv_cache** out) {
  return guarded([&]() -> moe_status {
    if (!out) return fail(nullptr, MOE_ERR_INVALID, "out is NULL");
    *out = nullptr;
    const char* why = check_desc(desc);
    if (!why && !desc->pages) why = "pages is NULL";
    if (!why && (!aligned16(desc->pages) || !aligned16(desc->bounds))) why = "pages and bounds must be 16-byte aligned";
    if (why) return fail(nullptr, MOE_ERR_INVALID, why);
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || desc->device < 0 || desc->device >= ndev) {
      cudaGetLastError();
      return fail(nullptr, MOE_ERR_INVALID, "no such CUDA device");
    }
    DeviceScope ds(desc->device);
    if (!ds.ok) return fail(nullptr, MOE_ERR_CUDA, "cudaSetDevice failed");
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, desc->device);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, desc->device);
    if (major != 10 || minor != 3) return fail(nullptr, MOE_ERR_UNSUPPORTED, "the library targets sm_103a (GB300) only");
    Kv* kv = new Kv();
    kv->d = *desc;
    set_sizes(kv);
    cudaDeviceGetAttribute(&kv->sms, cudaDevAttrMultiProcessorCount, desc->device);
    cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&kv->ws), Kv::kWorkspace);
    if (e == cudaSuccess) e = cudaMemset(kv->counters(), 0, Kv::kCounterBytes);
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
      return cuda_fail(nullptr, e, "key/value cache workspace");
    }
    *out = reinterpret_cast<moe_kv_cache*>(kv);
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv_destroy(moe_kv_cache* h) {
  return guarded([&]() -> moe_status {
    Kv* kv = reinterpret_cast<Kv*>(h);
    if (!kv) return fail(nullptr, MOE_ERR_INVALID, "handle is NULL");
    if (kv->busy.exchange(1)) return MOE_ERR_STATE;  // another call is running: stays as it is
    DeviceScope ds(kv->d.device);
    if (kv->have_last && (kv->last_stream != kDefaultStream || cudaEventRecord(kv->ev_done, nullptr) == cudaSuccess))
      cudaEventSynchronize(kv->ev_done);
    const bool late = take_timeout(kv);
    release(kv);
    return late ? fail(nullptr, MOE_ERR_TIMEOUT, "a bounded wait of an attention gave up: the last results are suspect; the handle is gone")
                : MOE_OK;
  });
}

extern "C" moe_status moe_kv_status(moe_kv_cache* h) {
  return on_handle(h, [](Kv*) { return MOE_OK; });
}

extern "C" moe_status moe_kv_debug_fail_next_attention(moe_kv_cache* h) {
  return on_handle(h, [](Kv* kv) {
    kv->fail_next = true;
    return MOE_OK;
  });
}

extern "C" moe_status moe_kv_append(moe_kv_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* k,
                                    const moe_kv_tensor* v, void* stream) {
  return on_handle(h, [&](Kv* kv) -> moe_status {
    const char* why = check_batch(kv, layer, batch);
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(k)) || (why = check_tensor(v))) return fail(kv, MOE_ERR_INVALID, why);
    const cudaError_t e =
        kv_append(*kv, view(kv, layer), batch_of(batch), static_cast<const uint16_t*>(k->data), rows_of(k),
                  static_cast<const uint16_t*>(v->data), rows_of(v), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv_append");
  });
}

extern "C" moe_status moe_kv_read(moe_kv_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* k,
                                  const moe_kv_tensor* v, void* stream) {
  return on_handle(h, [&](Kv* kv) -> moe_status {
    const char* why = check_batch(kv, layer, batch);
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(k)) || (why = check_tensor(v))) return fail(kv, MOE_ERR_INVALID, why);
    const cudaError_t e = kv_read(*kv, view(kv, layer), batch_of(batch), static_cast<uint16_t*>(k->data), rows_of(k),
                                  static_cast<uint16_t*>(v->data), rows_of(v), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv_read");
  });
}

extern "C" moe_status moe_kv_attention(moe_kv_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* q,
                                       int q_heads, float scale, int causal, const moe_kv_tensor* out, float* lse,
                                       const int32_t* pages, int budget, void* stream) {
  return on_handle(h, [&](Kv* kv) -> moe_status {
    const char* why = check_batch(kv, layer, batch);
    if (!why && (q_heads < 1 || q_heads % kv->d.kv_heads)) why = "q_heads must be a positive multiple of kv_heads";
    if (!why && (causal != 0 && causal != 1)) why = "causal must be 0 or 1";
    if (!why && pages && budget < 1) why = "budget must be >= 1 with pages";
    if (!why && !(scale == scale && scale - scale == 0.0f)) why = "scale must be finite";
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (pages && (int64_t)budget * (kv->d.page_size / kKvBlock) > 0x7fffff00)  // blocks are counted in 32 bits
      return fail(kv, MOE_ERR_UNSUPPORTED, "budget * page_size above 2^35 tokens");
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(q)) || (why = check_tensor(out))) return fail(kv, MOE_ERR_INVALID, why);
    if (q->data == out->data) return fail(kv, MOE_ERR_INVALID, "q and out must not overlap");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    KvAttnArgs a{view(kv, layer), batch_of(batch), static_cast<const uint16_t*>(q->data),
                 static_cast<uint16_t*>(out->data), lse, rows_of(q), rows_of(out), q_heads, scale, causal,
                 pages, pages ? budget : 0};
    Order order;
    cudaError_t e = order_before(kv, s, order);
    if (e == cudaSuccess) e = kv_attention(*kv, a, s);
    kv->fail_next = false;
    if (e == cudaSuccess) e = order_after(kv, s, order);
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv_attention");
  });
}

extern "C" moe_status moe_kv_select(moe_kv_cache* h, int layer, const moe_kv_batch* batch, const moe_kv_tensor* q,
                                    int q_heads, int budget, int keep_first, int keep_last, int32_t* pages_out,
                                    void* stream) {
  return on_handle(h, [&](Kv* kv) -> moe_status {
    const char* why = check_batch(kv, layer, batch);
    if (!why && (q_heads < 1 || q_heads % kv->d.kv_heads)) why = "q_heads must be a positive multiple of kv_heads";
    if (!why && (budget < 1 || keep_first < 0 || keep_last < 1 || (int64_t)keep_first + keep_last > budget))
      why = "budget must hold keep_first >= 0 and keep_last >= 1 pages";
    if (!why && !kv->d.bounds) why = "the cache has no bounds";
    if (!why && (int64_t)batch->table_pages * kv->d.kv_heads * 4 > (int64_t)Kv::kScoreBytes)
      return fail(kv, MOE_ERR_UNSUPPORTED, "kv_heads * table_pages above the selection's workspace (4,194,304 scores)");
    if (why) return fail(kv, MOE_ERR_INVALID, why);
    if (empty(batch)) return MOE_OK;
    if ((why = check_tensor(q))) return fail(kv, MOE_ERR_INVALID, why);
    if (!pages_out) return fail(kv, MOE_ERR_INVALID, "pages_out is NULL");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    KvSelectArgs a{view(kv, layer), batch_of(batch), static_cast<const uint16_t*>(q->data), rows_of(q), q_heads,
                   budget, keep_first, keep_last, pages_out};
    Order order;
    const bool shares = batch->table_pages > kKvSelOwn;  // otherwise the workspace is not used
    cudaError_t e = shares ? order_before(kv, s, order) : cudaSuccess;
    if (e == cudaSuccess) e = kv_select(*kv, a, s);
    if (e == cudaSuccess && shares) e = order_after(kv, s, order);
    return e == cudaSuccess ? MOE_OK : cuda_fail(kv, e, "moe_kv_select");
  });
}

extern "C" const char* moe_kv_last_error(const moe_kv_cache* kv) {
  return (kv ? reinterpret_cast<const Kv*>(kv)->last_error : g_kv_error).c_str();
}
