// What the C entry points of the key/value caches share: argument checks, one call at a time on
// a handle, the order of calls on different streams, errors.  Included into an anonymous namespace.
// A handle K has d (its descriptor, with device and num_layers), busy, last_error, err_host,
// ev_done, have_last and last_stream.
#pragma once

thread_local std::string g_kv_error;

template <typename K>
moe_status fail(K* kv, moe_status s, const char* msg) {
  (kv ? kv->last_error : g_kv_error) = msg;
  return s;
}
template <typename K>
moe_status cuda_fail(K* kv, cudaError_t e, const char* what) {
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

template <typename K>
struct Busy {  // one call at a time per handle
  K* kv;
  bool ok;
  explicit Busy(K* k) : kv(k), ok(k->busy.exchange(1) == 0) {}
  ~Busy() {
    if (ok) kv->busy.store(0);
  }
};

bool aligned16(const void* p) { return !(reinterpret_cast<uintptr_t>(p) & 15); }

const char* check_batch(int num_layers, int layer, const moe_kv_batch* b) {
  if (layer < 0 || layer >= num_layers) return "bad layer";
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
template <typename K>
cudaError_t order_before(K* kv, cudaStream_t s, Order& o) {
  cudaError_t e = stream_identity(s, o.capturing, o.stream);
  if (e != cudaSuccess || o.capturing || !kv->have_last || kv->last_stream == o.stream) return e;
  if (kv->last_stream == kDefaultStream && (e = cudaEventRecord(kv->ev_done, nullptr)) != cudaSuccess) return e;
  return cudaStreamWaitEvent(s, kv->ev_done, 0);
}
template <typename K>
cudaError_t order_after(K* kv, cudaStream_t s, const Order& o) {
  if (o.capturing) return cudaSuccess;
  const cudaError_t e = o.stream != kDefaultStream ? cudaEventRecord(kv->ev_done, s) : cudaSuccess;
  if (e == cudaSuccess) {
    kv->last_stream = o.stream;
    kv->have_last = true;
  }
  return e;
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
template <typename K>
bool take_timeout(K* kv) {
  if (!*kv->err_host) return false;
  *kv->err_host = 0;
  return true;
}
constexpr char kTimeoutMsg[] =
    "a bounded wait of an attention gave up: results of the calls since the last one that was reported as done are suspect; "
    "this call did nothing";

// The frame of a call on a handle: one at a time, its device current, no timeout unreported.
template <typename K, typename H, typename F>
moe_status on_handle(H* h, F&& f) noexcept {
  return guarded([&]() -> moe_status {
    K* kv = reinterpret_cast<K*>(h);
    if (!kv) return fail<K>(nullptr, MOE_ERR_INVALID, "handle is NULL");
    Busy busy(kv);
    if (!busy.ok) return MOE_ERR_STATE;  // the text is the other thread's to write
    DeviceScope ds(kv->d.device);
    if (!ds.ok) return fail(kv, MOE_ERR_CUDA, "cudaSetDevice failed");
    if (take_timeout(kv)) return fail(kv, MOE_ERR_TIMEOUT, kTimeoutMsg);
    return f(kv);
  });
}
