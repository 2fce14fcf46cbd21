// The launchers that csrc/kv8.cu calls, without kernels: each call goes to the log of fake_cuda.cpp.
#include "kv8_internal.h"

void say(const char* what, cudaStream_t s);

// what a kernel's wait that gave up leaves behind
extern "C" void fake_raise(moe_kv8_cache* h) { *reinterpret_cast<moe::Kv8*>(h)->err_host = 1; }

namespace moe {

cudaError_t kv8_append(const Kv8&, const KvView&, const KvBatch&, const uint16_t*, const KvRows&, const uint16_t*, const KvRows&,
                       float* mass, cudaStream_t s) {
  say(mass ? "append+mass" : "append", s);
  return cudaSuccess;
}
cudaError_t kv8_read(const Kv8&, const KvView&, const KvBatch&, uint16_t*, const KvRows&, uint16_t*, const KvRows&, cudaStream_t s) {
  say("read", s);
  return cudaSuccess;
}
cudaError_t kv8_attention(Kv8& kv, const KvAttnArgs&, float* mass, cudaStream_t s) {
  say(mass ? "weigh" : kv.fail_next ? "attention that fails" : "attention", s);
  return cudaSuccess;
}
cudaError_t kv8_evict(const Kv8&, const Kv8EvictArgs&, cudaStream_t s) {
  say("evict", s);
  return cudaSuccess;
}

}  // namespace moe
