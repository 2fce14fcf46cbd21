// The launchers that csrc/kv.cu calls, without kernels: each call goes to the log of fake_cuda.cpp.
#include "kv_internal.h"

void say(const char* what, cudaStream_t s);

// what a kernel's wait that gave up leaves behind
extern "C" void fake_raise(moe_kv_cache* h) { *reinterpret_cast<moe::Kv*>(h)->err_host = 1; }

namespace moe {

cudaError_t kv_append(const Kv&, const KvView&, const KvBatch&, const uint16_t*, const KvRows&, const uint16_t*,
                      const KvRows&, cudaStream_t s) {
  say("append", s);
  return cudaSuccess;
}
cudaError_t kv_read(const Kv&, const KvView&, const KvBatch&, uint16_t*, const KvRows&, uint16_t*, const KvRows&,
                    cudaStream_t s) {
  say("read", s);
  return cudaSuccess;
}
cudaError_t kv_attention(Kv&, const KvAttnArgs&, cudaStream_t s) {
  say("attention", s);
  return cudaSuccess;
}
cudaError_t kv_select(Kv&, const KvSelectArgs&, cudaStream_t s) {
  say("select", s);
  return cudaSuccess;
}

}  // namespace moe
