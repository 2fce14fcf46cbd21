// Attention over the 8-bit cache: which kernel takes a call.
#include "kv8_internal.h"

using namespace moe;

cudaError_t moe::kv8_attention(Kv8& kv, const KvAttnArgs& a, cudaStream_t s) {
  return kv.d.dtype == MOE_KV_BF16 ? kv8_decode_bf16(kv, a, s) : kv8_decode_f16(kv, a, s);
}
