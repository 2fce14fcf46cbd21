// Attention over the 4-bit cache: which kernel takes a call.
#include "kv_internal.h"

using namespace moe;

cudaError_t moe::kv_attention(Kv& kv, const KvAttnArgs& a, cudaStream_t s) {
  const bool bf16 = kv.d.dtype == MOE_KV_BF16;
  if (a.sel || (int64_t)a.b.max_new * (a.q_heads / a.c.heads) <= 32)
    return bf16 ? kv_decode_bf16(kv, a, s) : kv_decode_f16(kv, a, s);
  return bf16 ? kv_prompt_bf16(kv, a, s) : kv_prompt_f16(kv, a, s);
}
