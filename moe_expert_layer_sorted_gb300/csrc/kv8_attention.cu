// Attention over the 8-bit cache: which kernel takes a call.
#include "kv8_internal.h"

using namespace moe;

// By columns (rows of a sequence times the query heads that share a kv head).  The single-token
// kernel reads the cache once per 16 columns (8 where there are no more), the prompt kernel
// once per 256 but turns every code into shared memory first.
cudaError_t moe::kv8_attention(Kv8& kv, const KvAttnArgs& a, cudaStream_t s) {
  const bool bf16 = kv.d.dtype == MOE_KV_BF16;
  if ((int64_t)a.b.max_new * (a.q_heads / a.c.heads) <= 32) return bf16 ? kv8_decode_bf16(kv, a, s) : kv8_decode_f16(kv, a, s);
  return bf16 ? kv8_prompt_bf16(kv, a, s) : kv8_prompt_f16(kv, a, s);
}
