// Attention over the 4-bit cache: which kernel takes a call.
#include "kv_internal.h"

using namespace moe;

// By columns (rows of a sequence times the query heads that share a kv head).  The decode
// kernel reads the cache once per 16 columns (8 where there are no more), the prompt kernel
// once per 256 but turns every code into shared memory first.  Measured, both kernels, us
// (8 kv heads of 128 channels, bf16; decode / prompt):
//     columns                       16          32          64         128
//     1 sequence of 2,048       14.5 / 19   14.9 / 21   23 / 21     25 / 21
//     1 of 131,072                61 / 115   106 / 115  193 / 115   369 / 117
//     16 of 4,096                 41 / 60     66 / 60   117 / 60    219 / 62
//     64 of 2,048                 80 / 135   138 / 135  260 / 137   498 / 143
// so 32 is the last count that the decode kernel takes.  Rows with pages of their own have
// no tiles to share and always go there.
cudaError_t moe::kv_attention(Kv& kv, const KvAttnArgs& a, cudaStream_t s) {
  const bool bf16 = kv.d.dtype == MOE_KV_BF16;
  if (a.sel || (int64_t)a.b.max_new * (a.q_heads / a.c.heads) <= 32)
    return bf16 ? kv_decode_bf16(kv, a, s) : kv_decode_f16(kv, a, s);
  return bf16 ? kv_prompt_bf16(kv, a, s) : kv_prompt_f16(kv, a, s);
}
