// Attention over the 8-bit cache: which kernels take a call.
#include "kv8_internal.h"

using namespace moe;

// By columns (rows of a sequence times the query heads that share a kv head).  The single-token
// kernel reads the cache once per 16 columns (8 where there are no more), the prompt kernel
// once per 256 but turns every code into shared memory first.
//
// Weights: the single-token kernel leaves its scores behind where the workspace holds them, four
// bytes a token and column beside the 256 that it reads; otherwise they are made again from the keys.
cudaError_t moe::kv8_attention(Kv8& kv, const KvAttnArgs& a, float* mass, cudaStream_t s) {
  const bool bf16 = kv.d.dtype == MOE_KV_BF16;
  cudaError_t e;
  float* scores = nullptr;
  if ((int64_t)a.b.max_new * (a.q_heads / a.c.heads) <= 32) {
    const int64_t cap = std::min<int64_t>((int64_t)a.b.table_pages << a.c.page_shift, 0x7ffff000);
    const double floats = (double)a.b.batch * a.c.heads * (double)cap * score_width(a);
    if (mass && floats * 4 <= (double)Kv8::kScoreBytes) scores = kv.scores();
    e = bf16 ? kv8_decode_bf16(kv, a, scores, s) : kv8_decode_f16(kv, a, scores, s);
  } else {
    e = bf16 ? kv8_prompt_bf16(kv, a, s) : kv8_prompt_f16(kv, a, s);
  }
  return e == cudaSuccess && mass ? kv8_weigh(kv, a, mass, scores, s) : e;
}
