// Attention over the 8-bit cache: which kernels take a call.
#include "kv8_internal.h"

using namespace moe;

// By columns (rows of a sequence times the query heads that share a kv head).  The single-token
// kernel reads the cache once per 16 columns (8 where there are no more), the prompt kernel
// once per 256 but turns every code into shared memory first.  Measured, both kernels, us (8 kv heads
// of 128 channels, bf16; single tokens / prompts):
//     columns                        8         16          32         64
//     1 sequence of 2,048        12.4 / 21   14.7 / 21   16.3 / 21   - / 21
//     1 of 131,072                 55 / 131    74 / 131   131 / 131  - / 131
//     16 of 4,096                  37 / 72     49 / 72     82 / 73   - / 73
//     64 of 2,048                  58 / 153    92 / 154   162 / 154  - / 154
//
// Weights: the single-token kernel leaves its scores behind where the workspace holds them, four
// bytes a token and column beside the 256 that it reads; otherwise they are made again from the keys.
// What weights add, us: scores left, 16 columns of 1 sequence of 131,072 37, of 64 of 2,048 39; made again, of any number of
// columns up to 128, 181 and 182.
cudaError_t moe::kv8_attention(Kv8& kv, const KvAttnArgs& a, float* mass, cudaStream_t s) {
  const bool bf16 = kv.d.dtype == MOE_KV_BF16;
  cudaError_t e;
  Kv8Scores scores{};
  const int64_t columns = (int64_t)a.b.max_new * (a.q_heads / a.c.heads), pairs = a.b.rows * a.q_heads;
  size_t used = 0;  // of the scores' room, by references and sums: none where the single-token kernel's parts leave room
  if (mass) {
    const bool beside = columns <= kKv8Columns && pairs <= Kv8::kFewRefs;
    scores.refs = beside ? kv.few_refs() : reinterpret_cast<float2*>(kv.scores());
    scores.refs_limit = std::min<int64_t>(pairs, Kv8::kScoreBytes / sizeof(float2));
    used = beside ? 0 : (scores.refs_limit * sizeof(float2) + 511) / 512 * 512;
  }
  if (columns <= kKv8Columns) {
    if (mass && a.b.batch <= Kv8::kScoreSeqs) {
      scores.to = kv.scores() + used / sizeof(float);
      scores.base = kv.score_bases();
      scores.width = std::min((int)(columns + 3) / 4 * 4, 16);
      scores.ctiles = columns > 16 ? 2 : 1;  // as the kernel has them
      scores.limit = (int)((Kv8::kScoreBytes - used) / (128 * sizeof(float) * scores.width));
    }
    e = bf16 ? kv8_decode_bf16(kv, a, scores, s) : kv8_decode_f16(kv, a, scores, s);
  } else {
    e = bf16 ? kv8_prompt_bf16(kv, a, scores, s) : kv8_prompt_f16(kv, a, scores, s);
  }
  return e == cudaSuccess && mass ? kv8_weigh(kv, a, mass, scores, s) : e;
}
