#include "kv8_prompt.cuh"

cudaError_t moe::kv8_prompt_bf16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  return prompt8<__nv_bfloat16>(kv, a, scores, s);
}
