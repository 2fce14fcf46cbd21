#include "kv8_prompt.cuh"

cudaError_t moe::kv8_prompt_f16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  return prompt8<__half>(kv, a, scores, s);
}
