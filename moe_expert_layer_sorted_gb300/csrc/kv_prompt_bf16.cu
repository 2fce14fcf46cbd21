#include "kv_prompt.cuh"

cudaError_t moe::kv_prompt_bf16(Kv& kv, const KvAttnArgs& a, cudaStream_t s) { return prompt<__nv_bfloat16>(kv, a, s); }
