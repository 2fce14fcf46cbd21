#include "kv_prompt.cuh"

cudaError_t moe::kv_prompt_f16(Kv& kv, const KvAttnArgs& a, cudaStream_t s) { return prompt<__half>(kv, a, s); }
