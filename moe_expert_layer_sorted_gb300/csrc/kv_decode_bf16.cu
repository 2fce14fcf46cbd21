#include "kv_decode.cuh"

cudaError_t moe::kv_decode_bf16(Kv& kv, const KvAttnArgs& a, cudaStream_t s) { return decode<__nv_bfloat16>(kv, a, s); }
