#include "kv_decode.cuh"

cudaError_t moe::kv_decode_f16(Kv& kv, const KvAttnArgs& a, cudaStream_t s) { return decode<__half>(kv, a, s); }
