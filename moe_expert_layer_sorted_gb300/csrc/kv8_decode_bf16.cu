#include "kv8_decode.cuh"

cudaError_t moe::kv8_decode_bf16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  return decode8<__nv_bfloat16>(kv, a, scores, s);
}
