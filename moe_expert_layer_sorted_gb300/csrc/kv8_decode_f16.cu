#include "kv8_decode.cuh"

cudaError_t moe::kv8_decode_f16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  return decode8<__half>(kv, a, scores, s);
}
