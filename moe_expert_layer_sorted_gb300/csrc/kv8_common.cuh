// Device view of the 8-bit key/value cache (included by the kv8_*.cu files).
//
// A page holds, per kv head, P / 16 blocks of 16 tokens.  A block is one run of
// bytes,
//     K codes [16][D] | V codes [8 pairs of tokens][D][2] | params (16 bytes)
// (params: the keys' and the values' step in fp32, the keys' and the values'
// marks in 16 bits each, 32 zero bits).  A code is u + 128, u in -127..127, and
// the stored value is s u with the step s that the block's keys (values) share.
// A marked token held something that is not finite: it reads as NaN, its codes
// are 0 and it has no part in the step.
// The values of two neighbouring tokens lie channel by channel beside each other
// because the product of weights and values wants pairs of tokens in a register.
// Pieces of 16 bytes change places within a row of keys and a pair of values so
// that the eight lanes that load them at once hit all 32 banks of shared memory.
#pragma once

#include "kv_common.cuh"

namespace moe {

template <int D>
struct Kv8Geom {
  static_assert(D == 64 || D == 128, "head dims");
  static constexpr int kVOff = 16 * D;
  static constexpr int kParams = 32 * D;
  static constexpr int kBytes = 32 * D + 16;
  // place of the 16 channels from 16 i on in token t's row of keys, and of the 8 channels from 8 i on in a pair of values
  static __device__ __host__ constexpr int k_piece(int t, int i) { return D == 128 ? i ^ ((t & 1) << 2) : i; }
  static __device__ __host__ constexpr int v_piece(int pair, int i) {
    return D == 128 ? i ^ ((pair & 1) | (pair & 2) << 1) : i ^ (2 * (pair & 3));
  }
};

struct Kv8Params {
  float step[2];     // keys, values
  uint16_t mark[2];  // a bit per token
  uint32_t zero;
};
static_assert(sizeof(Kv8Params) == 16, "one 16-byte load");

// Bytes 2 i, 2 i + 1 of a word as a pair of fp16, u exactly: 1024 + (u + 128) - 1152.
template <int I>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(w, 0x64646464u, I ? 0x4342 : 0x4140)), "r"(0xe480e480u));
  return d;
}
// The codes of the two channels of a word of values, of the pair's token I.
template <int I>
__device__ __forceinline__ uint32_t kv8_token(uint32_t w) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(w, 0x64646464u, I ? 0x4341 : 0x4240)), "r"(0xe480e480u));
  return d;
}
// Byte i of a word as u in fp32.
__device__ __forceinline__ float kv8_code(uint32_t w, int i) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 | i)) - 8388736.0f;
}

}  // namespace moe
