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

// Quotients rounded to whole numbers, ties to even, with no rounding before that.  A product with the rounded
// reciprocal (or ratio) is within 2^-16 of the quotient and tells all but those near a half.  These are not rare: steps
// are 127ths of 16-bit numbers, and where both sides come from 8-bit mantissas one in some hundred quotients is within a
// few 2^-24 of a half, on one side or the other of it.  So the fast way gives a mask of them, and they are settled one by one.
constexpr float kKv8Whole = 12582912.0f + 128.0f;  // 1.5 2^23: added, a small number is rounded; 128 is the codes' offset
constexpr float kKv8Half = 0.49998f * 0.49998f;    // squares above belong to those

// a b / den to the nearest whole number, b of up to 8 bits, `about` the quotient within 2^-10 and near a half: the sign
// of what is left above the half, exact as two products and their errors, decides.
__device__ __forceinline__ float kv8_settle(float a, float b, float den, float about) {
  const float lo = floorf(about), half = lo + 0.5f, p = a * b, q = half * den;
  const float over = (p - q) + (fmaf(a, b, -p) - fmaf(half, den, -q));
  return over > 0.0f ? lo + 1.0f : over < 0.0f ? lo : 2.0f * rintf(0.5f * half);
}

__device__ __forceinline__ uint64_t kv8_two(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t kv8_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t kv8_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// x f + kKv8Whole of two numbers, rounded to whole ones; the mask (shifted up by two: the first one's bit the higher)
// gets the bits of those near a half.
__device__ __forceinline__ uint64_t kv8_round2(uint64_t x, uint64_t f, uint32_t& mask) {
  const uint64_t whole = kv8_two(kKv8Whole, kKv8Whole), y = kv8_fma2(x, f, whole);
  const uint64_t r = kv8_fma2(x, f, kv8_add2(whole, y ^ 0x8000000080000000ull));
  const uint64_t near = kv8_fma2(r, r ^ 0x8000000080000000ull, kv8_two(kKv8Half, kKv8Half));
  mask = __funnelshift_l((uint32_t)near, mask, 1);
  mask = __funnelshift_l((uint32_t)(near >> 32), mask, 1);
  return y;
}
// Four codes, each the low byte of kKv8Whole plus u, as a word.
__device__ __forceinline__ uint32_t kv8_word(uint64_t a, uint64_t b) {
  return __byte_perm(__byte_perm((uint32_t)a, (uint32_t)(a >> 32), 0x0040), __byte_perm((uint32_t)b, (uint32_t)(b >> 32), 0x0040),
                     0x5410);
}
// Codes of a word (u + 128 in each byte) times ratio, the products rounded to whole numbers.
__device__ __forceinline__ uint32_t kv8_scale(uint32_t w, float ratio) {
  const uint64_t f = kv8_two(ratio, ratio), whole = kv8_two(kKv8Whole, kKv8Whole), zero = kv8_two(-8388736.0f, -8388736.0f);
  auto raw = [&](int i) { return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 | i)); };
  return kv8_word(kv8_fma2(kv8_add2(kv8_two(raw(0), raw(1)), zero), f, whole), kv8_fma2(kv8_add2(kv8_two(raw(2), raw(3)), zero), f, whole));
}
// Codes of a word (u + 128 in each byte) times ratio, rounded; the bits of those near a half in the mask's lowest
// four, the first byte's the highest.
__device__ __forceinline__ uint32_t kv8_turn(uint32_t w, float ratio, uint32_t& mask) {
  const uint64_t f = kv8_two(ratio, ratio);
  const uint64_t a = kv8_round2(kv8_two(kv8_code(w, 0), kv8_code(w, 1)), f, mask);
  const uint64_t b = kv8_round2(kv8_two(kv8_code(w, 2), kv8_code(w, 3)), f, mask);
  return kv8_word(a, b);
}
// Byte i of a word, settled: u s / to.
__device__ __forceinline__ uint32_t kv8_settle_byte(uint32_t w, int i, float s, float to, float ratio) {
  const float u = (float)((int)((w >> (8 * i)) & 0xffu) - 128);
  return (uint32_t)((int)kv8_settle(s, u, to, u * ratio) + 128);
}
// A step as it enters here: nothing may leave fp32's range below it.
__device__ __forceinline__ float kv8_lift(float to) { return to < 0x1p-60f ? 0x1p80f : 1.0f; }

}  // namespace moe
