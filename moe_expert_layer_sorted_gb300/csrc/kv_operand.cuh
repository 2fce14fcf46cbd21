// Code words as matrix operands, for the attention kernels (included into an
// anonymous namespace after device_common.cuh).
#pragma once

constexpr float kNone = -1e30f;  // softmax reference of a row that has seen no token

template <typename T>
struct Frag;
template <>
struct Frag<__nv_bfloat16> {
  // weights are 2^(score - reference): the reference is set kLift above the largest score and
  // raised when one comes nearer than -kSlack, so that sums of weights times values of bf16's
  // largest stay finite and a step of 2^-90 still counts
  static constexpr float kLift = 32.0f, kSlack = -24.0f;
  static constexpr float kOffset = 136.0f;  // of the key operand: 128 + u = (u - 8) + 136
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
  }
  // fields at bits 4i of both half-words, as 128 + u
  template <int I>
  static __device__ __forceinline__ uint32_t raw(uint32_t x) {
    return and_or(x >> (4 * I), 0x000f000fu, 0x43004300u);
  }
  template <int I>
  static __device__ __forceinline__ uint32_t key(uint32_t x) {
    return raw<I>(x);
  }
  template <int I>
  static __device__ __forceinline__ uint32_t value(uint32_t x) {  // u - 8, exact
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(raw<I>(x)), "r"(0xc308c308u));  // -136
    return d;
  }
};
template <>
struct Frag<__half> {
  static constexpr float kLift = 0.0f, kSlack = 2.0f;  // 4 s stays below fp16's largest for any s a cache can hold
  static constexpr float kOffset = 0.0f;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  template <int I>
  static __device__ __forceinline__ uint32_t value(uint32_t x) {  // u - 8, exact
    uint32_t d;
    const uint32_t y = I >= 2 ? x >> 8 : x;
    if constexpr (I % 2 == 0) {  // 1024 + u - 1032
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(and_or(y, 0x000f000fu, 0x64006400u)), "r"(0xe408e408u));
    } else {  // (1024 + 16 u) / 16 - 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;"
          : "=r"(d)
          : "r"(and_or(y, 0x00f000f0u, 0x64006400u)), "r"(0x2c002c00u), "r"(0xd480d480u));
    }
    return d;
  }
  template <int I>
  static __device__ __forceinline__ uint32_t key(uint32_t x) {
    return value<I>(x);
  }
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
