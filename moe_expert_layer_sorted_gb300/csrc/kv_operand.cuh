// Code words as matrix operands, for the attention kernels (included into an
// anonymous namespace after device_common.cuh).
#pragma once

constexpr float kNone = -3.402823466e38f;  // softmax reference of a row that has seen no token: the lowest finite score

// 2^e, e in -126..127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2) of a positive normal fp32's bits (-127 of zero and subnormals, 128 of an infinity)
__device__ __forceinline__ int exponent(uint32_t bits) { return (int)(bits >> 23) - 127; }
// A partial result leaves with its reference m and its sum l as they are, so that equal scores of
// any size weigh the same in every part; where l is outside 2^-Span..2^Span its exponent, which
// this is, goes from l to m (there the reference went by the sizes of values).
template <int Span>
__device__ __forceinline__ int excess(float l) {
  const int e = exponent(__float_as_uint(l));
  return l > 0.0f && (e >= Span || e < -Span) ? min(e, 126) : 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// Scores from here on are rounded before the reference is taken off: the exact product differs
// from its rounded self, which the reference is, by a sixteenth there, and by any amount above.
constexpr float kCoarse = 1048576.0f;

// Fields I of both half-words of a word (4 bits each at bit 4 I) as a pair of fp16.
//   raw:     the bits themselves, a subnormal: u 2^-24, or for odd I u 2^-20.  One mask
//            (and a shift that fields 2 and 3 share); products with it are exact.
//   centred: u - 8, one instruction more.
template <int I>
__device__ __forceinline__ uint32_t raw_pair(uint32_t x) {
  return (I >= 2 ? x >> 8 : x) & (I % 2 ? 0x00f000f0u : 0x000f000fu);
}
template <int I>
__device__ __forceinline__ uint32_t centred_pair(uint32_t x) {
  uint32_t d;
  const uint32_t y = (I >= 2 ? x >> 8 : x);
  if constexpr (I % 2 == 0) {  // 1024 + u - 1032
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(and_or(y, 0x000f000fu, 0x64006400u)), "r"(0xe408e408u));
  } else {  // (1024 + 16 u) / 16 - 72
    asm("fma.rn.f16x2 %0, %1, %2, %3;"
        : "=r"(d)
        : "r"(and_or(y, 0x00f000f0u, 0x64006400u)), "r"(0x2c002c00u), "r"(0xd480d480u));
  }
  return d;
}

// Bounded wait for phase `parity` of bar.  One that gives up sets the handle's word, which the
// next call reports, and `gone` of its CTA, whose later waits then give up soon; no other CTA
// and no later launch is touched.
__device__ __forceinline__ bool kv_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gone, uint32_t* err) {
  for (uint32_t it = 0; it < (1u << 20); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 255u) == 255u && *gone) return false;
  }
  *gone = 1;
  *reinterpret_cast<volatile uint32_t*>(err) = kErrTimeout;
  __threadfence_system();
  return false;
}

// Registers of a warpgroup's threads from here on.
// `Launch`: what the block was launched with; the direction of the change has to match it.
template <int Launch, int R>
__device__ __forceinline__ void set_registers() {
  static_assert(R % 8 == 0 && R >= 24 && R <= 256 && R != Launch, "a multiple of 8 within the range");
  if constexpr (R > Launch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
// Adds 1; what this CTA wrote before (seen by this thread through a barrier) is visible to whoever
// reads the new count this way, and the other way round.
__device__ __forceinline__ unsigned add_acq_rel(unsigned* p) {
  unsigned d;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(d) : "l"(p) : "memory");
  return d;
}
// Whether a launch of `kernel` brings the registers per thread that its split deals out.
inline bool brings_registers(const void* kernel, int regs) {
  cudaFuncAttributes f{};
  return cudaFuncGetAttributes(&f, kernel) == cudaSuccess && f.numRegs == regs;
}
