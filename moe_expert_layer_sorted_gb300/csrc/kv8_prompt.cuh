// Attention of prompts over the 8-bit cache: many rows per kv head, on the
// tcgen05 tensor cores.  Included by kv8_prompt_bf16.cu and kv8_prompt_f16.cu.
//
// One CTA takes 256 rows x of one sequence and kv head (x = row * (heads per
// kv head) + head, so that the heads that share keys share a tile) as two tiles
// of 128, and walks over the tokens in tiles of 128:
//   S_t = Q_t U_K^T   (queries and key codes in shared memory, S fp32 in TMEM),
//   P_t = 2^(S_t scale log2 e s_K + log2 s_V - rz) in 16 bits over S_t's columns,
//   O_t += P_t U_V    (P as the TMEM operand, value codes token-major).
// The codes -127..127 are exact in fp16, and the blocks' steps cost nothing: s_K goes
// into the factor of a block's 16 columns, s_V into what is added there.  Roles:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row (a TMEM lane);
//   warps 8-11      stored codes -> 16-bit K and V tiles, two blocks of each a warp;
//   warp 12         tcgen05.mma issue, TMEM allocation.
// Rounding: P to 11 bits; everything else is exact or fp32 (a query row of bf16 is
// scaled by the power of two that brings its largest element to 2^14).
//
// Two references per row: ry, a score, of the sum of weights 2^(y - ry), and
// rz = ry - dz of the weights times steps.  In an ordinary tile the sum comes from P itself:
// a block's sum of P times 2^(lv0 - log2 s_V), lv0 the tile's largest log2 s_V, and the tile's
// times 2^(-dz - lv0).  Tiles with masks, with steps of very different sizes (or of zero), or
// far from what the row's references are made for, take two exponentials per score, one for
// the sum and one for P, so that values of any size take nothing from the sum, nor weights
// from the values.  A row's references are raised, and O rescaled in TMEM, only where a
// tile's P would outgrow fp16 (or its sum fp32), and rz is lowered, O scaled up, where a tile's P
// are all small: a token that takes most of a row's weight may have next to no value (a block's
// step says nothing of a single token of it), and what the others weigh then makes up the result.
//
// Where there are fewer tiles of rows than half the SMs, the tokens are cut into as
// many stretches as fill them, and a second kernel joins a tile's parts, in the order
// of the stretches.
//
// Masks: a score that its row may not see becomes -infinity.  Tokens that are not finite
// have codes of zeros; a row that sees one is remembered, and NaN in the end.
//
// Measured (bf16, 32 query and 8 kv heads of 128 channels): 8,192 rows at the end of 16,384 tokens 1,314 us, 1,255
// TFLOP/s (0.64 of the measured rate); with scores that never raise a reference 1,274; 4,096 rows (fp16) 158 us.
// Bound by two things of about the same length: the chain of a token tile, scores -> weights -> product, of which
// two row tiles alternate (without the loads of codes and the exponents it takes 1,130 us), and the warps that turn
// codes (without their loads 1,219).  What paid: a tile's words asked for as soon as the last one's are turned, what
// the softmax wants to know of a tile worked out a tile ahead (1,446 -> 1,267 us with scores that never raise).  Three
// ragged prompts of up to 333 rows over up to 2,500 tokens (fp16, 12 heads of 64): 39 us, ten token tiles one
// after the other, launch and join.
#pragma once

#include "kv8_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"
#include "kv_tcgen.cuh"

constexpr int kPrSoft = 8, kPrDequant = 4, kPrMma = kPrSoft + kPrDequant;
constexpr int kPrThreads = 512;  // four warpgroups; warps 13-15 only fill theirs
// Registers: the launch's 128 per thread are dealt out again between the warpgroups,
// 128 threads x (176 + 176 + 112 + 48) = 512 x 128.
constexpr int kPrRegs = 128, kPrSoftRegs = 176, kPrDequantRegs = 112, kPrMmaRegs = 48;
static_assert(2 * kPrSoftRegs + kPrDequantRegs + kPrMmaRegs == 4 * kPrRegs, "a split above the launch's registers never ends");
// rz is set kPrDrop below the largest weight times step and raised when a tile's sum comes to kPrLimit, so that this is 2^kPrAim:
// no P passes fp16's range.  Where the sum passes kPrFar, the scores are looked through again, which takes a tile three times as
// long (every raise so, 7 and 2^15, 4 and 2^15, 2 and 60,000: 1,542, 1,379 and 1,301 us for the chunk below, whose scores have a
// standard deviation of 2).
constexpr float kPrDrop = 2.0f, kPrLimit = 60000.0f, kPrAim = 5.0f, kPrFar = 0x1p60f;
// rz is lowered, the sum 2^kPrAim again, where the P of the tokens that a row sees of a tile are below kPrLow on average: fp16's
// last place below 2^-14 is 2^-24, so such a P is off by 2^-25 at most, and 128 of them by twice what 11 bits would be beside
// their sum.  By no more than 2^kPrFall since it was raised, which keeps O within fp32 (tiles' sums of 2^16 times 127, by 2^24
// tiles: 2^103); falls of less than kPrStep and what is below kPrGone are left alone.  Measured, never lowered / lowered, us: the
// 8,192 rows below 1,308 / 1,314, with scores that never raise a reference 1,271 / 1,274, the ragged prompts 39.3 / 39.3 (50 where
// the scores are looked through for it).
constexpr float kPrLow = 0x1p-15f, kPrGone = 0x1p-64f, kPrFall = 56.0f, kPrStep = 8.0f;
constexpr float kPrApart = 30.0f;       // log2 of how far an ordinary tile's steps may lie apart,
constexpr float kPrNear = 60.0f;        // and of how far they may be from the row's 2^-dz
constexpr float kPrMaxSum = 0x1p60f;    // ry is raised when a tile's weights sum to this
constexpr float kNoProduct = 1e38f;     // dz of a row that has seen no token

// A block's constants, in order with the other asm statements: loaded where they are wanted, not all at once.
__device__ __forceinline__ float4 load_block(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ float log2_fast(float x) {
  float d;
  asm("lg2.approx.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t load_word(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

struct Prompt8Args : PromptArgs {
  float2* refs;        // see Kv8Scores
  int64_t refs_limit;
};
// What a row leaves for its weights to be counted.
__device__ __forceinline__ void leave(const Prompt8Args& p, int64_t row, float reference, float sum) {
  if (row < p.refs_limit) p.refs[row] = make_float2(reference, 1.0f / sum);
}

// Floats of a stretch's part: results [D / 4][row] of four channels, then references, sums, 1 where a row is NaN.
template <int D>
constexpr int64_t kPr8Part = 2 * kPrTile * (D + 3);

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads, 1) kv8_prompt_kernel(const __grid_constant__ Prompt8Args p) {
  using Geo = Kv8Geom<D>;
  constexpr uint32_t kSlab = kPrTile * 128;          // 128 rows of 64 channels
  constexpr uint32_t kTileBytes = kSlab * (D / 64);  // a Q, K or V tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t kFull[2], kEmpty[2], vFull[2], vEmpty[2], sFull[2], pFull[2], qFull, oFull;
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t sh_gone;  // a wait gave up: results are wrong, the next call says so
  // per token tile (ring of 4): tokens that exist, tokens with keys, values that are not finite
  __shared__ uint4 sh_valid[4], sh_kbad[4], sh_vbad[4];
  __shared__ uint32_t sh_any_bad[4];           // whether there are any of the latter
  __shared__ float4 sh_block[4][8];            // and its blocks: the keys' step, log2 of the values', the factor of a sum of P
  __shared__ float4 sh_vs[4][2];               // and the values' step
  __shared__ float sh_lv0[4];                  // the largest log2 of the values' steps; NaN: not an ordinary tile, or not all there
  __shared__ float sh_qscale[2 * kPrTile];     // what a query row's scores are multiplied by
  const KvAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const PromptTile tile(p);
  const int nx = tile.nx, x0 = tile.x0;
  if (x0 >= nx) return;
  const int s = tile.s, h = tile.h, most = tile.most, splits = tile.splits, z = blockIdx.y;
  const KvSeq q = tile.q;
  if (z >= splits) return;
  const int base = (int)((int64_t)tile.all * z / splits) * kPrTile;  // this CTA's first token
  const int ntiles = (int)((int64_t)tile.all * (z + 1) / splits) - base / kPrTile;
  const bool two = nx > x0 + kPrTile;  // the second row tile has rows
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = smem, sk = smem + 2 * kTileBytes, sv = sk + 2 * kTileBytes;
  uint8_t* gen = smem_raw + (smem - smem_addr(smem_raw));  // the same places as a generic pointer

  if (tid == 0) {
    sh_gone = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&kFull[i]), kPrDequant);
      mbar_init(smem_addr(&kEmpty[i]), 1);
      mbar_init(smem_addr(&vFull[i]), kPrDequant);
      mbar_init(smem_addr(&vEmpty[i]), 1);
      mbar_init(smem_addr(&sFull[i]), 1);
      mbar_init(smem_addr(&pFull[i]), 4);
    }
    mbar_init(smem_addr(&qFull), 1);
    mbar_init(smem_addr(&oFull), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPrMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = tmem_base;

  if (warp < kPrSoft) {
    // ------------------------------------------------------------------ softmax
    set_registers<kPrRegs, kPrSoftRegs>();
    const int t = warp >> 2, quad = warp & 3;
    const int x = x0 + t * kPrTile + quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tm + t * kPrTile + lanes, to = tm + 2 * kPrTile + t * D + lanes;
    // tokens from `base` on that the row sees; rows past the last (zeros, not written) ask for no masks
    const int seen = (x < nx ? tile.seen(p, x) : most) - base;
    static_assert(kPrSoft * 32 == 2 * kPrTile, "two threads per row of a tile");
    load_queries<T, D>(gen, sh_qscale, a, s, h, q, p.per, x0, nx, tid);
    load_queries<T, D>(gen + kTileBytes, sh_qscale + kPrTile, a, s, h, q, p.per, x0 + kPrTile, nx, tid);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("bar.sync 2, %0;" ::"n"(kPrSoft * 32) : "memory");
    if (tid == 0) mbar_arrive(smem_addr(&qFull));
    const float kappa = a.scale * 1.4426950408889634f * sh_qscale[t * kPrTile + quad * 32 + lane];
    float ry = kNone, dz = kNoProduct, l = 0.0f;
    float fell = 0.0f;    // how far rz has been lowered since it was raised
    bool vnan = false;    // the row sees values that are not finite
    bool coarse = false;  // a row's scores are as large as kKv8Coarse
    for (int j = 0; j < (t == 0 || two ? ntiles : 0); ++j) {
      kv_wait(smem_addr(&sFull[t]), (uint32_t)j & 1u, &sh_gone, p.err);
      fence_after();
      uint32_t v[2][32];
      const uint32_t blocks = smem_addr(&sh_block[j & 3][0]);
      const float lv0 = sh_lv0[j & 3];
      // an ordinary tile, which every row of the warp sees in full (one that is NaN changes nothing for the others)
      auto ordinary = [&]() {
        return __all_sync(0xffffffffu, seen >= (j + 1) * kPrTile && (fabsf(dz + lv0) <= kPrNear || (l != l && lv0 == lv0))) && !coarse;
      };
      bool plain = ordinary();
      uint32_t pr[kPrTile / 2];
      auto mask_of = [&](int k) {  // tokens of the k-th 32 that the row sees
        const int n = seen - (j * kPrTile + 32 * k);
        return load_word(smem_addr(&sh_valid[j & 3]) + 4 * k) & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
      };
      // the k-th 32 scores, rounded, masked ones -infinity
      auto load = [&](int k, uint32_t (&v)[32]) {
        tmem_ld32(ts + 32 * k, v);
        tmem_wait_ld();
        const uint32_t mask = mask_of(k);
        const float f[2] = {kappa * load_block(blocks + 32 * k).x, kappa * load_block(blocks + 32 * k + 16).x};
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (mask >> i) & 1u ? __float_as_uint(__uint_as_float(v[i]) * f[i / 16]) : 0xff800000u;
      };
      uint64_t sum = 0, whole = 0;  // of P, and of the weights (an ordinary tile's: times 2^(dz + lv0))
      // v: sums of an ordinary tile, else rounded scores; lo, hi: the two blocks
      auto weights = [&](const uint32_t (&v)[32], int k, float4 lo, float4 hi, auto plain_) {
        constexpr bool plain = decltype(plain_)::value;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 b = y ? hi : lo;
          float e[16];  // step by step: independent instructions side by side
          auto total = [&]() {
            uint64_t part[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) part[i] = add2(pair2(e[2 * i], e[2 * i + 1]), pair2(e[2 * i + 8], e[2 * i + 9]));
            return add2(add2(part[0], part[1]), add2(part[2], part[3]));
          };
          if constexpr (plain) {
            const float f = kappa * b.x, add = (b.y + dz) - ry;
            const uint64_t f2 = pair2(f, f), plus = pair2(add, add);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              split2(fma2(pair2(__uint_as_float(v[16 * y + i]), __uint_as_float(v[16 * y + i + 1])), f2, plus), e[i], e[i + 1]);
          } else {
            const float plus = b.y + dz;
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = exp2_fast(__uint_as_float(v[16 * y + i]) - ry);
            whole = add2(whole, total());
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = (__uint_as_float(v[16 * y + i]) - ry) + plus;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) e[i] = exp2_fast(e[i]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) pr[16 * k + 8 * y + i / 2] = KvType<__half>::pack(e[i], e[i + 1]);
          const uint64_t part = total();
          sum = add2(sum, part);
          if constexpr (plain) whole = fma2(part, pair2(b.z, b.z), whole);
        }
      };
      // P against the references as they stand, and once more where they have to move: for the first tile, or where
      // a P or a weight is above its limit, which shows in the sum (that may reach the limit without one: no harm), or where
      // the row's P are all small.  Mostly the sum tells by how much, otherwise the scores are looked through.
      enum { kStay, kShift, kScan } move = j == 0 ? kScan : kStay;
      float by = 0.0f;
      while (true) {
        if (move != kStay) {
          float cur = dz, next = dz + by;
          if (move == kScan) {
            float top = kNone, most_z = -__int_as_float(0x7f800000);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              load(k, v[0]);
#pragma unroll
              for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(v[0][i]));
            }
            const float now = fmaxf(ry, top);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              load(k, v[0]);
              const float lv[2] = {load_block(blocks + 32 * k).y, load_block(blocks + 32 * k + 16).y};
#pragma unroll
              for (int i = 0; i < 32; ++i) most_z = fmaxf(most_z, (__uint_as_float(v[0][i]) - now) + lv[i / 16]);
            }
            l *= exp2_fast(ry - now);
            cur = fminf(dz - (ry - now), kNoProduct);
            const float want = kPrDrop - most_z;  // (infinite where there is nothing)
            next = want >= cur + kPrStep && want <= cur + 64.0f && fell <= kPrFall - kPrStep ? fminf(want, cur + (kPrFall - fell)) : fminf(want, cur);
            ry = now;
            coarse = coarse || __any_sync(0xffffffffu, ry != kNone && fabsf(ry) >= kKv8Coarse);
          }
          const float fo = next != cur ? exp2_fast(next - cur) : 1.0f;
          dz = next;
          fell = fmaxf(fell + (next - cur), 0.0f);
          plain = ordinary();
          if (j > 0 && __any_sync(0xffffffffu, fo != 1.0f)) {
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              tmem_ld32(to + 32 * k, v[0]);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[0][i] = __float_as_uint(__uint_as_float(v[0][i]) * fo);
              tmem_st32(to + 32 * k, v[0]);
            }
            tmem_wait_st();
          }
        }
        sum = whole = 0;
        if (plain) {
          tmem_ld32(ts, v[0]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // the next 32 scores arrive while these are worked on
            const float4 lo = load_block(blocks + 32 * k), hi = load_block(blocks + 32 * k + 16);
            tmem_wait_ld();
            if (k < 3) tmem_ld32(ts + 32 * (k + 1), v[(k + 1) & 1]);
            weights(v[k & 1], k, lo, hi, std::true_type());
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            load(k, v[0]);
            weights(v[0], k, load_block(blocks + 32 * k), load_block(blocks + 32 * k + 16), std::false_type());
          }
        }
        if (move == kScan) break;
        float s0, s1, w0, w1;
        split2(sum, s0, s1);
        split2(whole, w0, w1);
        s0 += s1;
        const bool large = !plain && w0 + w1 > kPrMaxSum;
        if (!__any_sync(0xffffffffu, s0 > kPrLimit || s0 < kPrLow * kPrTile || large)) break;
        if (__any_sync(0xffffffffu, s0 > kPrFar || large)) {
          move = kScan;
          continue;
        }
        if (move == kShift) break;
        const bool low = s0 < kPrLow * (float)min(seen - j * kPrTile, kPrTile) && s0 > kPrGone && fell <= kPrFall - kPrStep;
        by = s0 > kPrLimit || low ? fminf(kPrAim - log2_fast(s0), kPrFall - fell) : 0.0f;
        if (!__any_sync(0xffffffffu, by != 0.0f)) break;
        move = kShift;
      }
      {
        float w0, w1;
        split2(whole, w0, w1);
        l = plain ? fmaf(w0 + w1, exp2_fast(-dz - lv0), l) : l + (w0 + w1);
      }
      tmem_st32(ts, pr);
      tmem_st32(ts + 32, pr + 32);
      if (load_word(smem_addr(&sh_any_bad[j & 3]))) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          if (load_word(smem_addr(&sh_kbad[j & 3]) + 4 * k) & mask_of(k)) l = __int_as_float(0x7fffffff);
          if (load_word(smem_addr(&sh_vbad[j & 3]) + 4 * k) & mask_of(k)) vnan = true;
        }
      }
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&pFull[t]));
    }
    // ---- output
    if (ntiles > 0) {
      kv_wait(smem_addr(&oFull), 0, &sh_gone, p.err);
      fence_after();
    }
    // where a wait gave up, rows are NaN, their lse too, so that they add nothing to mass
    if (*static_cast<volatile uint32_t*>(&sh_gone)) l = __int_as_float(0x7fffffff);
    const int row = t * kPrTile + quad * 32 + lane;
    const bool has = t == 0 || two;
    auto sums = [&](int k, uint32_t (&v)[32]) {  // 32 channels of the row's O
      if (ntiles > 0) {
        tmem_ld32(to + 32 * k, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0;
      }
    };
    const PromptTile end(p);  // asked for anew rather than kept in registers
    const int xe = end.x0 + row, i = xe / p.per, hq = end.h * p.per + xe % p.per;
    uint16_t* dst = has && xe < end.nx ? a.out + kv_row_offset(a.b, a.os, end.s, end.q.row0, i) + (int64_t)hq * a.os.head : nullptr;
    // 2^-dz / l, in two steps that stay in range; a row that sees nothing is zero
    const float f1 = dz >= kNoProduct ? 1.0f : exp2f(-0.5f * dz);
    const float f0 = vnan ? __int_as_float(0x7fffffff) : l == 0.0f ? 0.0f : f1 / l;
    if (splits == 1) {
      if (has) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t v[32];
          sums(k, v);
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = KvType<T>::pack(__uint_as_float(v[2 * e]) * f0 * f1, __uint_as_float(v[2 * e + 1]) * f0 * f1);
          if (!dst) {
          } else if (reinterpret_cast<uintptr_t>(dst) & 31) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(dst + 32 * k + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {  // whole sectors
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * k + 2 * e), "r"(o[e]),
                           "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                           : "memory");
          }
        }
      }
      if (dst && a.lse) {
        const int64_t at = kv_row_index(a.b, end.s, end.q.row0, i) * a.q_heads + hq;
        a.lse[at] = l == 0.0f ? -__int_as_float(0x7f800000) : (ry + log2f(l)) * 0.6931471805599453f;
        leave(p, at, ry, l);
      }
    } else if (has) {  // a stretch's part
      float* part = p.ws + ((int64_t)blockIdx.x * p.splits + z) * kPr8Part<D>;
      const float g0 = l == 0.0f ? 0.0f : f1 / l;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t v[32];
        sums(k, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<float4*>(part)[(8 * k + e) * (2 * kPrTile) + row] =
              make_float4(__uint_as_float(v[4 * e]) * g0 * f1, __uint_as_float(v[4 * e + 1]) * g0 * f1,
                          __uint_as_float(v[4 * e + 2]) * g0 * f1, __uint_as_float(v[4 * e + 3]) * g0 * f1);
      }
      float* ends = part + 2 * kPrTile * D + row;
      ends[0] = ry;
      ends[2 * kPrTile] = l;
      ends[4 * kPrTile] = vnan ? 1.0f : 0.0f;
    }
  } else if (warp < kPrMma) {
    // ------------------------------------------------------------------ codes to K and V tiles
    set_registers<kPrRegs, kPrDequantRegs>();
    const int dw = warp - kPrSoft;  // blocks 2 dw and 2 dw + 1 of a tile
    constexpr int kKLanes = D / 16, kKRows = 32 / kKLanes, kVLanes = D / 8, kVPairs = 32 / kVLanes;
    constexpr int kLoads = 16 / kKRows;  // of 16 bytes, per block, keys and values each
    static_assert(kLoads == 8 / kVPairs, "as many for both");
    const int kc = lane % kKLanes, kr = lane / kKLanes, vc = lane % kVLanes, vp = lane / kVLanes;
    uint4 kq[2][kLoads], vq[2][kLoads];
    uint3 par[2];                           // steps and marks of a tile's blocks
    uint32_t there = 0;                     // its tokens that are in a page
    const uint8_t* at[2];                   // the blocks whose words are asked for next, nullptr: none
    int pid[2];                             // pages of the blocks one tile on
    const uint4 none = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
    auto page_of = [&](int j) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int pos = base + j * kPrTile + 32 * dw + 16 * y;
        pid[y] = j < ntiles && pos < most ? (int)kv_page(a.c, a.b, s, pos >> a.c.page_shift) : -1;
      }
    };
    auto find = [&](int j) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int pos = base + j * kPrTile + 32 * dw + 16 * y;
        at[y] = pid[y] < 0 ? nullptr
                           : a.c.pages + pid[y] * a.c.page_stride + h * a.c.head_stride +
                                 ((pos & (a.c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
      }
    };
    auto load_k = [&](auto y_) {
      constexpr int y = decltype(y_)::value;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kKRows + kr;
        kq[y][i] = at[y] ? *reinterpret_cast<const uint4*>(at[y] + r * D + Geo::k_piece(r, kc) * 16) : none;
      }
    };
    auto load_v = [&](auto y_) {
      constexpr int y = decltype(y_)::value;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kVPairs + vp;
        vq[y][i] = at[y] ? *reinterpret_cast<const uint4*>(at[y] + Geo::kVOff + r * 2 * D + Geo::v_piece(r, vc) * 16) : none;
      }
    };
    auto load_params = [&]() {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        par[y] = make_uint3(0, 0, 0);
        if (at[y]) {
          const uint4 x = *reinterpret_cast<const uint4*>(at[y] + Geo::kParams);
          par[y] = make_uint3(x.x, x.y, x.z);
        }
      }
      there = (at[0] ? 0xffffu : 0u) | (at[1] ? 0xffff0000u : 0u);
    };
    auto place = [&](uint8_t* tile, int r, int ch8) {  // channels 8 ch8 .. of token r
      return reinterpret_cast<uint4*>(tile + (ch8 / 8) * kSlab + r * 128 + ((ch8 % 8) ^ (r & 7)) * 16);
    };
    auto put_k = [&](uint8_t* tile, auto y_) {
      constexpr int y = decltype(y_)::value;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = 32 * dw + 16 * y + i * kKRows + kr;
        uint4 w = kq[y][i];
        // (128 channels: half of the lanes store the upper eight first, so that eight lanes hit all banks)
        const bool turn = D == 128 && kc >= 4;
        if (turn) w = make_uint4(w.z, w.w, w.x, w.y);
        const uint4 lo = make_uint4(kv8_pair<0>(w.x), kv8_pair<1>(w.x), kv8_pair<0>(w.y), kv8_pair<1>(w.y));
        const uint4 hi = make_uint4(kv8_pair<0>(w.z), kv8_pair<1>(w.z), kv8_pair<0>(w.w), kv8_pair<1>(w.w));
        *place(tile, r, 2 * kc + turn) = lo;
        *place(tile, r, 2 * kc + 1 - turn) = hi;
      }
    };
    auto put_v = [&](uint8_t* tile, auto y_) {
      constexpr int y = decltype(y_)::value;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = 32 * dw + 16 * y + 2 * (i * kVPairs + vp);
        const uint32_t w[4] = {vq[y][i].x, vq[y][i].y, vq[y][i].z, vq[y][i].w};
        *place(tile, r, vc) = make_uint4(kv8_token<0>(w[0]), kv8_token<0>(w[1]), kv8_token<0>(w[2]), kv8_token<0>(w[3]));
        *place(tile, r + 1, vc) = make_uint4(kv8_token<1>(w[0]), kv8_token<1>(w[1]), kv8_token<1>(w[2]), kv8_token<1>(w[3]));
      }
    };
    constexpr std::integral_constant<int, 0> b0;
    constexpr std::integral_constant<int, 1> b1;
    // what the softmax wants to know of the tile whose params are in hand; the tile's keys are announced later
    auto tell = [&](int slot) {
      if (lane < 2) reinterpret_cast<float*>(sh_vs[slot])[2 * dw + lane] = __uint_as_float(lane ? par[1].y : par[0].y);
      if (lane == 0) {
        reinterpret_cast<uint32_t*>(&sh_valid[slot])[dw] = there;
        reinterpret_cast<uint32_t*>(&sh_kbad[slot])[dw] = (par[0].z & 0xffffu) | par[1].z << 16;
        reinterpret_cast<uint32_t*>(&sh_vbad[slot])[dw] = par[0].z >> 16 | (par[1].z & 0xffff0000u);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kPrDequant * 32) : "memory");
      // the tile's largest and smallest step of values
      const float4 v0 = sh_vs[slot][0], v1 = sh_vs[slot][1];
      const float big = fmaxf(fmaxf(fmaxf(v0.x, v0.y), fmaxf(v0.z, v0.w)), fmaxf(fmaxf(v1.x, v1.y), fmaxf(v1.z, v1.w)));
      const float small = fminf(fminf(fminf(v0.x, v0.y), fminf(v0.z, v0.w)), fminf(fminf(v1.x, v1.y), fminf(v1.z, v1.w)));
      const float lv0 = log2_fast(big);
      if (lane < 2) {
        const float lv = log2_fast(__uint_as_float(lane ? par[1].y : par[0].y));  // -infinity of zero
        sh_block[slot][2 * dw + lane] = make_float4(__uint_as_float(lane ? par[1].x : par[0].x), lv, exp2_fast(lv0 - lv), 0.0f);
      }
      if (tid == kPrSoft * 32) {
        sh_lv0[slot] = lv0 - log2_fast(small) <= kPrApart ? lv0 : __int_as_float(0x7fffffff);
        const uint4 x = sh_kbad[slot], y = sh_vbad[slot];
        sh_any_bad[slot] = x.x | x.y | x.z | x.w | y.x | y.y | y.z | y.w;
      }
    };
    // the words of a tile are asked for as soon as the last one's are turned
    if (ntiles > 0) {
      page_of(0);
      find(0);
      load_k(b0);
      load_k(b1);
      load_v(b0);
      load_v(b1);
      load_params();
      page_of(1);
      tell(0);
    }
    for (int j = 0; j < ntiles; ++j) {
      const int st = j & 1;
      const uint32_t free_parity = ((uint32_t)(j >> 1) & 1u) ^ 1u;
      kv_wait(smem_addr(&kEmpty[st]), free_parity, &sh_gone, p.err);
      uint8_t* tk = gen + 2 * kTileBytes + st * kTileBytes;
      find(j + 1);
      put_k(tk, b0);
      load_k(b0);
      put_k(tk, b1);
      load_k(b1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&kFull[st]));
      load_params();
      page_of(j + 2);
      kv_wait(smem_addr(&vEmpty[st]), free_parity, &sh_gone, p.err);
      uint8_t* tv = gen + 4 * kTileBytes + st * kTileBytes;
      put_v(tv, b0);
      load_v(b0);
      put_v(tv, b1);
      load_v(b1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      const bool held = p.fail && blockIdx.x == 0 && z == 0 && j == ntiles - 1 && dw == 0;
      if (lane == 0 && !held) mbar_arrive(smem_addr(&vFull[st]));
      tell((j + 1) & 3);
    }
  } else {
    set_registers<kPrRegs, kPrMmaRegs>();
    // ------------------------------------------------------------------ MMA issue
    const uint32_t ids = idesc(kPrTile, false), ido = idesc(D, true);
    const int nt = two ? 2 : 1;
    const uint32_t leader = elect_leader();
    auto scores = [&](int t, int j) {
      const uint32_t qa = sq + t * kTileBytes, kb = sk + (j & 1) * kTileBytes;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(leader, tm + t * kPrTile, desc_k(qa + (k / 4) * kSlab + (k % 4) * 32),
               desc_k(kb + (k / 4) * kSlab + (k % 4) * 32), ids, k ? 1u : 0u);
      commit(leader, &sFull[t]);
      if (t == nt - 1) commit(leader, &kEmpty[j & 1]);
    };
    if (warp == kPrMma && ntiles > 0) {
      kv_wait(smem_addr(&qFull), 0, &sh_gone, p.err);
      kv_wait(smem_addr(&kFull[0]), 0, &sh_gone, p.err);
      fence_after();
      for (int t = 0; t < nt; ++t) scores(t, 0);
      for (int j = 0; j < ntiles; ++j) {
        // both operands of this round are usually there long before the weights
        kv_wait(smem_addr(&vFull[j & 1]), (uint32_t)(j >> 1) & 1u, &sh_gone, p.err);
        if (j + 1 < ntiles) kv_wait(smem_addr(&kFull[(j + 1) & 1]), (uint32_t)((j + 1) >> 1) & 1u, &sh_gone, p.err);
        for (int t = 0; t < nt; ++t) {
          kv_wait(smem_addr(&pFull[t]), (uint32_t)j & 1u, &sh_gone, p.err);
          fence_after();
          const uint32_t vb = sv + (j & 1) * kTileBytes;
#pragma unroll
          for (int k = 0; k < kPrTile / 16; ++k)
            mma_ts(leader, tm + 2 * kPrTile + t * D, tm + t * kPrTile + 8 * k, desc_mn(vb + k * 2048), ido, (j | k) ? 1u : 0u);
          if (t == nt - 1) commit(leader, &vEmpty[j & 1]);
          if (j + 1 < ntiles) scores(t, j + 1);
        }
      }
      commit(leader, &oFull);
      mbar_drain(smem_addr(&oFull), 0);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kPrMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(512));
  }
}

// Joins the stretches' parts of a pair of row tiles: a CTA takes 32 rows, lane by lane, a warp
// every eighth four channels.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_join_kernel(const __grid_constant__ Prompt8Args p) {
  const KvAttnArgs& a = p.a;
  const PromptTile tile(p);
  const int row = blockIdx.y * 32 + (threadIdx.x & 31);
  const int x = tile.x0 + row;
  if (x >= tile.nx || tile.splits == 1) return;
  const float* parts = p.ws + (int64_t)blockIdx.x * p.splits * kPr8Part<D>;
  const float* ends = parts + 2 * kPrTile * D + row;
  float m = kNone, l = 0.0f, bad = 0.0f;
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) m = fmaxf(m, __ldcg(ends + y * kPr8Part<D>));
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) {
    l = fmaf(exp2_fast(__ldcg(ends + y * kPr8Part<D>) - m), __ldcg(ends + y * kPr8Part<D> + 2 * kPrTile), l);
    bad += __ldcg(ends + y * kPr8Part<D> + 4 * kPrTile);
  }
  const float inv = bad > 0.0f ? __int_as_float(0x7fffffff) : l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is zero
  const int i = x / p.per, hq = tile.h * p.per + x % p.per;
  uint16_t* dst = a.out + kv_row_offset(a.b, a.os, tile.s, tile.q.row0, i) + (int64_t)hq * a.os.head;
  constexpr int kQuads = D / 4 / 8;  // of four channels, per thread
  float4 o[kQuads];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) {
    const float f = exp2_fast(__ldcg(ends + y * kPr8Part<D>) - m) * (__ldcg(ends + y * kPr8Part<D> + 2 * kPrTile) * inv);
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int d4 = (threadIdx.x >> 5) * kQuads + k;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(parts + y * kPr8Part<D>) + d4 * (2 * kPrTile) + row);
      o[k].x = fmaf(f, v.x, o[k].x);
      o[k].y = fmaf(f, v.y, o[k].y);
      o[k].z = fmaf(f, v.z, o[k].z);
      o[k].w = fmaf(f, v.w, o[k].w);
    }
  }
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int d4 = (threadIdx.x >> 5) * kQuads + k;
    *reinterpret_cast<uint2*>(dst + 4 * d4) = make_uint2(KvType<T>::pack(o[k].x, o[k].y), KvType<T>::pack(o[k].z, o[k].w));
  }
  if (a.lse && threadIdx.x < 32) {
    const int64_t at = kv_row_index(a.b, tile.s, tile.q.row0, i) * a.q_heads + hq;
    a.lse[at] = l == 0.0f ? -__int_as_float(0x7f800000) : (m + log2f(l)) * 0.6931471805599453f;
    leave(p, at, m, l);
  }
}

template <typename T, int D>
cudaError_t launch_prompt8(const Prompt8Args& p, unsigned ctas, cudaStream_t s) {
  const size_t smem = 1024 + (size_t)6 * kPrTile * D * 2;
  const auto kernel = kv8_prompt_kernel<T, D>;
  static const bool registers_fit = brings_registers(reinterpret_cast<const void*>(kernel), kPrRegs);
  if (!registers_fit) return cudaErrorInvalidKernelImage;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(ctas, (unsigned)p.splits), kPrThreads, smem, s>>>(p);
  if (p.splits > 1) kv8_join_kernel<T, D><<<dim3(ctas, 2 * kPrTile / 32), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t prompt8(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  Prompt8Args p{{a, a.q_heads / a.c.heads, 0, 1, kv.parts(), kv.err_dev, kv.fail_next}, scores.refs, scores.refs_limit};
  const int64_t tiles = ((int64_t)a.b.max_new * p.per + 2 * kPrTile - 1) / (2 * kPrTile);
  const int64_t ctas = tiles * a.c.heads * a.b.batch;
  if (ctas > 0x7fffffff || (int64_t)a.c.heads * a.b.batch > 0x7fffffff || tiles * 2 * kPrTile > 0x7fffffff)
    return cudaErrorInvalidConfiguration;
  p.tiles = (int)tiles;
  // the SMs hold one CTA each; the parts have to fit the workspace
  const int64_t slots = Kv8::kPartsBytes / (2 * kPrTile * (kv.d.head_dim + 3) * sizeof(float));
  p.splits = (int)std::max<int64_t>(std::min<int64_t>(kv.sms, slots) / ctas, 1);
  return kv.d.head_dim == 64 ? launch_prompt8<T, 64>(p, (unsigned)ctas, s) : launch_prompt8<T, 128>(p, (unsigned)ctas, s);
}

}  // namespace
