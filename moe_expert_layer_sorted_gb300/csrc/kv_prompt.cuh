// Attention of prompts over the 4-bit cache: many rows per kv head, on the
// tcgen05 tensor cores.  Included by kv_prompt_bf16.cu and kv_prompt_f16.cu.
//
// One CTA takes 256 rows x of one sequence and kv head (x = row * (heads per
// kv head) + head, so that the heads that share keys share a tile) as two tiles
// of 128, and walks over the tokens in tiles of 128:
//   S_t = Q_t K^T   (Q, K in shared memory, S fp32 in TMEM),
//   P_t = 2^(S_t scale log2 e - m) in 16 bits over S_t's columns of TMEM,
//   O_t += P_t V    (P as the TMEM operand, V token-major in shared memory).
// The two tiles alternate: while the tensor cores work for one, the softmax
// warps work for the other.  Roles:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row (a TMEM lane);
//                   the running reference m is raised, and O rescaled in TMEM,
//                   only where a tile's weights would outgrow fp16;
//   warps 8-11      stored codes -> 16-bit K and V tiles: a thread owns a
//                   token, its code words and params loaded a tile ahead;
//   warp 12         tcgen05.mma issue, TMEM allocation.
// Rounding: k, v and P to fp16, in caches of both types, k and v from c + s (u - 8)
// by one fma on exact operands; the sums are fp32.  (bf16's 2^-9 would be seen: in a
// score of several hundred, and in P and v as much as in a bf16 output.  What is
// left shows in an fp16 output only: 4.9e-4 of its norm at scores of a standard
// deviation of 1.5, 4.5e-4 by the keys, where its own rounding is 2.1e-4.)  So that
// nothing leaves fp16's range, powers of two are taken out and put back: of a query
// row, to its largest element (back in the row's factor scale log2 e); of a token
// whose keys are all tiny or huge (back on its column, in tiles that hold one); of
// all values, 2^E with E for a tile's ordinary size; of a token whose values are far
// larger or smaller than that, another one (back in its weights, which are computed
// once for the sums and once with it).  A row's reference goes by weight times that
// power, so that a huge value that the row does not see or hardly weighs takes
// nothing from its other tokens.  (A token's groups share its power: one whose
// values are 2^16 times smaller than another's begins to lose bits.)
//
// Where there are fewer tiles of rows than half the SMs, the tokens are cut into as
// many stretches as fill them, and a second kernel joins a tile's parts, in the order
// of the stretches (one CTA would take longer over them than over its tokens).
//
// Masks: a score that its row may not see becomes -infinity.  A masked weight
// is an exact zero, but zero times a NaN value is not: values of a poisoned
// group enter the tile as zeros and its groups are remembered per row that sees
// the token.
//
// Measured (bf16, 32 query and 8 kv heads of 128 channels, groups of 64): 8,192
// rows at the end of 16,384 tokens 1,170 us, 1,410 TFLOP/s, the tensor pipe busy
// 61 % of the time.  Bound by the chain of one token tile, scores -> weights ->
// product, of which two row tiles alternate: 1.8 us a token tile where the products
// alone take 1.1; issue slots 55 %, exponents 31 %.  16 softmax warps, two threads
// a row, have too few registers (1,780 us against 1,400 before other steps); halves
// of 64 tokens, the next one's scores computed during the weights of one, need
// products of N = 64 and twice the hand-overs (1,497 us).  Three ragged prompts of
// up to 333 rows over up to 2,500 tokens (fp16, 12 heads of 64): 33 us, some ten
// token tiles one after the other, launch and join.
#pragma once

#include "kv_internal.h"

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
// weights are 2^(score - reference): the reference is set kPrDrop below the largest score and
// raised when a tile's weights sum to kPrLimit; so no weight passes 2^15 and fp16 holds those
// 2^-31 of the largest
constexpr float kPrDrop = 7.0f, kPrLimit = 32768.0f;
constexpr float kPrJoin = 0x1p-50f;  // of the stretches' weights (up to 2^40 each): their sum with values stays in range

__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The eight stored values of a word in channel order, in fp16; par: step and centre as fp16.
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t par) {
  const uint32_t s2 = __byte_perm(par, par, 0x1010), c2 = __byte_perm(par, par, 0x3232);
  return make_uint4(fma_half2(centred_pair<0>(w), s2, c2), fma_half2(centred_pair<1>(w), s2, c2),
                    fma_half2(centred_pair<2>(w), s2, c2), fma_half2(centred_pair<3>(w), s2, c2));
}

// Floats of a stretch's part: O [D / 4][row] of four channels, then references, sums, poisoned
// groups, O's powers of two.
template <int D>
constexpr int64_t kPrPart = 2 * kPrTile * (D + 4);

template <typename T, int D, int G>
__global__ void __launch_bounds__(kPrThreads, 1) kv_prompt_kernel(const __grid_constant__ PromptArgs p) {
  using Geo = KvGeom<D, G>;
  constexpr int NG = D / G;
  constexpr uint32_t kSlab = kPrTile * 128;          // 128 rows of 64 channels
  constexpr uint32_t kTileBytes = kSlab * (D / 64);  // a Q, K or V tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t kFull[2], kEmpty[2], vFull[2], vEmpty[2], sFull[2], pFull[2], qFull, oFull;
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t sh_gone;  // a wait gave up: results are wrong, the next call says so
  // per token tile (ring of 4): tokens that exist, tokens with a poisoned value, tokens with scaled keys or values
  __shared__ uint4 sh_valid[4], sh_poison[4], sh_scaled[4];
  __shared__ float sh_kscale[4][kPrTile];      // what the scaled keys' scores are multiplied by
  __shared__ float sh_vshift[4][kPrTile];      // log2 of what the scaled values' weights are multiplied by
  __shared__ int sh_vtop[4][kPrDequant];       // exponents of the tile's largest values, one per warp
  __shared__ int sh_vexp[4];                   // E from the tile on
  __shared__ float sh_qscale[2 * kPrTile];     // what a query row's scores are multiplied by
  __shared__ uint8_t sh_pgroups[4][kPrTile];   // the poisoned groups of a token
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
    auto soft_sync = [&]() { asm volatile("bar.sync 2, %0;" ::"n"(kPrSoft * 32) : "memory"); };
    // Q: both tiles, rows past the last as zeros; two threads take a row, half of its channels each
    static_assert(kPrSoft * 32 == 2 * kPrTile, "two threads per row of a tile");
#pragma unroll 1
    for (int y = 0; y < 2; ++y) {
      const int r = tid >> 1, side = tid & 1, xr = x0 + y * kPrTile + r;
      uint4 raw[D / 16];
#pragma unroll
      for (int n = 0; n < D / 16; ++n) raw[n] = make_uint4(0, 0, 0, 0);
      if (xr < nx) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + kv_row_offset(a.b, a.qs, s, q.row0, xr / p.per) +
                                                          (int64_t)(h * p.per + xr % p.per) * a.qs.head + side * (D / 2));
#pragma unroll
        for (int n = 0; n < D / 16; ++n) raw[n] = src[n];
      }
      float back = 1.0f;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        uint32_t top = 0;  // largest magnitudes of the even and the odd channels (NaN above all)
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          const uint32_t w[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
        }
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top >> 16, top & 0xffffu);
        const int ex = (int)(top >> 7) - 127;  // to 2^14; an infinity or a NaN stays what it is
        const int by = top == 0u || ex > 127 ? 0 : min(max(14 - ex, -113), 113);
        const float up = pow2(by);
        back = pow2(-by);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t w[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = KvType<__half>::pack(KvType<T>::lo(w[e]) * up, KvType<T>::hi(w[e]) * up);
          raw[n] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (side == 0) sh_qscale[y * kPrTile + r] = back;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        const int ch = side * (D / 16) + n;
        *reinterpret_cast<uint4*>(gen + y * kTileBytes + (ch / 8) * kSlab + r * 128 + ((ch % 8) ^ (r & 7)) * 16) = raw[n];
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    soft_sync();
    if (tid == 0) mbar_arrive(smem_addr(&qFull));
    const float kappa = a.scale * 1.4426950408889634f * sh_qscale[t * kPrTile + quad * 32 + lane];
    const uint64_t kappa2 = pair2(kappa, kappa);
    float m = kNone;
    uint64_t l2 = 0;        // the two halves of the row's sum
    uint32_t poisoned = 0;  // groups with a NaN value that the row sees
    int vexp = 0;           // E so far
    bool coarse = false;    // a row's scores are as large as kCoarse
    for (int j = 0; j < (t == 0 || two ? ntiles : 0); ++j) {
      kv_wait(smem_addr(&sFull[t]), (uint32_t)j & 1u, &sh_gone, p.err);
      fence_after();
      uint32_t v[2][32];  // asked for before what the tile needs is known: nearly always the unmasked pass
      tmem_ld32(ts, v[0]);
      const uint4 valid4 = sh_valid[j & 3], poison4 = sh_poison[j & 3], scaled4 = sh_scaled[j & 3];
      const bool scaled = (scaled4.x | scaled4.y | scaled4.z | scaled4.w) != 0;
      const uint32_t valid[4] = {valid4.x, valid4.y, valid4.z, valid4.w};
      const uint32_t poison[4] = {poison4.x, poison4.y, poison4.z, poison4.w};
      // a tile that every row of the warp sees in full takes no masks
      bool plain = __all_sync(0xffffffffu, seen >= (j + 1) * kPrTile) &&
                   (valid4.x & valid4.y & valid4.z & valid4.w) == 0xffffffffu && !scaled && !coarse;
      uint32_t pr[kPrTile / 2];
      auto mask_of = [&](int k) {  // tokens of the k-th 32 that the row sees
        const int n = seen - (j * kPrTile + 32 * k);
        return valid[k] & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
      };
      // the k-th 32 scores, masked ones -infinity; shifted: of the weights with their tokens' powers of two
      auto load = [&](int k, uint32_t (&v)[32], bool shifted) {
        tmem_ld32(ts + 32 * k, v);
        tmem_wait_ld();
        const uint32_t mask = mask_of(k);
        if (scaled) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * sh_kscale[j & 3][32 * k + i]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (mask >> i) & 1u ? __float_as_uint(__uint_as_float(v[i]) * kappa) : 0xff800000u;
        if (shifted) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + sh_vshift[j & 3][32 * k + i]);
        }
      };
      uint64_t sum = 0, whole = 0;  // of the weights as operands, as they are
      auto weights = [&](const uint32_t (&v)[32], int k, uint64_t factor, uint64_t neg) {
        float e[32];  // step by step over all 32: independent instructions side by side
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          split2(fma2(pair2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), factor, neg), e[i], e[i + 1]);
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i] = exp2_fast(e[i]);
        uint64_t part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) part[i] = pair2(e[2 * i], e[2 * i + 1]);
#pragma unroll
        for (int i = 8; i < 32; i += 2) part[i / 2 % 4] = add2(part[i / 2 % 4], pair2(e[i], e[i + 1]));
#pragma unroll
        for (int i = 0; i < 32; i += 2) pr[16 * k + i / 2] = KvType<__half>::pack(e[i], e[i + 1]);
        sum = add2(sum, add2(add2(part[0], part[1]), add2(part[2], part[3])));
      };
      // weights against the reference as it stands, and once more where it has to rise: for the
      // first tile, with E, or where a weight (times its token's power of two) is above the limit,
      // which shows in the sum (that may reach the limit without one: no harm)
      bool raise = j == 0 || sh_vexp[j & 3] != vexp, asked = true;
      while (true) {
        if (raise) {
          // the reference takes over what E gives up (O stays as it is) and rises to the tile's largest
          // weight times its token's power of two, within 2^60 of the weights'; the sums shrink
          float best = kNone, top = kNone;
#pragma unroll 1
          for (int k = 0; k < (scaled ? 8 : 4); ++k) {
            load(k & 3, v[0], k < 4 && scaled);
            if (k == 4) {
              top = best;  // of the shifted ones
              best = kNone;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) best = fmaxf(best, __uint_as_float(v[0][i]));
          }
          if (scaled) {
            const float t = best;
            best = top;
            top = t;
          }
          asked = false;
          float l0, l1;
          split2(l2, l0, l1);
          if (l0 + l1 > 0.0f) top = fmaxf(top, m + (float)exponent(__float_as_uint(l0 + l1)));
          const int now = sh_vexp[j & 3];
          const float cur = m + (float)(vexp - now);
          best = fmaxf(fmaxf(best - kPrDrop, top - 60.0f), cur);
          const float f = exp2_fast(m - best), fo = exp2_fast(cur - best);
          m = best;
          vexp = now;
          coarse = coarse || __any_sync(0xffffffffu, m != kNone && fabsf(m) >= kCoarse);
          plain = plain && !coarse;
          l2 = pair2(l0 * f, l1 * f);
          if (j > 0) {
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
        const uint64_t neg = pair2(-m, -m);
        sum = 0;
        if (plain) {
          if (!asked) tmem_ld32(ts, v[0]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // the next 32 scores arrive while these are worked on
            tmem_wait_ld();
            if (k < 3) tmem_ld32(ts + 32 * (k + 1), v[(k + 1) & 1]);
            weights(v[k & 1], k, kappa2, neg);
          }
        } else {
          const uint64_t one = pair2(1.0f, 1.0f);
#pragma unroll 1
          for (bool shifted = false;; shifted = true) {  // scaled values: sums by the weights, operands by the shifted
            sum = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              load(k, v[0], shifted);
              weights(v[0], k, one, neg);
            }
            if (!shifted) whole = sum;
            if (shifted || !scaled) break;
          }
        }
        if (plain) whole = sum;
        if (raise) break;
        float s0, s1;
        split2(sum, s0, s1);
        raise = __any_sync(0xffffffffu, fmaxf(s0, s1) > kPrLimit);
        if (!raise) break;
      }
      l2 = add2(l2, whole);
      tmem_st32(ts, pr);
      tmem_st32(ts + 32, pr + 32);
      if (poison[0] | poison[1] | poison[2] | poison[3]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          for (uint32_t b = poison[k] & mask_of(k); b; b &= b - 1) poisoned |= sh_pgroups[j & 3][32 * k + __ffs(b) - 1];
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
    float s0, s1;
    split2(l2, s0, s1);
    const float l = s0 + s1;
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
    const int i = x / p.per, hq = h * p.per + x % p.per;
    uint16_t* dst = has && x < nx ? a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + (int64_t)hq * a.os.head : nullptr;
    auto write = [&](int k, const uint32_t (&v)[32], float f0, float f1) {  // 32 channels, times both factors
      // the groups of a poisoned value are NaN
      if ((poisoned >> (32 * k / G)) & 1u) f0 = __int_as_float(0x7fffffff);
      uint32_t o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        o[e] = KvType<T>::pack(__uint_as_float(v[2 * e]) * f0 * f1, __uint_as_float(v[2 * e + 1]) * f0 * f1);
      if (reinterpret_cast<uintptr_t>(dst) & 31) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(dst + 32 * k + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {  // whole sectors
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * k + 2 * e), "r"(o[e]),
                       "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                       : "memory");
      }
    };
    if (splits == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is zero
      if (has) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t v[32];
          sums(k, v);
          if (dst) write(k, v, inv, pow2(vexp));
        }
      }
      if (dst && a.lse)
        a.lse[kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq] =
            l == 0.0f ? -__int_as_float(0x7f800000) : (m + log2f(l)) * 0.6931471805599453f;
    } else if (has) {  // a stretch's part
      float* part = p.ws + ((int64_t)blockIdx.x * p.splits + z) * kPrPart<D>;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t v[32];
        sums(k, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(part)[(8 * k + e) * (2 * kPrTile) + row] =
              make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      }
      float* ends = part + 2 * kPrTile * D + row;
      const int by = excess<40>(l), up = vexp - by;  // up: the power of two that goes with O
      ends[0] = m + (float)by;
      ends[2 * kPrTile] = l * pow2(-by);
      ends[4 * kPrTile] = __uint_as_float(poisoned);
      ends[6 * kPrTile] = up < -126 ? 0.0f : pow2(min(up, 127));
    }
  } else if (warp < kPrMma) {
    // ------------------------------------------------------------------ codes to K and V tiles
    set_registers<kPrRegs, kPrDequantRegs>();
    const int t = tid - kPrSoft * 32;  // token of the tile
    const int dw = warp - kPrSoft;
    uint4 kq[D / 32], vq[D / 32];
    uint32_t kp[NG], vp[NG], vpn[NG];  // params of the keys, the values, the next tile's values
    bool ok = false;       // token of the K words in hand exists
    bool okv = false;
    const uint8_t* at = nullptr;  // its block
    constexpr int kNoExp = -1000;
    int vexp = kNoExp;            // E
    int vever = kNoExp;           // exponent of the largest value so far
    int64_t pid = -1;             // page of the token one tile on
    auto page_of = [&](int j) {
      const int pos = base + j * kPrTile + t;
      pid = j < ntiles && pos < most ? kv_page(a.c, a.b, s, pos >> a.c.page_shift) : -1;
    };
    const int row = t & 15;
    const uint32_t flip = (uint32_t)((t >> 2) & 1) * (D / 4);
    auto load_k = [&](int j) {
      const int pos = base + j * kPrTile + t;
      ok = pid >= 0;
      at = a.c.pages + pid * a.c.page_stride + h * a.c.head_stride +
           ((pos & (a.c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
      if (ok) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) kq[i] = *reinterpret_cast<const uint4*>(at + row * Geo::kRow + 16 * i);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          kp[g] = *reinterpret_cast<const uint32_t*>(at + Geo::kKPar + row * Geo::kParRow + 4 * g);
          vpn[g] = *reinterpret_cast<const uint32_t*>(at + Geo::kVPar + row * Geo::kParRow + 4 * g);
        }
      }
    };
    const uint8_t* atv = nullptr;
    auto load_v = [&]() {
      if (okv) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          vq[i] = *reinterpret_cast<const uint4*>(atv + Geo::kVOff + kv_v_row(row) * Geo::kRow + ((16 * i) ^ flip));
      }
    };
    auto put = [&](uint8_t* tile, int ch, uint4 v) {  // channels ch .. ch + 7 of token t
      *reinterpret_cast<uint4*>(tile + (ch / 64) * kSlab + t * 128 + ((ch % 64 / 8) ^ (t & 7)) * 16) = v;
    };
    if (ntiles > 0) {
      page_of(0);
      load_k(0);
      page_of(1);
    }
    for (int j = 0; j < ntiles; ++j) {
      const int st = j & 1;
      const uint32_t free_parity = ((uint32_t)(j >> 1) & 1u) ^ 1u;
      // this tile's values can be asked for now: their words arrive while the keys are turned
      okv = ok;
      atv = at;
      load_v();
#pragma unroll
      for (int g = 0; g < NG; ++g) vp[g] = vpn[g];
      kv_wait(smem_addr(&kEmpty[st]), free_parity, &sh_gone, p.err);
      uint8_t* tk = gen + 2 * kTileBytes + st * kTileBytes;
      uint32_t bad = 0;  // the token's poisoned groups
      float kscale = 1.0f, vbig = 0.0f;
      int vown;  // the power of two that its values are divided by
      if (ok) {
        float kbig = 0.0f;  // bound of the token's keys
#pragma unroll
        for (int g = 0; g < NG; ++g) kbig = fmaxf(kbig, fabsf(KvType<T>::hi(kp[g])) + 8.0f * KvType<T>::lo(kp[g]));
        float to = 1.0f;
        if (!(kbig >= 0x1p-8f && kbig <= 0x1p14f) && kbig > 0.0f) {
          const int by = min(max(13 - ((int)(__float_as_uint(kbig) >> 23) - 127), -126), 126);
          to = pow2(by);
          kscale = pow2(-by);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float big = fabsf(KvType<T>::hi(vp[g])) + 8.0f * KvType<T>::lo(vp[g]);
          vbig = fmaxf(vbig, big);
          if (big != big) {
            bad |= 1u << g;
            vp[g] = 0;  // enters as zeros
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)  // params as fp16
          kp[g] = KvType<__half>::pack(KvType<T>::lo(kp[g]) * to, KvType<T>::hi(kp[g]) * to);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t w[4] = {kq[i].x, kq[i].y, kq[i].z, kq[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 4 * i + e, quarter = n / (D / 32), rest = n % (D / 32), g = rest / (G / 32);
            put(tk, g * G + quarter * (G / 4) + rest % (G / 32) * 8,
                values8(w[e], kp[g]));
          }
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < D; ch += 8) put(tk, ch, make_uint4(0, 0, 0, 0));
      }
      const uint32_t bv = __ballot_sync(0xffffffffu, ok), bp = __ballot_sync(0xffffffffu, bad != 0);
      sh_kscale[j & 3][t] = kscale;
      if (lane == 0) {
        reinterpret_cast<uint32_t*>(&sh_valid[j & 3])[dw] = bv;
        reinterpret_cast<uint32_t*>(&sh_poison[j & 3])[dw] = bp;
      }
      if (bp) sh_pgroups[j & 3][t] = (uint8_t)bad;
      // E: the tile's ordinary size (the smallest of its warps' largest values) to about 2^7, changed
      // where that would pass 2^15 or fall below 2^-1, within 2^60 of the largest value ever
      const uint32_t vtop = __reduce_max_sync(0xffffffffu, __float_as_uint(vbig));
      if (lane == 0) sh_vtop[j & 3][dw] = vtop == 0 ? kNoExp : exponent(vtop);
      asm volatile("bar.sync 1, %0;" ::"n"(kPrDequant * 32) : "memory");
      int usual = -kNoExp;
#pragma unroll
      for (int i = 0; i < kPrDequant; ++i) {
        const int e = sh_vtop[j & 3][i];
        vever = max(vever, e);
        if (e != kNoExp) usual = min(usual, e);
      }
      if (usual != -kNoExp && (vexp == kNoExp || usual > vexp + 14 || usual < vexp - 1)) vexp = usual - 7;
      if (vexp != kNoExp) vexp = min(max(vexp, max(vever - 67, -60)), 120);
      // a token whose largest value would leave that range has a power of two of its own, which
      // goes with its weights (a token without values: the smallest)
      const int e = vbig > 0.0f ? exponent(__float_as_uint(vbig)) : -126, base = vexp == kNoExp ? 0 : vexp;
      vown = e > base + 14 || e < base - 1 ? max(e - 7, base - 60) : base;
      sh_vshift[j & 3][t] = (float)(vown - base);
      const uint32_t bs = __ballot_sync(0xffffffffu, kscale != 1.0f || (ok && vown != base));
      if (lane == 0) reinterpret_cast<uint32_t*>(&sh_scaled[j & 3])[dw] = bs;
      if (t == 0) sh_vexp[j & 3] = base;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&kFull[st]));
      // the next tile's keys
      load_k(j + 1);
      page_of(j + 2);
      kv_wait(smem_addr(&vEmpty[st]), free_parity, &sh_gone, p.err);
      uint8_t* tv = gen + 4 * kTileBytes + st * kTileBytes;
      if (okv) {
        const float to = pow2(-vown);
        uint32_t w[D / 8];
#pragma unroll
        for (int g = 0; g < NG; ++g) vp[g] = KvType<__half>::pack(KvType<T>::lo(vp[g]) * to, KvType<T>::hi(vp[g]) * to);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          w[4 * i] = vq[i].x;
          w[4 * i + 1] = vq[i].y;
          w[4 * i + 2] = vq[i].z;
          w[4 * i + 3] = vq[i].w;
        }
#pragma unroll
        for (int o = 0; o < D / 8; ++o) {  // channels 8 o ..
          put(tv, 8 * o, values8(kv_v_codes<D, G>(w, o, 0), vp[8 * o / G]));
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < D; ch += 8) put(tv, ch, make_uint4(0, 0, 0, 0));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      const bool held = p.fail && blockIdx.x == 0 && z == 0 && j == ntiles - 1 && dw == 0;
      if (lane == 0 && !held) mbar_arrive(smem_addr(&vFull[st]));
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
template <typename T, int D, int G>
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ PromptArgs p) {
  const KvAttnArgs& a = p.a;
  const PromptTile tile(p);
  const int row = blockIdx.y * 32 + (threadIdx.x & 31);
  const int x = tile.x0 + row;
  if (x >= tile.nx || tile.splits == 1) return;
  const float* parts = p.ws + (int64_t)blockIdx.x * p.splits * kPrPart<D>;
  const float* ends = parts + 2 * kPrTile * D + row;
  float m = kNone, l = 0.0f;
  uint32_t poisoned = 0;
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) m = fmaxf(m, __ldcg(ends + y * kPrPart<D>));
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) {
    l = fmaf(exp2_fast(__ldcg(ends + y * kPrPart<D>) - m) * kPrJoin, __ldcg(ends + y * kPrPart<D> + 2 * kPrTile), l);
    poisoned |= __float_as_uint(__ldcg(ends + y * kPrPart<D> + 4 * kPrTile));
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is zero
  const int i = x / p.per, hq = tile.h * p.per + x % p.per;
  uint16_t* dst = a.out + kv_row_offset(a.b, a.os, tile.s, tile.q.row0, i) + (int64_t)hq * a.os.head;
  constexpr int kQuads = D / 4 / 8;  // of four channels, per thread
  float4 o[kQuads];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int y = 0; y < tile.splits; ++y) {
    const float f = exp2_fast(__ldcg(ends + y * kPrPart<D>) - m) * kPrJoin * __ldcg(ends + y * kPrPart<D> + 6 * kPrTile);
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int d4 = (threadIdx.x >> 5) * kQuads + k;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(parts + y * kPrPart<D>) + d4 * (2 * kPrTile) + row);
      o[k].x = fmaf(f, v.x, o[k].x);
      o[k].y = fmaf(f, v.y, o[k].y);
      o[k].z = fmaf(f, v.z, o[k].z);
      o[k].w = fmaf(f, v.w, o[k].w);
    }
  }
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int d4 = (threadIdx.x >> 5) * kQuads + k;
    const float f = (poisoned >> (4 * d4 / G)) & 1u ? __int_as_float(0x7fffffff) : inv;
    *reinterpret_cast<uint2*>(dst + 4 * d4) =
        make_uint2(KvType<T>::pack(o[k].x * f, o[k].y * f), KvType<T>::pack(o[k].z * f, o[k].w * f));
  }
  if (a.lse && threadIdx.x < 32)
    a.lse[kv_row_index(a.b, tile.s, tile.q.row0, i) * a.q_heads + hq] =
        l == 0.0f ? -__int_as_float(0x7f800000) : (m + log2f(l * (1.0f / kPrJoin))) * 0.6931471805599453f;
}

template <typename T, int D, int G>
cudaError_t launch_prompt(const PromptArgs& p, unsigned ctas, cudaStream_t s) {
  const size_t smem = 1024 + (size_t)6 * kPrTile * D * 2;
  const auto kernel = kv_prompt_kernel<T, D, G>;
  static const bool registers_fit = brings_registers(reinterpret_cast<const void*>(kernel), kPrRegs);
  if (!registers_fit) return cudaErrorInvalidKernelImage;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(ctas, (unsigned)p.splits), kPrThreads, smem, s>>>(p);
  if (p.splits > 1) kv_join_kernel<T, D, G><<<dim3(ctas, 2 * kPrTile / 32), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t prompt(Kv& kv, const KvAttnArgs& a, cudaStream_t s) {
  PromptArgs p{a, a.q_heads / a.c.heads, 0, 1, kv.parts(), kv.err_dev, kv.fail_next};
  const int64_t tiles = ((int64_t)a.b.max_new * p.per + 2 * kPrTile - 1) / (2 * kPrTile);
  const int64_t ctas = tiles * a.c.heads * a.b.batch;
  if (ctas > 0x7fffffff || (int64_t)a.c.heads * a.b.batch > 0x7fffffff || tiles * 2 * kPrTile > 0x7fffffff)
    return cudaErrorInvalidConfiguration;
  p.tiles = (int)tiles;
  // the SMs hold one CTA each; the parts have to fit the workspace
  const int64_t slots = Kv::kPartsBytes / (2 * kPrTile * (kv.d.head_dim + 4) * sizeof(float));
  p.splits = (int)std::max<int64_t>(std::min<int64_t>(kv.sms, slots) / ctas, 1);
  cudaError_t e = cudaErrorInvalidValue;
  const int dg = kv.d.head_dim * 1000 + kv.d.group_size;
#define KV_CASE(DD, GG) \
  if (dg == DD * 1000 + GG) e = launch_prompt<T, DD, GG>(p, (unsigned)ctas, s);
  KV_CASE(64, 32)
  KV_CASE(64, 64)
  KV_CASE(128, 32)
  KV_CASE(128, 64)
  KV_CASE(128, 128)
#undef KV_CASE
  return e;
}

}  // namespace
