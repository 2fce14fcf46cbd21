// Attention of few rows over the 4-bit cache: a decode step's single tokens, a
// few speculated tokens, or any number of rows that each chose pages of their
// own.  Included by kv_decode_bf16.cu and kv_decode_f16.cu, one type each.
//
// Mathematics.  For the columns (row, query head) that share a kv head, the
// scores of 16 tokens are S^T = K q^T on the tensor cores with the tokens as
// the 16 rows of mma.m16n8k16 and up to 8 columns as its n, so a group of
// query heads costs what one head costs.  The operand is the code itself, not
// the stored value: with stored value c + s (u - 8) per token and group,
//     S[t][col] = sum over groups g of  s_g (u - 8)_g . q_g + c_g sum(q_g),
// the products are exact, and s and c enter in fp32 on the accumulators.
// (bf16 takes 128 + u, one mask, and corrects by 136 sum(q_g) s_g; fp16, whose
// 1024 + u would cost three more bits of the accumulator, takes u - 8.)
// O^T = V^T P^T is the second product, the channels as rows: P s_g per group is
// rounded to 16 bits (the one rounding before the output's: relative 2^-9 or
// 2^-12 of a weight, independent from token to token), u - 8 is exact, and the
// centres' part sum over t of P c_g is summed apart in fp32.
//
// Softmax: running reference per column, raised only when a score exceeds it by
// more than kSlack, so that most blocks rescale nothing; weights are at most
// 2^kSlack and the sums are fp32.  A column that sees no token keeps the sum 0.
//
// Work split: all blocks (16 tokens of one kv head and column tile) of the
// batch in one line, cut into equal runs, one per CTA; a run covers any number
// of items (sequence, head, column tile) or part of one.  Warp w of 8 takes
// every eighth block of the run through a ring of its own, each block one bulk
// copy.  At the end of an item's stretch the warps' (max, sum, O) are joined in
// shared memory; an item cut between CTAs is joined by the CTA that finishes
// last, in the order of the CTAs, so results do not depend on timing.
#pragma once

#include "kv_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"

constexpr int kDecWarps = 8;

// What the work is divided into.  A unit is 16 tokens of an item; an item is a
// (group, head, column tile); a group is a sequence, or with chosen pages one
// of its rows.  Unit numbers run over the groups, inside them over the items,
// inside them over the tokens.
struct DecPlan {
  int groups;     // sequences, or batch * max_new rows
  int items;      // items per group: heads * column tiles
  int ctiles;     // column tiles
  int per;        // query heads per kv head
  int min_units;  // a CTA's share is not made smaller than this
};

__device__ __forceinline__ int group_units(const KvAttnArgs& a, int gi) {
  if (a.sel) {
    const int s = gi / a.b.max_new, i = gi % a.b.max_new;
    return i < kv_seq(a.b, s).rows ? a.budget << (a.c.page_shift - 4) : 0;
  }
  const KvSeq q = kv_seq(a.b, gi);
  return q.rows > 0 ? (min(q.len, kv_capacity(a.c, a.b)) + 15) >> 4 : 0;
}

// First CTA whose share [total c / n, total (c + 1) / n) holds unit u.
__device__ __forceinline__ int owner(int64_t u, int64_t total, int n) { return (int)(((u + 1) * n - 1) / total); }

// A place in the line of units.
struct Cursor {
  int group;           // its group
  int64_t base, end;   // units of the group
  int units;           // units of each of the group's items
  // the current item
  int64_t item0, item_end;
  int item;

  __device__ __forceinline__ void enter(const KvAttnArgs& a, const DecPlan& p, int64_t u) {
    while (u >= end) {
      base = end;
      units = group_units(a, ++group);
      end = base + (int64_t)units * p.items;
    }
    item = (int)((u - base) / units);
    item0 = base + (int64_t)item * units;
    item_end = item0 + units;
  }
};

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(kDecWarps * 32, NT == 1 ? 2 : 1)
    kv_decode_kernel(KvAttnArgs a, DecPlan p, float* __restrict__ ws, unsigned* __restrict__ counters, uint32_t* err) {
  using Geo = KvGeom<D, G>;
  using F = Frag<T>;
  constexpr int C = 8 * NT, NG = D / G;
  constexpr int kStages = kDecStages<D, G>;
  constexpr int kSlot = C * (D + 2);  // floats of one partial result: O [C][D], max [C], sum [C]
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;                                                         // [warp][stage][block]
  float* mo = reinterpret_cast<float*>(smem + kDecWarps * kStages * Geo::kBytes);  // [warp][C][D + 4]
  float* mm = mo + kDecWarps * C * (D + 4);                                     // [warp][C] max, then sums
  float* ml = mm + kDecWarps * C;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + kDecWarps * C);             // [warp][stage]
  int* spos = reinterpret_cast<int*>(bars + kDecWarps * kStages);               // [warp][stage] position of a block, -1: none
  __shared__ int64_t sh_sum[kDecWarps];
  __shared__ int64_t sh_base;
  __shared__ int sh_group;
  __shared__ unsigned sh_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;

  if (lane < kStages) mbar_init(smem_addr(&bars[warp * kStages + lane]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // ---- the CTA's share: the sum of all units, then the group its first unit lies in
  auto block_sum = [&](int64_t v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) sh_sum[warp] = v;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) s += sh_sum[w];
    return s;
  };
  int64_t total = 0;
  for (int g0 = 0; g0 < p.groups; g0 += kDecWarps * 32) {
    const int gi = g0 + tid;
    total += block_sum(gi < p.groups ? (int64_t)group_units(a, gi) * p.items : 0);
  }
  // rows that see nothing at all (no unit in their group) are written by the last loop below
  const int n = (int)min((int64_t)gridDim.x, max((total + p.min_units - 1) / p.min_units, (int64_t)1));
  const int me = blockIdx.x;
  const int64_t first = me < n ? total * me / n : total, last = me < n ? total * (me + 1) / n : total;
  if (first < last) {
    int64_t before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kDecWarps * 32) {  // the group that holds unit `first`
      const int gi = g0 + tid;
      const int64_t v = gi < p.groups ? (int64_t)group_units(a, gi) * p.items : 0;
      int64_t x = v;  // inclusive prefix over the CTA
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) sh_sum[warp] = x;
      __syncthreads();
      int64_t all = 0;
      for (int w = 0; w < kDecWarps; ++w) {
        if (w < warp) x += sh_sum[w];
        all += sh_sum[w];
      }
      if (before + x - v <= first && first < before + x) {
        sh_group = gi;
        sh_base = before + x - v;
      }
      before += all;
      if (before > first) break;
    }
    __syncthreads();
    Cursor seed;
    seed.group = sh_group - 1;
    seed.end = sh_base;

    // ---- the producer side: this warp's units first + warp, + 8, ...
    Cursor pc = seed;
    int64_t pu = first + warp;
    int64_t pid = -1;       // page of unit pu (requested one step ahead of its copy)
    int ppos = -1, pblk = 0;  // its position in the sequence (-1: nothing to read), its block of the page
    pc.item_end = 0;
    auto locate = [&]() {
      if (pu >= last) return;
      if (pu >= pc.item_end) pc.enter(a, p, pu);
      const int ub = (int)(pu - pc.item0);
      const int per_page = a.c.page_shift - 4;
      int j = ub >> per_page;
      pblk = ub & ((1 << per_page) - 1);
      int s = pc.group;
      if (a.sel) {
        s = pc.group / a.b.max_new;
        const KvSeq q = kv_seq(a.b, s);
        const int i = pc.group % a.b.max_new;
        const int64_t row = kv_row_index(a.b, s, q.row0, i);
        j = a.sel[(row * a.c.heads + pc.item / p.ctiles) * a.budget + j];
        const int64_t seen = min(a.causal ? (int64_t)q.len - q.rows + i + 1 : (int64_t)q.len, (int64_t)kv_capacity(a.c, a.b));
        const int64_t pos = ((int64_t)j << a.c.page_shift) + 16 * pblk;
        ppos = j >= 0 && pos < seen ? (int)pos : -1;
        if (ppos < 0) j = 0;
      } else {
        ppos = ub * 16;
      }
      pid = kv_page(a.c, a.b, s, j);
    };
    auto issue = [&](int slot) {
      if (pu >= last) return;
      if (lane == 0) {
        const bool ok = ppos >= 0 && pid >= 0;
        spos[warp * kStages + slot] = ok ? ppos : -1;
        if (ok) {
          const uint32_t bar = smem_addr(&bars[warp * kStages + slot]);
          mbar_arrive_expect_tx(bar, Geo::kBytes);
          bulk_g2s(smem_addr(ring + (size_t)(warp * kStages + slot) * Geo::kBytes),
                   a.c.pages + pid * a.c.page_stride + (pc.item / p.ctiles) * a.c.head_stride + (int64_t)pblk * Geo::kBytes,
                   Geo::kBytes, bar);
        }
      }
      pu += kDecWarps;
      locate();
    };
    locate();
#pragma unroll 1
    for (int q = 0; q < kStages; ++q) issue(q);
    int slot = 0;
    uint32_t phases = 0;  // bit q: the parity slot q's next copy completes

    Cursor cc = seed;
    int64_t cu = first + warp;  // this warp's next unit
    for (int64_t seg = first; seg < last;) {
      cc.enter(a, p, seg);
      const int64_t seg_end = min(cc.item_end, last);
      // ---- the item's columns
      int s = cc.group, row_lo = 0, ncols;
      const int h = cc.item / p.ctiles, ct = cc.item % p.ctiles;
      if (a.sel) {
        s = cc.group / a.b.max_new;
        row_lo = cc.group % a.b.max_new;
      }
      const KvSeq q = kv_seq(a.b, s);
      ncols = (a.sel ? 1 : q.rows) * p.per;
      const int cap = kv_capacity(a.c, a.b);
      auto col_seen = [&](int col) {  // tokens that column `col` of the tile sees
        const int x = ct * C + col;
        if (x >= ncols) return 0x7fffffff;  // a column of nobody: zeros times anything, never written
        const int64_t pos = (int64_t)q.len - q.rows + row_lo + x / p.per;
        return (int)min(max(a.causal ? pos + 1 : (int64_t)q.len, (int64_t)0), (int64_t)cap);
      };
      uint32_t qf[NT][D / 8];   // this lane's query operand: column 8 nt + r, its quarter of every group
      float qsum[NT][NG][2];    // sums over a group's channels, columns 8 nt + 2c, + 1 (times scale log2 e)
      int seen[NT][2];
      const float kappa = a.scale * 1.4426950408889634f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int x = ct * C + nt * 8 + r;
        const uint16_t* src = nullptr;
        if (x < ncols)
          src = a.q + kv_row_offset(a.b, a.qs, s, q.row0, row_lo + x / p.per) + (int64_t)(h * p.per + x % p.per) * a.qs.head;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const int ch = w / (G / 32) * G + c * (G / 4) + w % (G / 32) * 8;
          const uint4 v = src ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0, 0, 0, 0);
          qf[nt][4 * w] = v.x;
          qf[nt][4 * w + 1] = v.y;
          qf[nt][4 * w + 2] = v.z;
          qf[nt][4 * w + 3] = v.w;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float t = 0.0f;
#pragma unroll
          for (int i = g * (G / 8); i < (g + 1) * (G / 8); ++i) t += KvType<T>::lo(qf[nt][i]) + KvType<T>::hi(qf[nt][i]);
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);  // column 8 nt + r
#pragma unroll
          for (int e = 0; e < 2; ++e) qsum[nt][g][e] = kappa * __shfl_sync(0xffffffffu, t, 4 * (2 * c + e));
        }
        seen[nt][0] = col_seen(nt * 8 + 2 * c);
        seen[nt][1] = col_seen(nt * 8 + 2 * c + 1);
      }
      int least = seen[0][0];  // blocks that end by here need no mask
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) least = min(least, min(seen[nt][0], seen[nt][1]));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));

      float acc[D / 16][NT][4];  // O^T: channel tiles by columns
      float oc[NT][NG][2];       // this lane's tokens' part of sum P c
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = kNone;
          l[nt][e] = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) oc[nt][g][e] = 0.0f;
        }
      }

      for (; cu < seg_end; cu += kDecWarps) {
        __syncwarp();
        const int pos = *reinterpret_cast<volatile int*>(&spos[warp * kStages + slot]);
        if (pos >= 0) {
          const uint32_t bar = smem_addr(&bars[warp * kStages + slot]);
          if (!mbar_wait(bar, (phases >> slot) & 1u, err)) mbar_drain(bar, (phases >> slot) & 1u);
          phases ^= 1u << slot;
          const uint8_t* blk = ring + (size_t)(warp * kStages + slot) * Geo::kBytes;
          // ---- scores of tokens r and r + 8, columns 2c and 2c + 1
          uint32_t kw[2][D / 32];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* src = blk + (r + 8 * e) * Geo::kRow + c * (D / 8);
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              kw[e][0] = v.x, kw[e][1] = v.y, kw[e][2] = v.z, kw[e][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              kw[e][0] = v.x, kw[e][1] = v.y;
            }
          }
          float sc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float d[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) d[nt][e] = 0.0f;
#pragma unroll
            for (int w = g * (G / 32); w < (g + 1) * (G / 32); ++w) {
              const uint32_t a0[4] = {F::template key<0>(kw[0][w]), F::template key<0>(kw[1][w]),
                                      F::template key<1>(kw[0][w]), F::template key<1>(kw[1][w])};
              const uint32_t a1[4] = {F::template key<2>(kw[0][w]), F::template key<2>(kw[1][w]),
                                      F::template key<3>(kw[0][w]), F::template key<3>(kw[1][w])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                F::mma(d[nt], a0, qf[nt][4 * w], qf[nt][4 * w + 1]);
                F::mma(d[nt], a1, qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t par = *reinterpret_cast<const uint32_t*>(blk + Geo::kKPar + (r + 8 * e) * Geo::kParRow + 4 * g);
              const float ks = KvType<T>::lo(par), kc = fmaf(-F::kOffset, ks, KvType<T>::hi(par)), kk = ks * kappa;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  sc[nt][2 * e + x] = fmaf(kk, d[nt][2 * e + x], fmaf(kc, qsum[nt][g][x], sc[nt][2 * e + x]));
            }
          }
          if (pos + 16 > least) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (pos + r + 8 * (e >> 1) >= seen[nt][e & 1]) sc[nt][e] = -__int_as_float(0x7f800000);
          }
          // ---- the reference, raised where a score is far above it
          bool raise = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) raise |= fmaxf(sc[nt][x], sc[nt][2 + x]) > m[nt][x] + F::kSlack;
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float t = fmaxf(sc[nt][x], sc[nt][2 + x]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                t = fmaxf(t + F::kLift, m[nt][x]);
                const float f = exp2_fast(m[nt][x] - t);
                m[nt][x] = t;
                l[nt][x] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) oc[nt][g][x] *= f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  acc[j][nt][x] *= f;
                  acc[j][nt][2 + x] *= f;
                }
              }
          }
          // ---- weights, their sums, and P s as the second product's operand
          uint32_t pf[NT][NG][2];
          float vs[2][NG], vc[2][NG];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const uint32_t par = *reinterpret_cast<const uint32_t*>(blk + Geo::kVPar + (r + 8 * e) * Geo::kParRow + 4 * g);
              vs[e][g] = KvType<T>::lo(par);
              vc[e][g] = KvType<T>::hi(par);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[e] = exp2_fast(sc[nt][e] - m[nt][e & 1]);
            l[nt][0] += pr[0] + pr[2];
            l[nt][1] += pr[1] + pr[3];
            // a masked token's weight is 0, but its params may be anything: not multiplied
            const bool part = pos + 16 > least;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              float y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[e] = pr[e] * vs[e >> 1][g];
                float z = pr[e] * vc[e >> 1][g];
                if (part && pos + r + 8 * (e >> 1) >= seen[nt][e & 1]) y[e] = z = 0.0f;
                oc[nt][g][e & 1] += z;
              }
              pf[nt][g][0] = transpose8x8(KvType<T>::pack(y[0], y[1]));
              pf[nt][g][1] = transpose8x8(KvType<T>::pack(y[2], y[3]));
            }
          }
          // ---- O^T += V^T P^T
          const uint8_t* vb = blk + Geo::kVOff + c * Geo::kRow;
          const int piece = (r ^ ((c >> 1) << 2)) * (D / 16);
          uint32_t vw[4][D / 64];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint8_t* src = vb + t * 4 * Geo::kRow + piece;
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              vw[t][0] = v.x, vw[t][1] = v.y;
            } else {
              vw[t][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const uint32_t lo0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), hi0 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
            const uint32_t lo1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), hi1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
            auto tile = [&](auto k_) {
              constexpr int K = decltype(k_)::value;
              const uint32_t av[4] = {F::template value<K>(lo0), F::template value<K>(hi0), F::template value<K>(lo1),
                                      F::template value<K>(hi1)};
              const int j = 4 * w + K, g = j / (G / 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) F::mma(acc[j][nt], av, pf[nt][g][0], pf[nt][g][1]);
            };
            tile(std::integral_constant<int, 0>());
            tile(std::integral_constant<int, 1>());
            tile(std::integral_constant<int, 2>());
            tile(std::integral_constant<int, 3>());
          }
        }
        __syncwarp();  // every lane is done with the slot
        issue(slot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
      }

      // ---- join the warps: O of this warp with its centres' part, then all of them
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int col = nt * 8 + 2 * c + x;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], o);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) oc[nt][g][x] += __shfl_xor_sync(0xffffffffu, oc[nt][g][x], o);
          if (r == 0) {
            mm[warp * C + col] = m[nt][x];
            ml[warp * C + col] = l[nt][x];
          }
          float* dst = mo + (warp * C + col) * (D + 4);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const int g = j / (G / 16), ch = g * G + r * (G / 8) + 2 * j % (G / 8);
            *reinterpret_cast<float2*>(dst + ch) = make_float2(acc[j][nt][x] + oc[nt][g][x], acc[j][nt][2 + x] + oc[nt][g][x]);
          }
        }
      __syncthreads();
      const bool whole = seg == cc.item0 && seg_end == cc.item_end;
      // partial results: a CTA's first stretch in slot 0, its last in slot 1
      float* part = ws + (int64_t)(2 * me + (seg == first ? 0 : 1)) * kSlot;
      auto finish = [&](int col, int d4, float4 o, float M, float L) {  // four channels of a column
        const int x = ct * C + col;
        if (x >= ncols) return;
        const int i = row_lo + x / p.per, hq = h * p.per + x % p.per;
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;  // a row that sees nothing is zero
        *reinterpret_cast<uint2*>(a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + (int64_t)hq * a.os.head + 4 * d4) =
            make_uint2(KvType<T>::pack(o.x * inv, o.y * inv), KvType<T>::pack(o.z * inv, o.w * inv));
        if (a.lse && d4 == 0)
          a.lse[kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq] =
              L == 0.0f ? -__int_as_float(0x7f800000) : (M + log2f(L)) * 0.6931471805599453f;
      };
      for (int x = tid; x < C * (D / 4); x += kDecWarps * 32) {
        const int col = x / (D / 4), d4 = x % (D / 4);
        float M = mm[col];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) M = fmaxf(M, mm[w * C + col]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float L = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float f = exp2_fast(mm[w * C + col] - M);
          const float4 v = *reinterpret_cast<const float4*>(mo + (w * C + col) * (D + 4) + 4 * d4);
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
          L = fmaf(f, ml[w * C + col], L);
        }
        if (whole) {
          finish(col, d4, o, M, L);
        } else {
          reinterpret_cast<float4*>(part)[x] = o;
          if (d4 == 0) {
            part[C * D + col] = M;
            part[C * D + C + col] = L;
          }
        }
      }
      if (!whole) {  // the CTA that finishes the item last joins its parts
        const int c0 = owner(cc.item0, total, n), c1 = owner(cc.item_end - 1, total, n);
        __threadfence();
        __syncthreads();
        if (tid == 0) sh_last = atomicAdd(&counters[c0], 1u);
        __syncthreads();
        if (sh_last == (unsigned)(c1 - c0)) {
          __threadfence();
          // the item began c0's last stretch: its only one if the item begins c0's share
          const int head = 2 * c0 + (cc.item0 == total * c0 / n ? 0 : 1);
          for (int x = tid; x < C * (D / 4); x += kDecWarps * 32) {
            const int col = x / (D / 4), d4 = x % (D / 4);
            float M = kNone, L = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int y = c0; y <= c1; ++y) M = fmaxf(M, __ldcg(ws + (int64_t)(y == c0 ? head : 2 * y) * kSlot + C * D + col));
#pragma unroll 4
            for (int y = c0; y <= c1; ++y) {
              const float* src = ws + (int64_t)(y == c0 ? head : 2 * y) * kSlot;
              const float f = exp2_fast(__ldcg(src + C * D + col) - M);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + x);
              o.x = fmaf(f, v.x, o.x);
              o.y = fmaf(f, v.y, o.y);
              o.z = fmaf(f, v.z, o.z);
              o.w = fmaf(f, v.w, o.w);
              L = fmaf(f, __ldcg(src + C * D + C + col), L);
            }
            finish(col, d4, o, M, L);
          }
          if (tid == 0) counters[c0] = 0;  // for the next call
        }
      }
      __syncthreads();  // the merge buffer is free
      seg = seg_end;
    }
  }

  // ---- groups without a unit: their rows see nothing
  for (int gi = me; gi < p.groups; gi += gridDim.x) {
    if (group_units(a, gi)) continue;
    const int s = a.sel ? gi / a.b.max_new : gi;
    const KvSeq q = kv_seq(a.b, s);
    const int lo = a.sel ? gi % a.b.max_new : 0, hi = a.sel ? min(lo + 1, q.rows) : q.rows;
    for (int i = lo; i < hi; ++i)
      for (int x = tid; x < a.q_heads * (D / 8); x += kDecWarps * 32) {
        const int hq = x / (D / 8);
        *reinterpret_cast<uint4*>(a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + (int64_t)hq * a.os.head + 8 * (x % (D / 8))) =
            make_uint4(0, 0, 0, 0);
        if (a.lse && x % (D / 8) == 0) a.lse[kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq] = -__int_as_float(0x7f800000);
      }
  }
}

template <typename T, int D, int G, int NT>
cudaError_t launch_decode(Kv& kv, const KvAttnArgs& a, const DecPlan& p, cudaStream_t s) {
  constexpr int C = 8 * NT;
  const size_t smem = (size_t)kDecWarps * kDecStages<D, G> * (KvGeom<D, G>::kBytes + 12) +
                      (size_t)kDecWarps * C * (D + 6) * sizeof(float);
  const auto kernel = kv_decode_kernel<T, D, G, NT>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv.sms * (NT == 1 ? 2 : 1), Kv::kMaxParts);
  static_assert((size_t)C * (D + 2) * sizeof(float) <= Kv::kPartBytes, "partial results fit their slots");
  kernel<<<grid, kDecWarps * 32, smem, s>>>(a, p, kv.parts(), kv.counters(), kv.err_dev);
  return cudaGetLastError();
}

template <typename T>
cudaError_t decode(Kv& kv, const KvAttnArgs& a, cudaStream_t s) {
  const int64_t groups = a.sel ? (int64_t)a.b.batch * a.b.max_new : a.b.batch;
  if (groups > 0x7fffffff) return cudaErrorInvalidConfiguration;
  DecPlan p;
  p.per = a.q_heads / a.c.heads;
  const int64_t cols = (int64_t)p.per * (a.sel ? 1 : a.b.max_new);
  const int nt = cols > 8 ? 2 : 1;
  p.groups = (int)groups;
  p.ctiles = (int)((cols + 8 * nt - 1) / (8 * nt));
  if ((int64_t)p.ctiles * a.c.heads > 0x7fffffff) return cudaErrorInvalidConfiguration;
  p.items = p.ctiles * a.c.heads;
  p.min_units = 8;
  cudaError_t e = cudaErrorInvalidValue;
  const int dg = kv.d.head_dim * 1000 + kv.d.group_size;
#define KV_CASE(DD, GG)                                                        \
  if (dg == DD * 1000 + GG)                                                    \
    e = nt == 1 ? launch_decode<T, DD, GG, 1>(kv, a, p, s) : launch_decode<T, DD, GG, 2>(kv, a, p, s);
  KV_CASE(64, 32)
  KV_CASE(64, 64)
  KV_CASE(128, 32)
  KV_CASE(128, 64)
  KV_CASE(128, 128)
#undef KV_CASE
  return e;
}

}  // namespace
