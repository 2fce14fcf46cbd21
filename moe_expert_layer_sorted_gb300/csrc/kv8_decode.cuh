// Attention of few rows over the 8-bit cache: a decode step's single tokens or a few
// speculated ones.  Included by kv8_decode_bf16.cu and kv8_decode_f16.cu, one type each.
//
// Mathematics.  For the columns (row, query head) that share a kv head, the scores
// of 16 tokens are S^T = U q^T on the tensor cores, the block's codes u as the 16
// rows of mma.m16n8k16 (exact in fp16) and up to 8 columns as its n, with q as fp16
// times a power of two that brings its largest element to 2^14; in log2 units
//     y[t][col] = S^T[t][col] (scale log2 e 2^-by[col]) s_K[block],  fp32.
// O^T = U_V^T P^T is the second product, the channels as rows, with weights times
// the block's step of the values as fp16 operands:
//     p^ = 2^(y + log2 s_V - rz),  rounded to 11 bits (the one rounding before the
// output's, independent from token to token).  Two references per column: ry of the
// sum of weights 2^(y - ry), and rz of the weights times steps, so that values of any
// size beside each other take nothing from the sum, nor weights from the values.
// They are raised only where a block passes them far (by 2^60, by 2^12), and rz is
// lowered where it is 2^8 above all of a block: a token that takes most of a row's weight may
// have next to no value (a block's step says nothing of a single token of it), and the
// result is then the others'.  Hardly any block rescales anything.
//
// Work split: as in the 4-bit cache's kernel (kv_rounds.cuh), rounds of 8 blocks of 16
// tokens cut into equal shares, one per CTA; each warp takes one block of a round and
// fetches it itself, with one bulk copy into a ring of its own some blocks ahead: no
// warp waits for another before an item's end, and no barrier says that a slot is
// free.  At the end of an item's stretch the warps' (ry, sum, rz, O) are joined in the
// slots of the blocks that they have just used; an item cut between CTAs is joined by
// the CTA that finishes last, in the order of the CTAs, so results do not depend on
// timing.
//
// Measured (8 kv heads of 128 channels): 64 sequences of up to 8,191 tokens, 32 query heads, bf16: 115 us, 5.7 TB/s,
// 0.85 of the measured copy rate (112 with an rz that only rises); 2 of 131,072, 64 query heads, fp16: 94 us, 5.7 TB/s; one of 777: 12 us.  Bound by
// the memory, and some 12 us of launch, shares, first round and joins (one token of 2,048 takes 13 us, 64 sequences of
// 2,048 59).  A block takes about 200 instructions where the memory's rate leaves 700 issue slots, so that codes
// can be turned to exact fp16 numbers one by one.  Shares of at least 2 or 4 rounds: one sequence of 777 tokens
// 15.3 and 17.8 us, of 4,096 14.2 and 14.8 (against 15.1), of 16,384 20.7 and 18.8 (against 21.0).
#pragma once

#include "kv8_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"
#include "kv_rounds.cuh"

constexpr int kDec8Threads = kDecWarps * 32;
constexpr int kDec8MaxParts = 304;        // CTAs, so parts of an item
constexpr float kRaiseSum = 60.0f, kRaiseProduct = 12.0f;  // weights reach 2^60, weights times steps 2^12
constexpr float kNoProduct = 1e38f;       // ry - rz of a column that has seen no value
// rz is lowered where a block's largest weight times step is below 2^kLower (fp16's last place below 2^-14 is 2^-24: of such a
// block all sixteen together are off by 2^-13 of the largest), by no more than kLowerMost since it was raised, which keeps O
// within fp32; what is 2^kGone below rz is left alone, as are the last eight of kLowerMost.
constexpr float kLower = -8.0f, kLowerMost = 56.0f, kGone = -64.0f;

// Slots of a warp's ring: two CTAs share an SM for 8 columns, one takes it for 16 (whose O takes two slots).
template <int NT>
constexpr int kDec8Slots = NT == 1 ? 3 : 6;
// Bytes of a slot: a block, the O of 8 columns, or the references and sums of an eighth of an item's parts.
template <int D>
constexpr int kDec8Slot = D == 128 ? Kv8Geom<D>::kBytes : 2560;

// W: references, sums and scores are written down too.
template <typename T, int D, int NT, bool W>
__global__ void __launch_bounds__(kDec8Threads, NT == 1 ? 2 : 1)
    kv8_decode_kernel(const __grid_constant__ KvAttnArgs a, const __grid_constant__ DecPlan p, float* __restrict__ ws,
                      unsigned* __restrict__ counters, uint32_t* err, const __grid_constant__ Kv8Scores scores) {
  using Geo = Kv8Geom<D>;
  constexpr int C = 8 * NT, S = kDec8Slots<NT>;
  constexpr int kPart = C * (D + 2);  // floats of one partial result: O [C][D], max [C], sum [C]
  constexpr int kSlot = kDec8Slot<D>;
  constexpr int kParts = kDec8MaxParts / NT;
  static_assert(Geo::kBytes <= kSlot && 8 * D * 4 <= kSlot && (kParts + 7) / 8 * 2 * C * 4 <= kSlot && kSlot % 16 == 0, "what a slot holds");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kDecWarps * S];
  __shared__ int sh_sum[kDecWarps], sh_base, sh_group;
  __shared__ Item sh_item;
  __shared__ unsigned sh_last;
  __shared__ uint32_t sh_gone;  // a wait gave up: results are wrong, the next call says so
  __shared__ float mm[kDecWarps * C], ml[kDecWarps * C], mz[kDecWarps * C];  // references and sums
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * S * kSlot;

  if (tid == 0) sh_gone = 0;
  if (lane < S) mbar_init(smem_addr(&full[warp * S + lane]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // ---- the CTA's share: the sum of all rounds, and the group its first round lies in
  auto scan = [&](int v, int& all) {  // inclusive prefix over the CTA's threads, and the sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) sh_sum[warp] = v;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) v += sh_sum[w];
      all += sh_sum[w];
    }
    return v;
  };
  int total = 0, mine = 0, upto = 0;  // the last groups' (for up to kDec8Threads groups: the only) prefix
  for (int g0 = 0; g0 < p.groups; g0 += kDec8Threads) {
    const int gi = g0 + tid;
    int all;
    mine = gi < p.groups ? group_rounds(a, gi) * p.items : 0;
    upto = scan(mine, all);
    total += all;
  }
  const int n = max(min((int)gridDim.x, (total + p.min_rounds - 1) / p.min_rounds), 1);
  const int me = blockIdx.x;
  const int first = me < n ? share(total, me, n) : total, last = me < n ? share(total, me + 1, n) : total;
  if (first < last) {
    if (p.groups <= kDec8Threads) {
      if (upto - mine <= first && first < upto) {
        sh_group = tid;
        sh_base = upto - mine;
      }
    } else {
      int before = 0;
      for (int g0 = 0; g0 < p.groups && before <= first; g0 += kDec8Threads) {
        const int gi = g0 + tid;
        int all;
        mine = gi < p.groups ? group_rounds(a, gi) * p.items : 0;
        upto = before + scan(mine, all);
        if (upto - mine <= first && first < upto) {
          sh_group = gi;
          sh_base = upto - mine;
        }
        before += all;
      }
    }
    __syncthreads();
    const Cursor seed{sh_group - 1, sh_base, 0, 0, 0, 0};

    // ---- fetching: this warp's block of round f goes to the next slot; the page of its block one round on is asked for
    Cursor pc = seed;
    const int32_t* table = nullptr;
    int visible = 0;               // positions from here on are not read
    int64_t head_off = 0;
    int f = first, fpos = -1, fpid = -1;  // the round to fetch, its block's position and page
    auto look = [&]() {
      fpos = fpid = -1;
      if (f >= last) return;
      if (f >= pc.item_end) {
        pc.enter(a, p, f);
        const KvSeq q = kv_seq(a.b, pc.group);
        visible = min(q.len, kv_capacity(a.c, a.b));
        table = a.b.table + (int64_t)pc.group * a.b.table_stride;
        head_off = pc.item / p.ctiles * a.c.head_stride;
      }
      fpos = ((f - pc.item0) * kDecWarps + warp) * 16;
      if (fpos < visible) fpid = table[fpos >> a.c.page_shift];
    };
    int pos_of[S];  // positions of the blocks in the ring, -1: none
    int fslot = 0;
    uint32_t flying = 0;  // slots whose copy has not been waited for
    bool dead = false;    // a wait of this warp gave up: nothing more is fetched
    auto fetch = [&]() {
      if (f >= last) return;
      const bool ok = (uint32_t)fpid < (uint32_t)a.c.num_pages && !dead;
      const uint8_t* from = a.c.pages + (int64_t)fpid * a.c.page_stride + head_off +
                            (int64_t)((fpos & (a.c.page_size - 1)) >> 4) * Geo::kBytes;
#pragma unroll
      for (int y = 0; y < S; ++y)
        if (y == fslot) pos_of[y] = ok ? fpos : -1;
      flying |= (uint32_t)ok << fslot;
      if (ok && lane == 0) {
        const uint32_t bar = smem_addr(&full[warp * S + fslot]);
        mbar_arrive_expect_tx(bar, Geo::kBytes);
        if (!(p.fail && me == 0 && warp == 0 && f == last - 1))
          bulk_g2s(smem_addr(ring + fslot * kSlot), from, Geo::kBytes, bar);
      }
      fslot = fslot + 1 == S ? 0 : fslot + 1;
      ++f;
      look();
    };
    look();
#pragma unroll
    for (int y = 0; y < S; ++y) pos_of[y] = -1;
#pragma unroll 1
    for (int y = 0; y < S - NT; ++y) fetch();

    int slot = 0;
    uint32_t parity = 0;  // a bit per slot
    // where this lane's words lie in a block
    uint32_t at_k[D / 64], at_v[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      at_k[i] = r * D + Geo::k_piece(r, c + 4 * i) * 16;
      at_v[i] = Geo::kVOff + c * 2 * D + Geo::v_piece(c, D == 128 ? 2 * r + i : r) * 16;
    }
    volatile Item& it = sh_item;
    if (tid == 0) store(it.at, seed);
    for (int seg = first; seg < last;) {
      if (tid == 0) {
        Cursor cc = load(it.at);
        cc.enter(a, p, seg);
        const KvSeq q = kv_seq(a.b, cc.group);
        store(it.at, cc);
        if constexpr (W)
          if (scores.base && cc.item == 0 && cc.item0 == seg) scores.base[cc.group] = cc.end <= scores.limit ? seg : -1;
        it.s = cc.group;
        it.head = cc.item / p.ctiles;
        it.ctile = cc.item % p.ctiles;
        it.row_lo = 0;
        it.cols = q.rows * p.per;
        it.rows = q.rows;
        it.len = q.len;
        it.row0 = q.row0;
      }
      __syncthreads();
      const int seg_end = min(it.at.item_end, last);
      // ---- the item's columns
      uint32_t qf[NT][D / 8];  // this lane's query operand: column 8 nt + r, the channels that match its words
      float factor[NT][2];     // scale log2 e 2^-by of columns 8 nt + 2 c, + 1
      int seen[NT][2];         // tokens that they see
      int least = 0x7fffffff;  // over the columns
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const KvSeq q = it.seq();
        const int x = it.ctile * C + nt * 8 + r;  // a column of nobody is zeros, never written
        const bool real = x < it.cols;
        const int i = real ? x / p.per : 0;
        const uint16_t* src = a.q + kv_row_offset(a.b, a.qs, it.s, q.row0, i) + (int64_t)(it.head * p.per + x % p.per) * a.qs.head;
        uint4 raw[D / 32];
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {  // 8 channels: half a piece of 16
          raw[w] = real ? *reinterpret_cast<const uint4*>(src + (c + 4 * (w / 2)) * 16 + w % 2 * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = max(top, max(__float_as_uint(fabsf(KvType<T>::lo(v[e]))), __float_as_uint(fabsf(KvType<T>::hi(v[e])))));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (int)(top >> 23) - 127;  // the largest element to 2^14; an infinity or a NaN stays what it is
        const int by = top == 0u || ex > 127 ? 0 : min(max(14 - ex, -113), 113);
        const float up = pow2(by);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[nt][4 * w + e] = KvType<__half>::pack(KvType<T>::lo(v[e]) * up, KvType<T>::hi(v[e]) * up);
        }
        const int64_t pos = (int64_t)q.len - q.rows + i;
        const int see = pos < 0 ? 0 : (int)min(a.causal ? pos + 1 : (int64_t)q.len, (int64_t)kv_capacity(a.c, a.b));
        const float back = a.scale * 1.4426950408889634f * pow2(-by);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          factor[nt][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
          seen[nt][e] = __shfl_sync(0xffffffffu, see, 4 * (2 * c + e));
        }
        least = min(least, __reduce_min_sync(0xffffffffu, see));
      }

      float acc[D / 16][NT][4];  // O^T: channel tiles by columns
      float ry[NT][2], l[NT][2], dz[NT][2];  // reference, sum of weights, ry - rz
      float fell[NT][2];         // how far rz has been lowered since it was raised
      float bad[NT][2];          // NaN where the column sees a token of NaN values
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ry[nt][e] = kNone;
          dz[nt][e] = kNoProduct;
          l[nt][e] = bad[nt][e] = fell[nt][e] = 0.0f;
        }
      }

      auto block = [&](const uint8_t* blk, int pos) {
        const uint4 par = *reinterpret_cast<const uint4*>(blk + Geo::kParams);
        const float ks = __uint_as_float(par.x), lv = log2f(__uint_as_float(par.y));
        // ---- scores of tokens r and r + 8, columns 2 c and 2 c + 1
        float y[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[nt][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t lo[4], hi[4];
          load_words(lo, blk + at_k[i]);
          load_words(hi, blk + at_k[i] + 8 * D);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = kv8_pair<0>(lo[w]), a1 = kv8_pair<0>(hi[w]), a2 = kv8_pair<1>(lo[w]), a3 = kv8_pair<1>(hi[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(y[nt], a0, a1, a2, a3, qf[nt][8 * i + 2 * w], qf[nt][8 * i + 2 * w + 1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[nt][e] *= factor[nt][e & 1] * ks;  // (together first: they may lie far apart)
        if (par.z != 0) {  // tokens that read as NaN
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = r + 8 * (e >> 1);
              if ((par.z >> t) & 1u) y[nt][e] = __int_as_float(0x7fffffff);
              if ((par.z >> (16 + t)) & 1u && pos + t < seen[nt][e & 1]) bad[nt][e & 1] = __int_as_float(0x7fffffff);
            }
        }
        if (pos + 16 > least) {  // some column does not see some of these
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (pos + r + 8 * (e >> 1) >= seen[nt][e & 1]) y[nt][e] = -__int_as_float(0x7f800000);
        }
        if constexpr (W) {
          if (it.at.end <= scores.limit) {
            float* to = scores.to + ((int64_t)it.at.item0 * (16 * kDecWarps) + pos + r) * scores.width + 2 * c;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (2 * c + 8 * nt < scores.width) {
                *reinterpret_cast<float2*>(to + 8 * nt) = make_float2(y[nt][0], y[nt][1]);
                *reinterpret_cast<float2*>(to + 8 * nt + 8 * scores.width) = make_float2(y[nt][2], y[nt][3]);
              }
          }
        }
        // ---- references
        uint32_t some = 0, raise = 0;  // columns (a bit each) of which some token is not small; the highest bit: one is too large
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float t = fmaxf(y[nt][x], y[nt][2 + x]) - ry[nt][x], z = t + (lv + dz[nt][x]);
            if (t > kRaiseSum || z > kRaiseProduct) raise = 1u << 31;
            if (z > kLower) some |= 1u << (8 * nt + 4 * x);
          }
        if (__reduce_or_sync(0xffffffffu, some << c | raise) != (1u << C) - 1u) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float t = fmaxf(fmaxf(y[nt][x], y[nt][2 + x]), kNone);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
              const float now = fmaxf(ry[nt][x], t);  // (a column that sees nothing here stays)
              const float up = ry[nt][x] - now;
              l[nt][x] *= exp2_fast(up);
              float to = fminf(dz[nt][x] - up, kNoProduct);  // rz as it is, from the new ry
              const float most = -((t - now) + lv);          // rz at this block's largest product
              const bool lower = most > to - kLower && most < to - kGone && fell[nt][x] <= kLowerMost - 8.0f;
              if ((most < to || lower) && t != kNone) {
                const float next = fminf(most, to + (kLowerMost - fell[nt][x])), by = exp2_fast(next - to);
                fell[nt][x] = fmaxf(fell[nt][x] + (next - to), 0.0f);
                to = next;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  acc[j][nt][x] *= by;
                  acc[j][nt][2 + x] *= by;
                }
              }
              ry[nt][x] = now;
              dz[nt][x] = to;
            }
        }
        // ---- weights, their sums, and the second product's operand
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float t = y[nt][e] - ry[nt][e & 1];
            l[nt][e & 1] += exp2_fast(t);
            w[e] = exp2_fast(t + (lv + dz[nt][e & 1]));
          }
          pf[nt][0] = transpose8x8(KvType<__half>::pack(w[0], w[1]));
          pf[nt][1] = transpose8x8(KvType<__half>::pack(w[2], w[3]));
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t lo[4], hi[4];
          load_words(lo, blk + at_v[i]);
          load_words(hi, blk + at_v[i] + 8 * D);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = kv8_pair<0>(lo[w]), a1 = kv8_pair<1>(lo[w]), a2 = kv8_pair<0>(hi[w]), a3 = kv8_pair<1>(hi[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(acc[4 * i + w][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        }
      };

      for (int cu = seg; cu < seg_end; ++cu) {
        fetch();  // into the slot that was used last
        int pos = -1;
#pragma unroll
        for (int y = 0; y < S; ++y)
          if (y == slot) pos = pos_of[y];
        if (pos >= 0) {
          if (__all_sync(0xffffffffu, kv_wait(smem_addr(&full[warp * S + slot]), (parity >> slot) & 1u, &sh_gone, err))) {
            parity ^= 1u << slot;
            flying ^= 1u << slot;
            block(ring + slot * kSlot, pos);
          } else {
            dead = true;
          }
        }
        __syncwarp();  // every lane is done with the slot
        slot = slot + 1 == S ? 0 : slot + 1;
      }

      // ---- join the warps: O of each in the slots that it used last, which are not being filled
      const int used = slot == 0 ? S - 1 : slot - 1;  // NT = 2: and the one before
      auto place = [&](int nt) {
        const int y = used - nt;
        return (y < 0 ? y + S : y) * kSlot;
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* dst = reinterpret_cast<float*>(ring + place(nt));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int col = 2 * c + x;
          float poison = bad[nt][x];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], o);
            poison += __shfl_xor_sync(0xffffffffu, poison, o);
          }
          if (r == 0) {
            mm[warp * C + nt * 8 + col] = ry[nt][x];
            ml[warp * C + nt * 8 + col] = l[nt][x];
            mz[warp * C + nt * 8 + col] = dz[nt][x];
          }
          // lane r holds channels D / 8 r ..; quads of channels change places by c, so that eight lanes hit all banks
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            reinterpret_cast<float4*>(dst)[col * (D / 4) + ((r * (D / 32) + i) ^ c)] =
                make_float4(acc[2 * i][nt][x] + poison, acc[2 * i][nt][2 + x] + poison, acc[2 * i + 1][nt][x] + poison,
                            acc[2 * i + 1][nt][2 + x] + poison);
        }
      }
      __syncthreads();
      // Where a wait gave up, the rows whose blocks are missing are NaN, their lse too, so that they add nothing to mass.
      const bool gone = *static_cast<volatile uint32_t*>(&sh_gone);
      const int item0 = it.at.item0, item_end = it.at.item_end;
      const bool whole = seg == item0 && seg_end == item_end;
      // partial results: a CTA's first stretch in slot 0, its last in slot 1
      float* part = ws + (int64_t)(2 * me + (seg == first ? 0 : 1)) * kPart;
      auto finish = [&](int col, int d4, float4 o, float M, float L) {  // four channels of a column
        const int x = it.ctile * C + col, s = it.s;
        if (x >= it.cols) return;
        const int i = x / p.per, hq = it.head * p.per + x % p.per;
        const KvSeq q = it.seq();
        *reinterpret_cast<uint2*>(a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + (int64_t)hq * a.os.head + 4 * d4) =
            make_uint2(KvType<T>::pack(o.x, o.y), KvType<T>::pack(o.z, o.w));
        const int64_t row = kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq;
        if (a.lse && d4 == 0) a.lse[row] = L == 0.0f ? -__int_as_float(0x7f800000) : (M + log2f(L)) * 0.6931471805599453f;
        if constexpr (W)
          if (d4 == 0 && row < scores.refs_limit) scores.refs[row] = make_float2(M, 1.0f / L);
      };
      for (int x = tid; x < C * (D / 4); x += kDec8Threads) {
        const int col = x / (D / 4), d4 = x % (D / 4), nt = col / 8, cc = col % 8;
        // the largest ry, and the largest rz = ry - dz, both against the former
        float M = mm[col];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) M = fmaxf(M, mm[w * C + col]);
        float Z = -kNoProduct, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float d = mm[w * C + col] - M;
          Z = fmaxf(Z, d - mz[w * C + col]);
          L = fmaf(exp2_fast(d), ml[w * C + col], L);
        }
        if (gone) L = __int_as_float(0x7fffffff);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float f = exp2_fast(mm[w * C + col] - M - mz[w * C + col] - Z);
          const float4 v = reinterpret_cast<const float4*>(smem + w * S * kSlot + place(nt))[cc * (D / 4) + (d4 ^ (cc >> 1))];
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
        }
        // a row that sees nothing is zero; 2^Z goes in two steps, its halves within fp32's range
        const float half = exp2f(0.5f * fmaxf(Z, -280.0f)), inv = L == 0.0f ? 0.0f : half / L;
        o = make_float4(o.x * inv * half, o.y * inv * half, o.z * inv * half, o.w * inv * half);
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
        const int c0 = owner(item0, total, n), c1 = owner(item_end - 1, total, n);
        __syncthreads();  // every thread's part is written: one release covers them
        if (tid == 0) sh_last = add_acq_rel(&counters[c0]);
        __syncthreads();
        if (sh_last == (unsigned)(c1 - c0)) {
          // the item began c0's last stretch: its only one if the item begins c0's share
          const int head = 2 * c0 + (item0 == share(total, c0, n) ? 0 : 1);
          auto slot_of = [&](int y) { return ws + (int64_t)(y == c0 ? head : 2 * y) * kPart; };
          // the parts' references and sums first, all at once, into the warps' slots: an eighth of the parts in each
          auto record = [&](int y) { return reinterpret_cast<float*>(smem + (y & 7) * S * kSlot + place(0)) + (y >> 3) * 2 * C; };
          for (int x = tid; x < (c1 - c0 + 1) * 2 * C; x += kDec8Threads)
            record(x / (2 * C))[x % (2 * C)] = __ldcg(slot_of(c0 + x / (2 * C)) + C * D + x % (2 * C));
          __syncthreads();
          for (int x = tid; x < C * (D / 4); x += kDec8Threads) {
            const int col = x / (D / 4), d4 = x % (D / 4);
            float M = kNone, L = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int y = 0; y <= c1 - c0; ++y) M = fmaxf(M, record(y)[col]);
#pragma unroll 4
            for (int y = 0; y <= c1 - c0; ++y) L = fmaf(exp2_fast(record(y)[col] - M), record(y)[C + col], L);
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll 8
            for (int y = c0; y <= c1; ++y) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(slot_of(y)) + x);
              const float f = exp2_fast(record(y - c0)[col] - M) * (record(y - c0)[C + col] * inv);
              o.x = fmaf(f, v.x, o.x);
              o.y = fmaf(f, v.y, o.y);
              o.z = fmaf(f, v.z, o.z);
              o.w = fmaf(f, v.w, o.w);
            }
            finish(col, d4, o, M, L);
          }
          if (tid == 0) counters[c0] = 0;  // for the next call
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the slots are bulk copies' again
      __syncthreads();
      seg = seg_end;
    }
    // whoever gave up no longer waits for what was fetched: it has landed before the CTA ends
    if (*static_cast<volatile uint32_t*>(&sh_gone)) {
#pragma unroll
      for (int y = 0; y < S; ++y)
        if ((flying >> y) & 1u) mbar_drain(smem_addr(&full[warp * S + y]), (parity >> y) & 1u);
    }
  }

  // ---- groups without a round: their rows see nothing
  for (int gi = me; gi < p.groups; gi += gridDim.x) {
    if (group_rounds(a, gi)) continue;
    const KvSeq q = kv_seq(a.b, gi);
    for (int i = 0; i < q.rows; ++i)
      for (int x = tid; x < a.q_heads * (D / 8); x += kDec8Threads) {
        const int hq = x / (D / 8);
        *reinterpret_cast<uint4*>(a.out + kv_row_offset(a.b, a.os, gi, q.row0, i) + (int64_t)hq * a.os.head + 8 * (x % (D / 8))) =
            make_uint4(0, 0, 0, 0);
        if (a.lse && x % (D / 8) == 0) a.lse[kv_row_index(a.b, gi, q.row0, i) * a.q_heads + hq] = -__int_as_float(0x7f800000);
      }
  }
}

template <typename T, int D, int NT>
cudaError_t launch_decode8(Kv8& kv, const KvAttnArgs& a, const DecPlan& p, const Kv8Scores& scores, cudaStream_t s) {
  constexpr int C = 8 * NT;
  const size_t smem = (size_t)kDecWarps * kDec8Slots<NT> * kDec8Slot<D>;
  const auto kernel = scores.refs ? kv8_decode_kernel<T, D, NT, true> : kv8_decode_kernel<T, D, NT, false>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv.sms * 2, kDec8MaxParts) / NT;
  static_assert(kDec8MaxParts <= Kv8::kCounters, "a counter per CTA");
  static_assert(2 * (size_t)kDec8MaxParts * C * (D + 2) * sizeof(float) <= Kv8::kFewPartsBytes, "two partial results per CTA");
  kernel<<<grid, kDec8Threads, smem, s>>>(a, p, kv.parts(), kv.counters(), kv.err_dev, scores);
  return cudaGetLastError();
}

template <typename T>
cudaError_t decode8(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s) {
  DecPlan p;
  p.per = a.q_heads / a.c.heads;
  const int64_t cols = (int64_t)p.per * a.b.max_new;
  const int nt = cols > 8 ? 2 : 1;
  const int64_t ctiles = (cols + 8 * nt - 1) / (8 * nt), items = ctiles * a.c.heads;
  const int64_t rounds = (((int64_t)a.b.table_pages << (a.c.page_shift - 4)) + kDecWarps - 1) / kDecWarps;
  if (items > 0x7fffffff || a.b.batch * items > 0x7fffffff / rounds) return cudaErrorInvalidConfiguration;  // rounds are numbered in 32 bits
  p.groups = a.b.batch;
  p.ctiles = (int)ctiles;
  p.items = (int)items;
  p.min_rounds = 1;
  p.fail = kv.fail_next;
  if (kv.d.head_dim == 64) return nt == 1 ? launch_decode8<T, 64, 1>(kv, a, p, scores, s) : launch_decode8<T, 64, 2>(kv, a, p, scores, s);
  return nt == 1 ? launch_decode8<T, 128, 1>(kv, a, p, scores, s) : launch_decode8<T, 128, 2>(kv, a, p, scores, s);
}

}  // namespace
