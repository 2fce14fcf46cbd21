// Attention of few rows over the 4-bit cache: a decode step's single tokens, a
// few speculated tokens, or any number of rows that each chose pages of their
// own.  Included by kv_decode_bf16.cu and kv_decode_f16.cu, one type each.
//
// Mathematics.  For the columns (row, query head) that share a kv head, the
// scores of 16 tokens are S^T = K q^T on the tensor cores with the tokens as
// the 16 rows of mma.m16n8k16 and up to 8 columns as its n, so a group of
// query heads costs what one head costs.  The operand is the code itself, not
// the stored value: with stored value c + s (u - 8) per token and group,
//     S[t][col] = sum over groups g of  s_g (u_g . q_g) + (c_g - 8 s_g) sum(q_g),
// where u enters as its four bits in an fp16 subnormal (one mask, exact), q as
// fp16 times a power of two that brings its largest element to 2^14, and s and
// c in fp32 on the accumulators.  O^T = V^T P^T is the second product, the
// channels as rows: P s_g per group is rounded to fp16 (the one rounding before
// the output's, 2^-12 of a weight and independent from token to token); the
// centres' part is summed apart in fp32.  bf16 outputs take the values' codes
// as they are too (their offset of 8 s makes that rounding three times larger,
// far below bf16's); fp16 outputs take u - 8.
//
// Softmax: weights are 2^(score - reference) with a running reference per
// column, raised only when a score passes it by 4, so that most blocks rescale
// nothing; sums are fp32.  O is carried times 2^-E, with E for values of
// ordinary size.  In a block that holds other sizes the reference goes by weight
// times value: a huge value that a column does not see, or hardly weighs, takes
// nothing from its other tokens, and a token of nearly all the weight and hardly
// any value leaves room for the rest.  What is rounded to fp16 is then below
// 2^-24 of the column's largest product.  (The groups of a token share this:
// one whose values are 2^16 times smaller than another's begins to lose bits.)
// A column that sees no token keeps the sum 0.
//
// Work split: all rounds (8 blocks of 16 tokens of one kv head and column tile)
// of the batch in one line, cut into equal shares, one per CTA; a share covers
// any number of items (sequence, head, column tile) or part of one.  Rounds come
// through a ring in shared memory, one bulk copy per page (or its 128 tokens),
// fetched by a ninth warp, its page numbers asked for a round ahead; each of the
// 8 others takes one block of a round.  At the end of an item's stretch the
// warps' (max, sum, O) are joined in shared memory; an item cut between CTAs is
// joined by the CTA that finishes last, in the order of the CTAs, so results do
// not depend on timing.
//
// Measured (8 kv heads of 128 channels): 64 sequences of up to 8,191 tokens, 32
// query heads, bf16, groups of 64: 92.5 us, 4.0 TB/s; 2 of 131,072, 64 query
// heads, fp16, groups of 32: 82 us, 4.1 TB/s; one of 777: 11.4 us.  The fetch alone
// takes 72 and 61 us: the bytes at the memory's rate (54 and 50) and launch, shares,
// first round, joins; the rest is the blocks' own work that the fetch does not
// cover: some 350 instructions a block and warp, 57 and 65 % of the issue slots,
// the integer pipe (the masks that make operands of codes) 48 and 42 %.  Telling
// sizes of values and scores apart where the reference rises costs 4 and 2 us of it.
// Two blocks at once a warp, or the next block's scores early, need more than the
// 104 registers that two CTAs per SM leave, and lose (104 and 105 us for the first).
#pragma once

#include "kv_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"

constexpr int kDecWarps = 8;                         // that compute
constexpr int kDecThreads = (kDecWarps + 4) * 32;  // and one that fetches; three only fill its warpgroup
// Registers, two CTAs per SM for 8 columns and one for 16: the launch's are dealt out
// again between the warpgroups.
template <int NT>
struct DecRegs {
  static constexpr int kLaunch = NT == 1 ? 80 : 168, kCompute = NT == 1 ? 104 : 232, kFetch = NT == 1 ? 32 : 40;
  static_assert(2 * kCompute + kFetch <= 3 * kLaunch, "a split above the launch's registers never ends");
};
constexpr int kDecMaxParts = kDecWarps * (64 + 4);  // CTAs, so parts of an item, whose references fit the merge buffer
constexpr float kDecSlack = 4.0f;      // weights reach 2^4
constexpr int kDecRoom = 14;           // |c| + 8 s stays below 2^(E + 14): weights times steps below 2^15
constexpr int kDecAim = 10;            // a column's largest weight times value is raised to about 2^(E + 10)
constexpr float kDecPartScale = 0x1p-40f;  // of parts' weights (up to 2^30 each): their sum with values stays in range

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kDecWarps * 32) : "memory"); }
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {  // 4 N contiguous, aligned bytes
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// What the work is divided into.  A round is 8 blocks of an item; an item is a
// (group, head, column tile); a group is a sequence, or with chosen pages one
// of its rows.  Round numbers run over the groups, inside them over the items,
// inside them over the tokens.
struct DecPlan {
  int groups;      // sequences, or batch * max_new rows
  int items;       // items per group: heads * column tiles
  int ctiles;      // column tiles
  int per;         // query heads per kv head
  int min_rounds;  // a CTA's share is not made smaller than this
  int fail;        // test hook: the first CTA's last round is not fetched
};

__device__ __forceinline__ int group_rounds(const KvAttnArgs& a, int gi) {
  if (a.sel) {
    const int s = gi / a.b.max_new, i = gi % a.b.max_new;
    return i < kv_seq(a.b, s).rows ? ((a.budget << (a.c.page_shift - 4)) + kDecWarps - 1) / kDecWarps : 0;
  }
  const KvSeq q = kv_seq(a.b, gi);
  return q.rows > 0 ? (min(q.len, kv_capacity(a.c, a.b)) + 16 * kDecWarps - 1) / (16 * kDecWarps) : 0;
}

// First CTA whose share [total c / n, total (c + 1) / n) holds round u.
__device__ __forceinline__ int owner(int u, int total, int n) { return (int)((((int64_t)u + 1) * n - 1) / total); }
__device__ __forceinline__ int share(int total, int c, int n) { return (int)((int64_t)total * c / n); }

// A place in the line of rounds.
struct Cursor {
  int group, end, rounds;  // the group, its end, the rounds of each of its items
  int item, item0, item_end;

  __device__ __forceinline__ void enter(const KvAttnArgs& a, const DecPlan& p, int u) {
    int base = end - rounds * p.items;
    while (u >= end) {
      base = end;
      rounds = group_rounds(a, ++group);
      end = base + rounds * p.items;
    }
    item = (u - base) / rounds;
    item0 = base + item * rounds;
    item_end = item0 + rounds;
  }
};

// State that the block loop does not touch lives in shared memory, not in registers.
struct Item {  // the item at hand
  Cursor at;
  int s, head, ctile, row_lo, cols;  // sequence, kv head, column tile, first row, columns of all tiles
  int rows, len;                     // KvSeq
  int64_t row0;
  __device__ __forceinline__ KvSeq seq() const volatile { return {row0, rows, len}; }
};
__device__ __forceinline__ Cursor load(const volatile Cursor& c) {
  return {c.group, c.end, c.rounds, c.item, c.item0, c.item_end};
}
__device__ __forceinline__ void store(volatile Cursor& c, const Cursor& v) {
  c.group = v.group, c.end = v.end, c.rounds = v.rounds;
  c.item = v.item, c.item0 = v.item0, c.item_end = v.item_end;
}

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 2 : 1)
    kv_decode_kernel(const __grid_constant__ KvAttnArgs a, const __grid_constant__ DecPlan p, float* __restrict__ ws,
                     unsigned* __restrict__ counters, uint32_t* err) {
  using Geo = KvGeom<D, G>;
  constexpr bool kCentred = std::is_same<T, __half>::value;
  constexpr int C = 8 * NT, NG = D / G;
  constexpr int kStages = kDecStages<D, G>;
  constexpr int kSlot = C * (D + 2);  // floats of one partial result: O [C][D], max [C], sum [C]
  extern __shared__ __align__(128) uint8_t smem[];
  float* mo = reinterpret_cast<float*>(smem + kDecWarps * kStages * Geo::kBytes);  // [warp][C][D + 4]; below: [stage][block]
  float* mm = mo + kDecWarps * C * (D + 4);                                     // [warp][C] max, then sums
  float* ml = mm + kDecWarps * C;
  uint64_t* full = reinterpret_cast<uint64_t*>(ml + kDecWarps * C);             // [stage]
  uint64_t* empty = full + kStages;                                             // [stage]
  int* spos = reinterpret_cast<int*>(empty + kStages);                          // [stage][block] its position, -1: not there
  __shared__ int sh_sum[kDecThreads / 32];
  __shared__ int sh_base, sh_group;
  __shared__ Item sh_item;
  __shared__ unsigned sh_last;
  __shared__ uint32_t sh_gone;  // a wait gave up: results are wrong, the next call says so
  __shared__ int2 sh_exp[kDecWarps];  // a warp's E, exponent of the largest value it has seen
  __shared__ float sh_up[kDecWarps * C];
  __shared__ float2 sh_lift[C];       // of the item's columns; every warp writes the same
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;

  if (tid == 0) sh_gone = 0;
  if (tid < kStages) {
    mbar_init(smem_addr(&full[tid]), 1);
    mbar_init(smem_addr(&empty[tid]), kDecWarps);
  }
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
    for (int w = 0; w < kDecThreads / 32; ++w) {
      if (w < warp) v += sh_sum[w];
      all += sh_sum[w];
    }
    return v;
  };
  int total = 0, mine = 0, upto = 0;  // the last groups' (for up to kDecThreads groups: the only) prefix
  for (int g0 = 0; g0 < p.groups; g0 += kDecThreads) {
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
    if (p.groups <= kDecThreads) {
      if (upto - mine <= first && first < upto) {
        sh_group = tid;
        sh_base = upto - mine;
      }
    } else {
      int before = 0;
      for (int g0 = 0; g0 < p.groups && before <= first; g0 += kDecThreads) {
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

    if (warp >= kDecWarps) {
      set_registers<DecRegs<NT>::kLaunch, DecRegs<NT>::kFetch>();
      if (warp == kDecWarps) {
      // ---- fetching: lane b < 8 looks after block b of each round
      Cursor pc = seed;
      const int per_page = a.c.page_shift - 4;
      const int run = min(1 << per_page, kDecWarps);  // blocks per copy
      int head = 0, seen = 0;                         // kv head; positions from `seen` on are not read
      const int32_t *table = nullptr, *list = nullptr;  // of the sequence's pages, of the chosen ones
      int pos = 0, pid = -1;                          // of the block
      const uint8_t* src = nullptr;
      auto look = [&](int u) {  // asks for the pages of round u
        if (u >= last) return;
        if (u >= pc.item_end) {
          pc.enter(a, p, u);
          head = pc.item / p.ctiles;
          const int s = a.sel ? pc.group / a.b.max_new : pc.group;
          const KvSeq q = kv_seq(a.b, s);
          int64_t n = q.len;
          if (a.sel) {
            const int i = pc.group % a.b.max_new;
            list = a.sel + (kv_row_index(a.b, s, q.row0, i) * a.c.heads + head) * a.budget;
            if (a.causal) n = (int64_t)q.len - q.rows + i + 1;
          }
          seen = (int)min(n, (int64_t)kv_capacity(a.c, a.b));
          table = a.b.table + (int64_t)s * a.b.table_stride;
          src = a.c.pages + head * a.c.head_stride;
        }
        const int ub = (u - pc.item0) * kDecWarps + lane;
        int j = ub >> per_page;
        pos = ub * 16;
        if (a.sel) {
          j = j < a.budget ? list[j] : -1;
          // pages beyond the row's are skipped (compared as pages: positions could wrap)
          const bool in = j >= 0 && j <= (seen - 1) >> a.c.page_shift;
          pos = in ? (j << a.c.page_shift) + 16 * (ub & ((1 << per_page) - 1)) : 0x7fffffff;
        }
        pid = lane < kDecWarps && pos < seen ? table[j] : -1;
      };
      int stage = 0;
      uint32_t parity = 1;  // of the stage's last release; a fresh barrier reports it as done
      look(first);
      for (int u = first; u < last; ++u) {
        const uint8_t* from = src + (int64_t)pid * a.c.page_stride + (int64_t)((pos & (a.c.page_size - 1)) >> 4) * Geo::kBytes;
        const bool ok = (uint32_t)pid < (uint32_t)a.c.num_pages;
        const int at = ok ? pos : -1;
        look(u + 1);
        const uint32_t there = __ballot_sync(0xffffffffu, ok);
        if (!kv_wait(smem_addr(&empty[stage]), parity, &sh_gone, err)) break;
        if (p.fail && me == 0 && u == last - 1) break;
        if (lane < kDecWarps) spos[stage * kDecWarps + lane] = at;
        __syncwarp();
        const uint32_t bar = smem_addr(&full[stage]);
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(there) * Geo::kBytes);
        __syncwarp();
        // the blocks of a page that are there are its first ones: one copy
        const int count = __popc(there >> lane & ((1u << run) - 1u));
        if (ok && lane % run == 0)
          bulk_g2s(smem_addr(smem) + (stage * kDecWarps + lane) * Geo::kBytes, from, count * Geo::kBytes, bar);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }
      // whoever gave up no longer waits for what was fetched: it has landed before the CTA ends
      if (*static_cast<volatile uint32_t*>(&sh_gone)) {
        for (int st = 0; st < kStages; ++st) {
          const uint32_t fill = st < stage ? parity ^ 1u : parity;  // of its last fill; a barrier never filled is passed
          mbar_drain(smem_addr(&full[st]), fill);
        }
      }
      }
    } else {
    set_registers<DecRegs<NT>::kLaunch, DecRegs<NT>::kCompute>();
    int stage = 0;         // of the round at hand
    uint32_t parity = 0;   // of its fill
    // where this lane's words lie in a block
    const int at_k = r * Geo::kRow + c * (D / 8), at_p = Geo::kKPar + r * Geo::kParRow;
    const int at_v = Geo::kVOff + c * Geo::kRow + (r ^ ((c >> 1) << 2)) * (D / 16);
    volatile Item& it = sh_item;
    if (tid == 0) store(it.at, seed);
    for (int seg = first; seg < last;) {
      if (tid == 0) {
        Cursor cc = load(it.at);
        cc.enter(a, p, seg);
        const int s = a.sel ? cc.group / a.b.max_new : cc.group;
        const KvSeq q = kv_seq(a.b, s);
        store(it.at, cc);
        it.s = s;
        it.head = cc.item / p.ctiles;
        it.ctile = cc.item % p.ctiles;
        it.row_lo = a.sel ? cc.group % a.b.max_new : 0;
        it.cols = (a.sel ? 1 : q.rows) * p.per;
        it.rows = q.rows;
        it.len = q.len;
        it.row0 = q.row0;
      }
      compute_sync();
      const int seg_end = min(it.at.item_end, last);
      // ---- the item's columns
      uint32_t qf[NT][D / 8];    // this lane's query operand: column 8 nt + r, its quarter of every group
      float qsum[NT][NG][2];     // 2^-24 sums over a group's channels, columns 8 nt + 2c, + 1
      float factor[NT][2];       // what makes the columns' sums scores (log2)
      int seen[NT][2];           // tokens that the columns see
      int least = 0x7fffffff, most = 0;  // over the columns
      // the scores are multiplied by sh_lift and the factor (then 1) before anything else: where a
      // factor would leave fp32's range, and where they are as large as kCoarse
      bool lifted = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int s = it.s, h = it.head, row_lo = it.row_lo, ncols = it.cols;
        const KvSeq q = it.seq();
        const int cap = kv_capacity(a.c, a.b);
        const int x = it.ctile * C + nt * 8 + r;  // column 8 nt + r; a column of nobody is zeros, never written
        const bool real = x < ncols;
        const int i = row_lo + (real ? x / p.per : 0);
        const uint16_t* src = a.q + kv_row_offset(a.b, a.qs, s, q.row0, i) + (int64_t)(h * p.per + x % p.per) * a.qs.head;
        uint4 raw[D / 32];
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const int ch = w / (G / 32) * G + c * (G / 4) + w % (G / 32) * 8;
          raw[w] = real ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0, 0, 0, 0);
          const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = max(top, max(__float_as_uint(fabsf(KvType<T>::lo(v[e]))), __float_as_uint(fabsf(KvType<T>::hi(v[e])))));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (int)(top >> 23) - 127;  // the largest element to 2^14; an infinity or a NaN stays what it is
        const int by = top == 0u || ex > 127 ? 0 : min(14 - ex, 113);
        const float up = pow2(by), up16 = pow2(by - 4);  // the odd fields are 16 u
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] = 0.0f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = KvType<T>::lo(v[e]), hi = KvType<T>::hi(v[e]), f = e % 2 ? up16 : up;
            qf[nt][4 * w + e] = KvType<__half>::pack(lo * f, hi * f);
            sum[w / (G / 32)] += lo * (up * 0x1p-24f) + hi * (up * 0x1p-24f);
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
#pragma unroll
          for (int e = 0; e < 2; ++e) qsum[nt][g][e] = __shfl_sync(0xffffffffu, sum[g], 4 * (2 * c + e));
        }
        const int64_t pos = (int64_t)q.len - q.rows + i;
        const int see = pos < 0 ? 0 : (int)min(a.causal ? pos + 1 : (int64_t)q.len, (int64_t)cap);
        // scale log2 e 2^(24 - by), of which what would leave fp32's range stays with the scores
        const float base = a.scale * 1.4426950408889634f;
        const int over = min(max((int)(__float_as_uint(fabsf(base)) >> 23) - 127 + 24 - by - 126, 0), 126);
        const int pw = 24 - by - over;  // -89..137: in two steps
        const float back = base * pow2(pw / 2) * pow2(pw - pw / 2);
        if (c == 0) sh_lift[nt * 8 + r] = make_float2(pow2(over), back);
        lifted |= __any_sync(0xffffffffu, over > 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          factor[nt][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
          seen[nt][e] = __shfl_sync(0xffffffffu, see, 4 * (2 * c + e));
        }
        least = min(least, __reduce_min_sync(0xffffffffu, see));
        most = max(most, __reduce_max_sync(0xffffffffu, see));
      }
      if (lane == 0) sh_exp[warp] = make_int2(0, -127);
      __syncwarp();  // sh_lift, sh_exp
      auto lift = [&](float (&sc)[NT][4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 by = sh_lift[nt * 8 + 2 * c + (e & 1)];
            sc[nt][e] = sc[nt][e] * by.x * by.y;
          }
      };
      auto factor_one = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) factor[nt][0] = factor[nt][1] = 1.0f;
      };
      if (lifted) factor_one();

      float acc[D / 16][NT][4];  // O^T: channel tiles by columns
      float oc[NT][NG][2];       // this lane's tokens' part of sum P (c - 8 s), or of sum P c
      float m[NT][2], l[NT][2];
      float vlimit = -1.0f;            // the values' bound for this E; negative before the first value
      float vdown = 0.0f;              // 2^-E
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

      // Scores of a block's tokens r and r + 8, columns 2c and 2c + 1 (what is masked may be anything).
      auto scores = [&](const uint8_t* blk, float (&sc)[NT][4]) {
        uint32_t kw[2][D / 32], kp[2][NG];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          load_words(kw[e], blk + at_k + 8 * e * Geo::kRow);
          load_words(kp[e], blk + at_p + 8 * e * Geo::kParRow);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float d[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[nt][e] = 0.0f;
#pragma unroll
          for (int w = g * (G / 32); w < (g + 1) * (G / 32); ++w) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(d[nt], raw_pair<0>(kw[0][w]), raw_pair<0>(kw[1][w]), raw_pair<1>(kw[0][w]), raw_pair<1>(kw[1][w]),
                      qf[nt][4 * w], qf[nt][4 * w + 1]);
              mma_f16(d[nt], raw_pair<2>(kw[0][w]), raw_pair<2>(kw[1][w]), raw_pair<3>(kw[0][w]), raw_pair<3>(kw[1][w]),
                      qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ks = KvType<T>::lo(kp[e][g]), kc = fmaf(-8.0f, ks, KvType<T>::hi(kp[e][g]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float z = g ? fmaf(kc, qsum[nt][g][x], sc[nt][2 * e + x]) : kc * qsum[nt][g][x];
                sc[nt][2 * e + x] = fmaf(ks, d[nt][2 * e + x], z);
              }
          }
        }
      };
      // One block from its scores.  part: some column does not see some of its tokens.
      auto block = [&](const uint8_t* blk, int pos, float (&sc)[NT][4], auto part_) {
        constexpr bool part = decltype(part_)::value;
        // params of tokens r and r + 8, values' codes of tokens 2c, 2c + 1, 2c + 8, 2c + 9
        uint32_t vp[2][NG], vw[4][D / 64];
#pragma unroll
        for (int e = 0; e < 2; ++e) load_words(vp[e], blk + at_p + Geo::kVPar - Geo::kKPar + 8 * e * Geo::kParRow);
#pragma unroll
        for (int t = 0; t < 4; ++t) load_words(vw[t], blk + at_v + t * 4 * Geo::kRow);
        bool hidden[NT][4];  // scores that their column does not see
        if constexpr (part) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (pos + r + 8 * e >= most)  // what no column sees may be anything
#pragma unroll
              for (int g = 0; g < NG; ++g) vp[e][g] = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) hidden[nt][e] = pos + r + 8 * (e >> 1) >= seen[nt][e & 1];
        }
        // exponents against the reference; it and E are raised where one passes it
        float ex[NT][4];
        auto exponents = [&]() {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ex[nt][e] = fmaf(sc[nt][e], factor[nt][e & 1], -m[nt][e & 1]);
              if constexpr (part)
                if (hidden[nt][e]) ex[nt][e] = -__int_as_float(0x7f800000);
            }
        };
        exponents();
        float vs[2][NG], vc[2][NG], big[2] = {0.0f, 0.0f};  // bounds of tokens r and r + 8 (of NaN groups: none)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            vs[e][g] = KvType<T>::lo(vp[e][g]);
            vc[e][g] = KvType<T>::hi(vp[e][g]);
            big[e] = fmaxf(big[e], fmaf(8.0f, vs[e][g], fabsf(vc[e][g])));
            if constexpr (!kCentred) vc[e][g] = fmaf(-8.0f, vs[e][g], vc[e][g]);
          }
        float top = ex[0][0];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, ex[nt][e]);
        if (__any_sync(0xffffffffu, top > kDecSlack || fmaxf(big[0], big[1]) > vlimit)) {
          auto score = [&](int nt, int x, float (&y)[2]) {  // of the column's two tokens here, and the block's largest
            float t = kNone;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[e] = sc[nt][2 * e + x] * factor[nt][x];
              if constexpr (part)
                if (hidden[nt][2 * e + x]) y[e] = kNone;
              t = fmaxf(t, y[e]);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            return t;
          };
          auto rescale = [&](int nt, int x, float f, float fo) {  // sum, O
            l[nt][x] *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) oc[nt][g][x] *= fo;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[j][nt][x] *= fo;
              acc[j][nt][2 + x] *= fo;
            }
          };
          // values of ordinary size, within 2^16 of the limit (at first: within 2^12 of each other), and
          // no token without any?
          bool ordinary = !__any_sync(0xffffffffu, fmaxf(big[0], big[1]) > vlimit || fminf(big[0], big[1]) < vlimit * 0x1p-16f);
          float shift = 0.0f;
          int to = 0;
          if (!ordinary) {
            // E becomes that of what is of ordinary size: an even block's largest value, at first also
            // an uneven one's smallest; within 2^64 of the largest ever
            const uint32_t b0 = __float_as_uint(big[0]), b1 = __float_as_uint(big[1]);
            const uint32_t vtop = __reduce_max_sync(0xffffffffu, max(b0, b1));
            const int hi_e = exponent(vtop);
            const int lo_e = exponent(__reduce_min_sync(0xffffffffu, min(b0 - 1u, b1 - 1u)));  // zero counts as none
            const int2 was = sh_exp[warp];
            to = was.x;
            if (vtop) {
              const bool even = hi_e - lo_e <= 12;
              if (vlimit < 0.0f) to = (even ? hi_e : lo_e) - kDecAim;
              else if (even && (hi_e >= was.x + kDecRoom || hi_e < was.x + kDecAim - 8)) to = hi_e - kDecAim;
              to = min(max(to, max(max(was.y, hi_e) - kDecAim - 64, -60)), 115);
              ordinary = vlimit < 0.0f && even && to == hi_e - kDecAim &&
                         __all_sync(0xffffffffu, fminf(big[0], big[1]) > 0.0f);
              if (vlimit >= 0.0f) shift = (float)(was.x - to);
              vdown = pow2(-to);
              vlimit = pow2(min(to + kDecRoom, 127));
            }
            __syncwarp();
            if (lane == 0) sh_exp[warp] = make_int2(to, max(was.y, hi_e));
          }
          if (ordinary) {  // the reference rises to the largest score
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float y[2];
                const float ref = fmaxf(score(nt, x, y), m[nt][x]), f = exp2_fast(m[nt][x] - ref);
                m[nt][x] = ref;
                rescale(nt, x, f, f);
              }
          } else {
            // the reference takes over what E gives up (O stays as it is) and rises by weight times
            // value, within 2^60 of the weights'
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float y[2];
                const float t = score(nt, x, y);
                // the weights so far, and the largest weight times value
                float w = l[nt][x] > 0.0f ? m[nt][x] + (float)exponent(__float_as_uint(l[nt][x])) : kNone, z = kNone;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (big[e] > 0.0f) z = fmaxf(z, y[e] + (float)(exponent(__float_as_uint(big[e])) - to));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                  w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
                  z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
                }
                const float cur = m[nt][x] + shift;
                float ref = fmaxf(fmaxf(cur, z - kDecAim), fmaxf(t, w) - 60.0f);
                if (t - ref <= 12.0f) ref = fmaxf(ref, t);  // so that the next blocks pass
                const float f = exp2_fast(m[nt][x] - ref);
                m[nt][x] = ref;
                rescale(nt, x, f, exp2_fast(cur - ref));
              }
          }
          float far = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) far = fmaxf(far, m[nt][x] == kNone ? 0.0f : fabsf(m[nt][x]));
          if (!lifted && __any_sync(0xffffffffu, far >= kCoarse)) {
            lifted = true;
            lift(sc);
            factor_one();
          }
          exponents();
        }
        // ---- weights, their sums, and P s as the second product's operand
        uint32_t pf[NT][NG][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[e] = exp2_fast(ex[nt][e]);
          l[nt][0] += pr[0] + pr[2];
          l[nt][1] += pr[1] + pr[3];
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[e] *= vdown;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = pr[e] * vs[e >> 1][g];
              float z = fmaf(pr[e], vc[e >> 1][g], oc[nt][g][e & 1]);
              if constexpr (part)  // zero times a poisoned centre is not zero: masked tokens are left out
                if (hidden[nt][e]) {
                  y[e] = 0.0f;
                  z = oc[nt][g][e & 1];
                }
              oc[nt][g][e & 1] = z;
            }
            pf[nt][g][0] = transpose8x8(KvType<__half>::pack(y[0], y[1]));
            pf[nt][g][1] = transpose8x8(KvType<__half>::pack(y[2], y[3]));
          }
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          const uint32_t lo0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), hi0 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
          const uint32_t lo1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), hi1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
          auto tile = [&](auto k_) {
            constexpr int K = decltype(k_)::value;
            const int j = 4 * w + K, g = j / (G / 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (kCentred)
                mma_f16(acc[j][nt], centred_pair<K>(lo0), centred_pair<K>(hi0), centred_pair<K>(lo1), centred_pair<K>(hi1),
                        pf[nt][g][0], pf[nt][g][1]);
              else
                mma_f16(acc[j][nt], raw_pair<K>(lo0), raw_pair<K>(hi0), raw_pair<K>(lo1), raw_pair<K>(hi1), pf[nt][g][0],
                        pf[nt][g][1]);
            }
          };
          tile(std::integral_constant<int, 0>());
          tile(std::integral_constant<int, 1>());
          tile(std::integral_constant<int, 2>());
          tile(std::integral_constant<int, 3>());
        }
      };

      // a round's stage, once it is there: this warp's block and its position
      auto arrive = [&](int st, uint32_t par, int& pos) {
        const uint32_t bar = smem_addr(&full[st]);
        pos = kv_wait(bar, par, &sh_gone, err) ? spos[st * kDecWarps + warp] : -1;
        return smem + (st * kDecWarps + warp) * Geo::kBytes;
      };
      for (int cu = seg; cu < seg_end; ++cu) {
        int pos;
        const uint8_t* blk = arrive(stage, parity, pos);
        if (pos >= 0) {
          float sc[NT][4];
          scores(blk, sc);
          if (lifted) lift(sc);
          if (pos + 16 > least) block(blk, pos, sc, std::true_type());
          else block(blk, pos, sc, std::false_type());
        }
        __syncwarp();  // every lane is done with the stage
        if (lane == 0) mbar_arrive(smem_addr(&empty[stage]));
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }

      // ---- join the warps: O of this warp with its centres' part, then all of them
      constexpr float even = kCentred ? 1.0f : 0x1p24f, odd = kCentred ? 1.0f : 0x1p20f;  // of the codes as subnormals
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
          const int by = excess<30>(l[nt][x]), up = sh_exp[warp].x - by;  // up: the power of two that goes with O
          if (r == 0) {
            mm[warp * C + col] = m[nt][x] + (float)by;
            ml[warp * C + col] = l[nt][x] * pow2(-by);
            sh_up[warp * C + col] = up < -126 ? 0.0f : pow2(min(up, 127));
          }
          float* dst = mo + (warp * C + col) * (D + 4);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const int g = j / (G / 16), ch = g * G + r * (G / 8) + 2 * j % (G / 8);
            const float f = j % 2 ? odd : even;
            *reinterpret_cast<float2*>(dst + ch) =
                make_float2(fmaf(acc[j][nt][x], f, oc[nt][g][x]), fmaf(acc[j][nt][2 + x], f, oc[nt][g][x]));
          }
        }
      compute_sync();
      const int item0 = it.at.item0, item_end = it.at.item_end;
      const bool whole = seg == item0 && seg_end == item_end;
      // partial results: a CTA's first stretch in slot 0, its last in slot 1
      float* part = ws + (int64_t)(2 * me + (seg == first ? 0 : 1)) * kSlot;
      auto finish = [&](int col, int d4, float4 o, float M, float L) {  // four channels of a column
        const int x = it.ctile * C + col, s = it.s;
        if (x >= it.cols) return;
        const int i = it.row_lo + x / p.per, hq = it.head * p.per + x % p.per;
        const KvSeq q = it.seq();
        *reinterpret_cast<uint2*>(a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + (int64_t)hq * a.os.head + 4 * d4) =
            make_uint2(KvType<T>::pack(o.x, o.y), KvType<T>::pack(o.z, o.w));
        if (a.lse && d4 == 0)
          a.lse[kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq] =
              L == 0.0f ? -__int_as_float(0x7f800000) : (M + log2f(L)) * 0.6931471805599453f;
      };
      auto normalise = [&](float4& o, float& L) {  // a row that sees nothing is zero
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        L *= 1.0f / kDecPartScale;
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
          const float p = exp2_fast(mm[w * C + col] - M) * kDecPartScale, f = p * sh_up[w * C + col];
          const float4 v = *reinterpret_cast<const float4*>(mo + (w * C + col) * (D + 4) + 4 * d4);
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
          L = fmaf(p, ml[w * C + col], L);
        }
        normalise(o, L);
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
        compute_sync();  // every thread's part is written: one release covers them
        if (tid == 0) sh_last = add_acq_rel(&counters[c0]);
        compute_sync();
        if (sh_last == (unsigned)(c1 - c0)) {
          // the item began c0's last stretch: its only one if the item begins c0's share
          const int head = 2 * c0 + (item0 == share(total, c0, n) ? 0 : 1);
          auto slot_of = [&](int y) { return ws + (int64_t)(y == c0 ? head : 2 * y) * kSlot; };
          // the parts' references first, all at once, into the merge buffer (at most kDecMaxParts of them)
          for (int x = tid; x < (c1 - c0 + 1) * C; x += kDecWarps * 32) mo[x] = __ldcg(slot_of(c0 + x / C) + C * D + x % C);
          compute_sync();
          for (int x = tid; x < C * (D / 4); x += kDecWarps * 32) {
            const int col = x / (D / 4), d4 = x % (D / 4);
            float M = kNone, L = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int y = 0; y <= c1 - c0; ++y) M = fmaxf(M, mo[y * C + col]);
#pragma unroll 8
            for (int y = c0; y <= c1; ++y) {
              const float* src = slot_of(y);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + x);
              const float w = __ldcg(src + C * D + C + col), f = exp2_fast(mo[(y - c0) * C + col] - M) * (w * kDecPartScale);
              o.x = fmaf(f, v.x, o.x);
              o.y = fmaf(f, v.y, o.y);
              o.z = fmaf(f, v.z, o.z);
              o.w = fmaf(f, v.w, o.w);
              L += f;
            }
            normalise(o, L);
            finish(col, d4, o, M, L);
          }
          if (tid == 0) counters[c0] = 0;  // for the next call
        }
      }
      compute_sync();  // the merge buffer is free
      seg = seg_end;
    }
    }
  }

  // ---- groups without a round: their rows see nothing
  for (int gi = me; gi < p.groups; gi += gridDim.x) {
    if (group_rounds(a, gi)) continue;
    const int s = a.sel ? gi / a.b.max_new : gi;
    const KvSeq q = kv_seq(a.b, s);
    const int lo = a.sel ? gi % a.b.max_new : 0, hi = a.sel ? min(lo + 1, q.rows) : q.rows;
    for (int i = lo; i < hi; ++i)
      for (int x = tid; x < a.q_heads * (D / 8); x += kDecThreads) {
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
  const size_t smem = (size_t)kDecStages<D, G> * (kDecWarps * (KvGeom<D, G>::kBytes + 4) + 16) +
                      (size_t)kDecWarps * C * (D + 6) * sizeof(float);
  const auto kernel = kv_decode_kernel<T, D, G, NT>;
  static const bool registers_fit = brings_registers(reinterpret_cast<const void*>(kernel), DecRegs<NT>::kLaunch);
  if (!registers_fit) return cudaErrorInvalidKernelImage;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv.sms * (NT == 1 ? 2 : 1), kDecMaxParts);
  static_assert(kDecMaxParts <= Kv::kCounters, "a counter per CTA");
  static_assert(2 * (size_t)kDecMaxParts * C * (D + 2) * sizeof(float) <= Kv::kPartsBytes, "two partial results per CTA");
  kernel<<<grid, kDecThreads, smem, s>>>(a, p, kv.parts(), kv.counters(), kv.err_dev);
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
  const int64_t items = (int64_t)p.ctiles * a.c.heads;
  const int64_t blocks = (int64_t)(a.sel ? a.budget : a.b.table_pages) << (a.c.page_shift - 4);
  if (items > 0x7fffffff || groups * items > 0x7fffffff / ((blocks + kDecWarps - 1) / kDecWarps))
    return cudaErrorInvalidConfiguration;  // rounds are numbered in 32 bits
  p.items = (int)items;
  p.min_rounds = 1;
  p.fail = kv.fail_next;
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
