// Attention of few rows: the line of rounds that its work is cut into, and what else the single-token
// kernels of the caches share (included into an anonymous namespace after kv_operand.cuh).
#pragma once

constexpr int kDecWarps = 8;  // that compute

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
