// tcgen05 products of tiles of 128 rows and 128 tokens, for the attention kernels of prompts
// (included into an anonymous namespace after kv_operand.cuh).
#pragma once

constexpr int kPrTile = 128;  // rows of a row tile, tokens of a token tile

// K-major operand, 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Token-major (MN-major) operand, 128-byte swizzle: rows of 64 channels, 8-token
// groups 1024 bytes apart, the next 64 channels one slab (16 KB) on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)((kPrTile * 128) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ constexpr uint32_t idesc(int N, bool b_mn) {  // fp16 operands, fp32 sums
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kPrTile >> 4) << 24);
}
// The whole warp runs these, one lane (`leader`, from elect.sync) acts: without a branch around
// them the descriptors stay in uniform registers, where the instruction wants them.
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t d;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(d));
  return d;
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two fp32 in one register pair
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {  // (not rounded where an add2 of it follows: one instruction then)
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

struct PromptArgs {
  KvAttnArgs a;
  int per;        // query heads per kv head
  int tiles;      // row-tile pairs per sequence and head, at most
  int splits;     // stretches of tokens per row-tile pair, at most
  float* ws;      // [pair][split] partial results
  uint32_t* err;
  int fail;       // test hook: the first CTA's last values are not announced
};

// A pair of row tiles: its rows x0 .. of the nx of sequence s and kv head h, and its tokens.
struct PromptTile {
  int s, h;
  KvSeq q;
  int nx, x0;     // numbered in 32 bits
  int64_t first;  // position of row 0
  int cap, most;          // tokens that its last row sees
  int all, splits;        // token tiles, stretches they are cut into

  __device__ __forceinline__ PromptTile(const PromptArgs& p) {
    // heavy tiles first: the last rows of every sequence see the most
    const int hs = blockIdx.x % (p.a.c.heads * p.a.b.batch);
    const int rt = p.tiles - 1 - blockIdx.x / (p.a.c.heads * p.a.b.batch);
    h = hs % p.a.c.heads;
    s = hs / p.a.c.heads;
    q = kv_seq(p.a.b, s);
    nx = q.rows * p.per;
    x0 = rt * 2 * kPrTile;
    cap = kv_capacity(p.a.c, p.a.b);
    first = (int64_t)q.len - q.rows;
    most = x0 < nx ? seen(p, min(x0 + 2 * kPrTile, nx) - 1) : 0;
    all = (most + kPrTile - 1) / kPrTile;
    splits = min(p.splits, max(all / 2, 1));
  }
  __device__ __forceinline__ int seen(const PromptArgs& p, int x) const {  // tokens that row x sees
    const int64_t pos = first + x / p.per;
    return pos < 0 ? 0 : (int)min(p.a.causal ? pos + 1 : (int64_t)q.len, (int64_t)cap);
  }
};

// 128 query rows from x0 on of a sequence and kv head (those from nx on as zeros) as a K-major fp16 tile, by 256
// threads, two to a row; scale: what the rows' scores are multiplied by, since a row of bf16 is brought to 2^14 by
// a power of two.
template <typename T, int D>
__device__ __forceinline__ void load_queries(uint8_t* tile, float* scale, const KvAttnArgs& a, int s, int h, const KvSeq& q, int per,
                                             int x0, int nx, int tid) {
  const int r = tid >> 1, side = tid & 1, x = x0 + r;
  uint4 raw[D / 16];
#pragma unroll
  for (int n = 0; n < D / 16; ++n) raw[n] = make_uint4(0, 0, 0, 0);
  if (x < nx) {
    const uint4* src = reinterpret_cast<const uint4*>(a.q + kv_row_offset(a.b, a.qs, s, q.row0, x / per) +
                                                      (int64_t)(h * per + x % per) * a.qs.head + side * (D / 2));
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
    const int ex = (int)(top >> 7) - 127;  // an infinity or a NaN stays what it is
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
  if (side == 0) scale[r] = back;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) {
    const int ch = side * (D / 16) + n;
    *reinterpret_cast<uint4*>(tile + (ch / 8) * (kPrTile * 128) + r * 128 + ((ch % 8) ^ (r & 7)) * 16) = raw[n];
  }
}
