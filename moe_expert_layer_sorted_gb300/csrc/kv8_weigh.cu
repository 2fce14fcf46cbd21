// The weight of every token: the softmax weights of an attention's rows, summed over the rows and
// query heads that see the token, are added to the token's mass.
//
// With lse from the attention a weight is 2^(y - lse log2 e), y the score in log2 units.  Where the
// single-token kernel has written its scores (kv8_decode.cuh), a thread adds up four tokens'.  Otherwise the
// scores are made again, transposed, on the tensor cores, and the sums run along registers:
//     S^T = U_K Q^T   (128 tokens by 128 columns (row, query head) in TMEM),
// a thread having a token (a TMEM lane) and half of the columns.  A column's power of two and lse come from
// shared memory, a token's step is its thread's.  Columns that see nothing of a tile are not visited; the
// columns of a tile are dealt out to as many CTAs as fill the SMs, whose sums a second kernel adds in
// order, so that results do not depend on timing.
//
// Each CTA loads the next 128 queries while the tensor cores work on one half of TMEM and the threads on
// the other; two CTAs share an SM, so that one's barrier is covered by the other's exponents.
//
// Measured (8 kv heads of 128 channels): 4,096 rows over themselves, 32 query heads, fp16: 159 us for 2.1 million
// rows and tokens a query head; the exponents alone would take 58.  Bound by the queries' way into shared memory,
// which every token tile takes again (without it 105 us), and by the columns' constants (133).  From scores: 32 sequences
// of up to 4,160 tokens 8 us, latency.
#include "kv8_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"
#include "kv_tcgen.cuh"

constexpr int kWeThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct WeighArgs {
  KvAttnArgs a;
  float* mass;
  int per;        // query heads per kv head
  int tiles;      // token tiles of a sequence, at most
  int splits;     // CTAs per token tile and kv head
  float* parts;   // [sequence][head][tile][split][128], splits > 1
  uint32_t* err;
};

// Adds sum to the mass of token `pos` of sequence s, head h.
__device__ __forceinline__ void add_mass(const WeighArgs& w, int s, int h, int pos, float sum) {
  const int64_t pid = kv_page(w.a.c, w.a.b, s, pos >> w.a.c.page_shift);
  if (pid >= 0) w.mass[(pid * w.a.c.heads + h) * w.a.c.page_size + (pos & (w.a.c.page_size - 1))] += sum;
}

struct WeighTile {
  int s, h, t, len, nx;
  int64_t first;  // position of row 0
  KvSeq q;
  int c0, cn;     // column tiles that see something of the token tile

  __device__ __forceinline__ WeighTile(const WeighArgs& w, int index) {
    // tiles that the most rows see first
    h = index % w.a.c.heads;
    s = index / w.a.c.heads % w.a.b.batch;
    t = index / w.a.c.heads / w.a.b.batch;
    q = kv_seq(w.a.b, s);
    len = min(q.len, kv_capacity(w.a.c, w.a.b));
    nx = q.rows * w.per;
    first = (int64_t)q.len - q.rows;
    cn = c0 = 0;
    if (t * kPrTile < len && nx > 0) {
      const int64_t skip = w.a.causal ? max((int64_t)t * kPrTile - first, (int64_t)0) : max(-first, (int64_t)0);
      if (skip * w.per < nx) {
        c0 = (int)(skip * w.per / kPrTile);
        cn = (nx + kPrTile - 1) / kPrTile - c0;
      }
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWeThreads, 2) kv8_weigh_kernel(const __grid_constant__ WeighArgs w) {
  using Geo = Kv8Geom<D>;
  constexpr uint32_t kTileBytes = kPrTile * 128 * (D / 64);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done[2];                     // products of a half of TMEM
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t sh_gone;
  // (four of each: threads that are one barrier ahead write a tile's while others read the last but one's)
  __shared__ float4 sh_col[4][kPrTile / 2];        // two columns' factors and -lse log2 e
  __shared__ __align__(16) int sh_seen[4][kPrTile];              // tokens that a column sees
  __shared__ float sh_step[kPrTile], sh_sum[kPrTile];
  const KvAttnArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / w.splits, z = blockIdx.x % w.splits;
  const WeighTile tile(w, item);
  const int mine = z < tile.cn ? (tile.cn - z + w.splits - 1) / w.splits : 0;  // column tiles c0 + z, c0 + z + splits, ..
  const int base = tile.t * kPrTile;
  float* part = w.parts + ((int64_t)item * w.splits + z) * kPrTile;
  if (mine == 0) {
    if (w.splits > 1 && tid < kPrTile) part[tid] = 0.0f;
    return;
  }
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (smem - smem_addr(smem_raw));  // keys, then two query tiles
  if (tid == 0) {
    sh_gone = 0;
    mbar_init(smem_addr(&done[0]), 1);
    mbar_init(smem_addr(&done[1]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(256));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // ---- the keys: a warp takes a block of 16 tokens
  {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int pos = base + 16 * warp, kc = lane % kLanes, kr = lane / kLanes;
    const int64_t pid = pos < tile.len ? kv_page(a.c, a.b, tile.s, pos >> a.c.page_shift) : -1;
    const uint8_t* blk = a.c.pages + pid * a.c.page_stride + tile.h * a.c.head_stride +
                         ((pos & (a.c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
#pragma unroll
    for (int i = 0; i < 16 / kRows; ++i) {
      const int r = i * kRows + kr, row = 16 * warp + r;
      uint4 v = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
      if (pid >= 0) v = *reinterpret_cast<const uint4*>(blk + r * D + Geo::k_piece(r, kc) * 16);
      auto place = [&](int ch8) {
        return reinterpret_cast<uint4*>(gen + (ch8 / 8) * (kPrTile * 128) + row * 128 + ((ch8 % 8) ^ (row & 7)) * 16);
      };
      *place(2 * kc) = make_uint4(kv8_pair<0>(v.x), kv8_pair<1>(v.x), kv8_pair<0>(v.y), kv8_pair<1>(v.y));
      *place(2 * kc + 1) = make_uint4(kv8_pair<0>(v.z), kv8_pair<1>(v.z), kv8_pair<0>(v.w), kv8_pair<1>(v.w));
    }
    if (lane < 16) sh_step[16 * warp + lane] = pid >= 0 ? *reinterpret_cast<const float*>(blk + Geo::kParams) : 0.0f;
  }
  auto column = [&](int i) { return (tile.c0 + z + i * w.splits) * kPrTile; };
  // the queries of the i-th column tile, zeros where lse is not finite: asked for, and later written.  D / 8 lanes take a
  // row, a warp sixteen of them.
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kLoads = 16 / kRows;
  const int qc = lane % kLanes, qr = 16 * warp + lane / kLanes;
  uint4 raw[kLoads];
  float row_lse[kLoads];
  const uint16_t* const head = a.q + kv_row_offset(a.b, a.qs, tile.s, tile.q.row0, 0) + (int64_t)tile.h * w.per * a.qs.head + 8 * qc;
  const float* const lse = a.lse + kv_row_index(a.b, tile.s, tile.q.row0, 0) * a.q_heads + tile.h * w.per;
  auto ask = [&](int i_) {
    const int x = column(i_) + qr, i = x / w.per;
    int hq = x - i * w.per;
    const uint16_t* src = head + i * a.qs.row + hq * a.qs.head;
    const float* ls = lse + (int64_t)i * a.q_heads + hq;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      raw[n] = make_uint4(0, 0, 0, 0);
      row_lse[n] = __int_as_float(0x7fffffff);
      if (x + n * kRows < tile.nx) {
        row_lse[n] = *ls;
        raw[n] = *reinterpret_cast<const uint4*>(src);
      }
      hq += kRows;
      src += kRows * a.qs.head;
      ls += kRows;
      while (hq >= w.per) {  // the next row's first head
        hq -= w.per;
        src += a.qs.row - w.per * a.qs.head;
        ls += a.q_heads - w.per;
      }
    }
  };
  auto put = [&](int i_) {
    uint8_t* to = gen + kTileBytes * (1 + (i_ & 1)) + (qc / 8) * (kPrTile * 128);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int r = qr + n * kRows;
      const bool fine = fabsf(row_lse[n]) < __int_as_float(0x7f800000);
      if (!fine) raw[n] = make_uint4(0, 0, 0, 0);
      float back = 1.0f;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // by the power of two that brings the row to 2^14
        uint32_t v[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
        uint32_t top = __vmaxu2(__vmaxu2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu), __vmaxu2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = max(top >> 16, top & 0xffffu);
        const int ex = (int)(top >> 7) - 127;
        const int by = top == 0u || ex > 127 ? 0 : min(max(14 - ex, -113), 113);
        const float up = pow2(by);
        back = pow2(-by);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = KvType<__half>::pack(KvType<T>::lo(v[e]) * up, KvType<T>::hi(v[e]) * up);
        raw[n] = make_uint4(v[0], v[1], v[2], v[3]);
      }
      *reinterpret_cast<uint4*>(to + r * 128 + ((qc % 8) ^ (r & 7)) * 16) = raw[n];
      if (qc == 0) {
        float* col = reinterpret_cast<float*>(&sh_col[i_ & 3][r >> 1]);
        col[r & 1] = a.scale * kLog2e * back;
        col[2 + (r & 1)] = fine ? -row_lse[n] * kLog2e : -__int_as_float(0x7f800000);
      }
    }
    if (tid < kPrTile) {
      const int x = column(i_) + tid;
      const int64_t p = tile.first + x / w.per;
      sh_seen[i_ & 3][tid] = x >= tile.nx || p < 0 ? 0 : (int)min(a.causal ? p + 1 : (int64_t)tile.len, (int64_t)tile.len);
    }
  };
  const uint32_t id = idesc(kPrTile, false);
  uint32_t tm = 0;
  auto multiply = [&](int b) {  // by the first warp
    const uint32_t leader = elect_leader();
    const uint32_t qa = smem + kTileBytes * (1 + b);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_ss(leader, tm + b * kPrTile, desc_k(smem + (k / 4) * (kPrTile * 128) + (k % 4) * 32),
             desc_k(qa + (k / 4) * (kPrTile * 128) + (k % 4) * 32), id, k ? 1u : 0u);
    commit(leader, &done[b]);
  };
  ask(0);
  put(0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  tm = tmem_base;
  if (warp == 0) multiply(0);
  if (mine > 1) ask(1);

  const int quad = warp & 3, half = warp >> 2;  // the warp's lanes of TMEM, its columns of a tile
  const int token = quad * 32 + lane;
  const float ks = sh_step[token];
  const uint64_t ks2 = pair2(ks, ks);
  uint64_t sum[2] = {0, 0};
  for (int i = 0; i < mine; ++i) {
    const int b = i & 1, x0 = column(i);
    if (i + 1 < mine) {  // into the other half, whose products are done
      put(i + 1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fence_before();
      __syncthreads();
      if (warp == 0) {
        fence_after();
        multiply(b ^ 1);
      }
      if (i + 2 < mine) ask(i + 2);  // they arrive during the exponents
    }
    kv_wait(smem_addr(&done[b]), (uint32_t)(i >> 1) & 1u, &sh_gone, w.err);
    fence_after();
    const uint32_t ts = tm + b * kPrTile + half * 64 + ((uint32_t)(quad * 32) << 16);
    auto consume = [&](auto masked_) {
      constexpr bool masked = decltype(masked_)::value;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[32];
        tmem_ld32(ts + 32 * k, v);
        tmem_wait_ld();
        const float4* col = &sh_col[i & 3][half * 32 + 16 * k];
        const int2* seen = reinterpret_cast<const int2*>(&sh_seen[i & 3][half * 64 + 32 * k]);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float4 f = col[e / 2];
          uint64_t y = mul2(pair2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), pair2(f.x, f.y));
          y = fma2(y, ks2, pair2(f.z, f.w));
          float y0, y1;
          split2(y, y0, y1);
          y0 = exp2_fast(y0);
          y1 = exp2_fast(y1);
          if constexpr (masked) {
            const int2 n = seen[e / 2];
            y0 = base + token < n.x ? y0 : 0.0f;
            y1 = base + token < n.y ? y1 : 0.0f;
          }
          sum[e / 2 & 1] = add2(sum[e / 2 & 1], pair2(y0, y1));
        }
      }
    };
    // every column sees the whole token tile?
    if (tile.first + x0 / w.per >= base + kPrTile - 1 || (!a.causal && tile.first >= 0)) consume(std::false_type());
    else consume(std::true_type());
  }
  float s0, s1;
  split2(add2(sum[0], sum[1]), s0, s1);
  if (half) sh_sum[token] = s0 + s1;
  fence_before();
  __syncthreads();
  if (!half) {
    const float all = (s0 + s1) + sh_sum[token];
    if (w.splits > 1) part[token] = all;
    else if (base + token < tile.len) add_mass(w, tile.s, tile.h, base + token, all);
  }
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(256));
  }
}

// Adds the sums of a token tile's CTAs, in order.
__global__ void __launch_bounds__(kPrTile) kv8_weigh_join_kernel(const __grid_constant__ WeighArgs w) {
  const WeighTile tile(w, blockIdx.x);
  const int pos = tile.t * kPrTile + threadIdx.x;
  if (tile.cn == 0 || pos >= tile.len) return;
  const float* part = w.parts + (int64_t)blockIdx.x * w.splits * kPrTile + threadIdx.x;
  float sum = 0.0f;
#pragma unroll 8
  for (int z = 0; z < w.splits; ++z) sum += part[z * kPrTile];
  add_mass(w, tile.s, tile.h, pos, sum);
}

// From the scores that the single-token kernel wrote: a thread adds up the columns of four tokens (of one page).
constexpr int kWeTokens = 4 * kWeThreads;
__global__ void __launch_bounds__(kWeThreads) kv8_weigh_scores_kernel(const __grid_constant__ WeighArgs w, const float* __restrict__ scores,
                                                                      int width, int chunks) {
  __shared__ float sh_lse[kKv8Columns];
  const KvAttnArgs& a = w.a;
  const int h = blockIdx.x % a.c.heads, s = blockIdx.x / a.c.heads / chunks, chunk = blockIdx.x / a.c.heads % chunks;
  const KvSeq q = kv_seq(a.b, s);
  const int cols = min(q.rows * w.per, kKv8Columns), len = min(q.len, kv_capacity(a.c, a.b));
  if ((int64_t)chunk * kWeTokens >= len) return;
  if ((int)threadIdx.x < cols) {
    const float ls = a.lse[kv_row_index(a.b, s, q.row0, threadIdx.x / w.per) * a.q_heads + h * w.per + threadIdx.x % w.per];
    sh_lse[threadIdx.x] = fabsf(ls) < __int_as_float(0x7f800000) ? ls * kLog2e : __int_as_float(0x7f800000);
  }
  const int pos = chunk * kWeTokens + 4 * threadIdx.x, n = min(len - pos, 4);
  const int64_t pid = n > 0 ? kv_page(a.c, a.b, s, pos >> a.c.page_shift) : -1;
  __syncthreads();
  if (pid < 0) return;
  float* mass = w.mass + (pid * a.c.heads + h) * a.c.page_size + (pos & (a.c.page_size - 1));
  const float4* y = reinterpret_cast<const float4*>(scores + (((int64_t)s * a.c.heads + h) * kv_capacity(a.c, a.b) + pos) * width);
  const float4 had = *reinterpret_cast<const float4*>(mass);
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int x = 0; x < cols; x += 4) {
    float4 v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = y[(t * width + x) / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ls = x + i < cols ? sh_lse[x + i] : __int_as_float(0x7f800000);
      if (ls == __int_as_float(0x7f800000)) continue;
#pragma unroll
      for (int t = 0; t < 4; ++t) sum[t] += exp2_fast((i == 0 ? v[t].x : i == 1 ? v[t].y : i == 2 ? v[t].z : v[t].w) - ls);
    }
  }
  const float now[4] = {had.x + sum[0], had.y + sum[1], had.z + sum[2], had.w + sum[3]};
  if (n == 4) {
    *reinterpret_cast<float4*>(mass) = make_float4(now[0], now[1], now[2], now[3]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t < n) mass[t] = now[t];
  }
}

}  // namespace

cudaError_t moe::kv8_weigh(Kv8& kv, const KvAttnArgs& a, float* mass, const float* scores, cudaStream_t s) {
  WeighArgs w{a, mass, a.q_heads / a.c.heads, 0, 1, kv.parts(), kv.err_dev};
  const int64_t cap = std::min<int64_t>((int64_t)a.b.table_pages << a.c.page_shift, 0x7ffff000);
  if (scores) {
    const int64_t chunks = (cap + kWeTokens - 1) / kWeTokens, ctas = chunks * a.c.heads * a.b.batch;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv8_weigh_scores_kernel<<<(unsigned)ctas, kWeThreads, 0, s>>>(w, scores, score_width(a), (int)chunks);
    return cudaGetLastError();
  }
  const int64_t tiles = (cap + kPrTile - 1) / kPrTile, items = tiles * a.c.heads * a.b.batch;
  const int64_t columns = ((int64_t)a.b.max_new * w.per + kPrTile - 1) / kPrTile;
  if (items > 0x7fffffff || columns * kPrTile > 0x7fffffff) return cudaErrorInvalidConfiguration;
  w.tiles = (int)tiles;
  // CTAs enough for four rounds of the SMs, which hold two each; their sums have to fit the workspace
  const int64_t want = std::min<int64_t>((8 * (int64_t)kv.sms + items - 1) / items, columns);
  const int64_t room = (int64_t)(Kv8::kPartsBytes / (kPrTile * sizeof(float))) / items;
  w.splits = (int)std::max<int64_t>(std::min(want, room), 1);
  if (items * w.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV8_DISPATCH(kv.d, {
    const size_t smem = std::max<size_t>(1024 + (size_t)3 * kPrTile * D * 2, 80 << 10);  // two CTAs an SM, as many as TMEM holds
    const auto kernel = kv8_weigh_kernel<T, D>;
    e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e == cudaSuccess) {
      kernel<<<(unsigned)(items * w.splits), kWeThreads, smem, s>>>(w);
      e = cudaGetLastError();
    }
  });
  if (e == cudaSuccess && w.splits > 1) {
    kv8_weigh_join_kernel<<<(unsigned)items, kPrTile, 0, s>>>(w);
    e = cudaGetLastError();
  }
  return e;
}
