// The weight of every token: the softmax weights of an attention's rows, summed over the rows and
// query heads that see the token, are added to the token's mass.
//
// With the reference r of a row and its sum of weights l from the attention (Kv8Scores) a weight is 2^(y - r) / l, y the
// score in log2 units, rounded as there: whatever the size of the scores, a row's weights are those that the attention took, and
// come to 1.  (Or 2^(y - lse log2 e), which is off by |lse| 2^-23, for rows of scores below kKv8Coarse.)  Where the
// single-token kernel has written its scores (kv8_decode.cuh), a thread adds up four tokens'.  Otherwise the
// scores are made again, transposed, on the tensor cores, and the sums run along registers:
//     S^T = U_K Q^T   (twice 128 tokens by 128 columns (row, query head) in TMEM),
// a thread having a token (a TMEM lane) and half of the columns.  A column's power of two and lse come from
// shared memory, a token's step is its thread's.  Columns that see nothing of a tile are not visited.  All the batch's
// work (sequence, head, 256 tokens, 128 columns) lies in one line that is cut into equal shares, a CTA each SM, so that
// neither the table's size nor uneven sequences matter; a token tile that is cut between CTAs is added up by the one
// that finishes it last, in the order of the CTAs, so results do not depend on timing.  (A grid over the table's
// tiles took 1,500 us for 32 single tokens whose table could hold 131,072.)
//
// Each CTA loads the next 128 queries while the tensor cores work on one half of TMEM and the threads on
// the other.
//
// Measured (8 kv heads of 128 channels): 4,096 rows over themselves, 32 query heads, fp16: 149 us for 2.1 million
// rows and tokens a query head; the exponents alone would take 58.  Bound by instructions, those that bring the queries to
// shared memory among them: 128 tokens a CTA and two CTAs an SM, which did that twice as often, took 162.  From scores: 32
// sequences of up to 4,160 tokens 8 us, latency.
#include "kv8_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"
#include "kv_tcgen.cuh"

constexpr int kWeThreads = 512, kWeWarps = kWeThreads / 32;
constexpr int kWeTile = 256;  // tokens of a CTA at a time, two tiles of the tensor cores
constexpr float kLog2e = 1.4426950408889634f;

// A token tile's first products wait for its keys: it counts as so many more pieces of work, behind its own.  Measured,
// 4,096 rows over themselves, tiles of 128 tokens: 166 us without, 162 with 1 or 2, 164 with 4.
constexpr int kWeTurn = 1;

struct WeighArgs {
  KvAttnArgs a;
  float* mass;
  int per;             // query heads per kv head
  const float2* refs;  // of the first refs_limit rows and query heads
  int64_t refs_limit;
  const int* scored;   // nullptr, or >= 0 for sequences whose scores were left (kv8_weigh_scores_kernel takes those)
  float* parts;        // [CTA][2][kWeTile]
  unsigned* counters;  // a CTA each, zero between calls
  uint32_t* err;
  int fail;            // test hook: the first CTA's first products are not announced
};
static_assert(2 * size_t(Kv8::kCounters) * kWeTile * sizeof(float) <= Kv8::kFewPartsBytes, "two partial results per CTA");

// Adds sum to the mass of token `pos` of sequence s, head h.
__device__ __forceinline__ void add_mass(const WeighArgs& w, int s, int h, int pos, float sum) {
  const int64_t pid = kv_page(w.a.c, w.a.b, s, pos >> w.a.c.page_shift);
  if (pid >= 0) w.mass[(pid * w.a.c.heads + h) * w.a.c.page_size + (pos & (w.a.c.page_size - 1))] += sum;
}

// Reference and 1 / sum of a row and query head, and whether it adds anything (rows whose results are not finite do not).
__device__ __forceinline__ float2 reference(const WeighArgs& w, int64_t row) {
  if (row < w.refs_limit) return w.refs[row];
  const float lse = w.a.lse[row];
  return make_float2(lse * kLog2e, 1.0f);
}
__device__ __forceinline__ bool adds(float2 ref) {
  constexpr uint32_t kInf = 0x7f800000u;
  return fabsf(ref.x) < __uint_as_float(kInf) && ref.y > 0.0f && ref.y < __uint_as_float(kInf);
}

// A sequence's pieces of work: for each head and tile of kWeTile tokens, the tiles of 128 columns that see some of it.  Tile t
// is seen by column tiles c0(t) .. n - 1, c0(t) = max(0, step t - skip): causal, row i sees it from i = kWeTile t - first on, so
// columns from per (kWeTile t - first) on, and kWeTile t per / 128 is whole.  Sums of c0 over tiles have a closed form.
struct WeighSeq {
  KvSeq q;
  int len, tiles, n, step;
  int64_t first, skip;  // position of row 0
  WeighSeq() = default;
  __device__ __forceinline__ WeighSeq(const WeighArgs& w, int s) {
    q = kv_seq(w.a.b, s);
    len = min(q.len, kv_capacity(w.a.c, w.a.b));
    first = (int64_t)q.len - q.rows;
    n = (int)(((int64_t)q.rows * w.per + kPrTile - 1) / kPrTile);
    tiles = n && !(w.scored && w.scored[s] >= 0) ? (len + kWeTile - 1) / kWeTile : 0;
    step = w.a.causal ? kWeTile / kPrTile * w.per : 0;
    const int64_t before = (w.a.causal ? first : min(first, (int64_t)0)) * w.per;  // rounded up, below zero too
    skip = before >= 0 ? (before + kPrTile - 1) / kPrTile : -(-before / kPrTile);
  }
  __device__ __forceinline__ int c0(int t) const { return (int)max((int64_t)t * step - skip, (int64_t)0); }
  __device__ __forceinline__ int64_t before(int t) const {  // column tiles of the token tiles below t
    int64_t out = 0;
    if (step == 0) {
      out = t * max(-skip, (int64_t)0);
    } else {
      const int64_t t1 = skip < 0 ? 0 : skip / step + 1;  // the first tile that some do not see
      if (t > t1) out = step * ((t - 1) * (int64_t)t / 2 - (t1 - 1) * t1 / 2) - skip * (t - t1);
    }
    return (int64_t)(n + kWeTurn) * t - out;
  }
};

// CTAs that share a line of pieces, a token tile of one column tile each at least.
__device__ __forceinline__ int weigh_ctas(int64_t total) { return (int)min((int64_t)gridDim.x, total / (1 + kWeTurn)); }

// A place in the line of pieces, which runs over the sequences, their heads, their token tiles and the column tiles.
struct WeighPlace {
  int s, h, t;
  int64_t tile;  // number of the token tile's first piece
};

// The work at hand: `count` column tiles from c on of a token tile.
struct WeighItem {
  WeighPlace at;
  WeighSeq q;
  int nx, c, count, pieces;  // columns of the sequence; pieces: of the token tile
};

// The weights of 64 columns from x0 on for token `pos` of step ks, with the rows' own references and sums, and the scores as the
// attention rounds them.  (A call, so that the ordinary tiles' registers stay what they are.)
__device__ __noinline__ float coarse_weights(const WeighArgs& w, const WeighItem& it, uint32_t ts, int x0, const float4* col, const int* seen,
                                             int pos, float ks) {
  const int64_t row0 = kv_row_index(w.a.b, it.at.s, it.q.q.row0, 0) * w.a.q_heads + it.at.h * w.per;
  float sum = 0.0f;
#pragma unroll 1
  for (int k = 0; k < 64; k += 32) {
    uint32_t v[32];
    tmem_ld32(ts + k, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int x = x0 + k + e, row = x / w.per;
      const float2 ref = x < it.nx ? reference(w, row0 + (int64_t)row * w.a.q_heads + (x - row * w.per)) : make_float2(0.0f, 0.0f);
      if (!adds(ref) || pos >= seen[k + e]) continue;
      const float f = reinterpret_cast<const float*>(col + (k + e) / 2)[e & 1] * ks;
      sum = fmaf(exp2_fast(__fadd_rn(__fmul_rn(__uint_as_float(v[e]), f), -ref.x)), ref.y, sum);
    }
  }
  return sum;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWeThreads, 1) kv8_weigh_kernel(const __grid_constant__ WeighArgs w) {
  using Geo = Kv8Geom<D>;
  constexpr uint32_t kTileBytes = kPrTile * 128 * (D / 64);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done[2];                     // products of a half of TMEM
  __shared__ uint64_t drained;                     // all of them, after a wait that gave up
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t sh_gone;                     // a wait gave up: nothing more is multiplied or added to mass
  enum : uint32_t { kNothing, kSome, kEvery };
  // (four of each: threads that are one barrier ahead write a tile's while others read the last but one's)
  __shared__ float4 sh_col[4][kPrTile / 2];        // two columns' factors and -lse log2 e
  __shared__ uint4 sh_mode[4];                     // what its columns see of either half of the tokens; whether coarse_weights takes it
  __shared__ __align__(16) int sh_seen[4][kPrTile];              // tokens that a column sees
  __shared__ float sh_step[kWeTile], sh_sum[kWeTile];
  __shared__ WeighItem sh;
  __shared__ int64_t sh_scan[kWeWarps], sh_base;
  __shared__ volatile int64_t line[3];  // the share's first piece, its end, the end of all (not in registers)
  __shared__ int sh_seq;
  __shared__ unsigned sh_last;
  const KvAttnArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- the CTA's share of the line, and the sequence that it begins in
  int64_t total = 0, first = 0, last = 0;
  for (int pass = 0; pass < 2; ++pass) {  // the sum; the sequence
    int64_t before = 0;
    for (int g0 = 0; g0 < a.b.batch; g0 += kWeThreads) {
      int64_t mine = 0;
      if (g0 + tid < a.b.batch) {
        const WeighSeq q(w, g0 + tid);
        mine = q.before(q.tiles) * a.c.heads;
      }
      int64_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) sh_scan[warp] = upto;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int y = 0; y < kWeWarps; ++y) {
        if (y < warp) upto += sh_scan[y];
        all += sh_scan[y];
      }
      upto += before;
      if (pass && upto - mine <= first && first < upto) {
        sh_seq = g0 + tid;
        sh_base = upto - mine;
      }
      before += all;
    }
    if (pass == 0) {
      total = before;
      const int64_t n = weigh_ctas(total);
      if (blockIdx.x >= n) return;
      first = total * blockIdx.x / n;
      last = total * (blockIdx.x + 1) / n;
    }
  }
  if (tid == 0) {
    line[0] = first;
    line[1] = last;
    line[2] = total;
  }
  __syncthreads();
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (smem - smem_addr(smem_raw));  // two tiles of keys, then two of queries
  if (tid == 0) {
    sh_gone = sh_mode[0].z = 0;
    mbar_init(smem_addr(&done[0]), 1);
    mbar_init(smem_addr(&done[1]), 1);
    mbar_init(smem_addr(&drained), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const uint32_t id = idesc(kPrTile, false);
  uint32_t tm = 0;
  uint32_t parity = 0;  // a bit per half of TMEM; the next one: a wait of this thread gave up
  auto gone = [&]() { return *static_cast<volatile uint32_t*>(&sh_gone) != 0; };
  auto multiply = [&](int b, bool announce = true) {  // by the first warp
    if (__any_sync(0xffffffffu, parity & 4u)) return;
    const uint32_t leader = elect_leader();
    const uint32_t qa = smem + kTileBytes * (2 + b);
#pragma unroll
    for (int y = 0; y < kWeTile / kPrTile; ++y)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(leader, tm + b * kWeTile + y * kPrTile, desc_k(smem + y * kTileBytes + (k / 4) * (kPrTile * 128) + (k % 4) * 32),
               desc_k(qa + (k / 4) * (kPrTile * 128) + (k % 4) * 32), id, k ? 1u : 0u);
    if (announce) commit(leader, &done[b]);
  };
  fence_before();
  __syncthreads();
  fence_after();
  tm = tmem_base;
  // the warp's lanes of TMEM, its columns of a tile, its tile of tokens
  const int quad = warp & 3, half = warp >> 2 & 1, part = warp >> 3;
  const int token = part * kPrTile + quad * 32 + lane;
  for (int64_t u = line[0]; u < line[1];) {
    if (tid == 0) {
      WeighPlace at = sh.at;
      if (u == line[0]) {
        at.s = sh_seq;
        const WeighSeq q(w, at.s);
        sh.q = q;
        const int64_t head = q.before(q.tiles);
        at.h = (int)((u - sh_base) / head);
        const int64_t in_head = (u - sh_base) - at.h * head;
        int t0 = 0, t1 = q.tiles;  // the last tile with before(t) <= in_head lies in t0 .. t1 - 1
        while (t1 - t0 > 1) {
          const int mid = (t0 + t1) / 2;
          if (q.before(mid) <= in_head) t0 = mid;
          else t1 = mid;
        }
        at.t = t0;
        at.tile = u - (in_head - q.before(t0));
      } else {  // a token tile's first piece
        at.tile = u;
        if (++at.t == sh.q.tiles) {
          at.t = 0;
          if (++at.h == a.c.heads) {
            at.h = 0;
            do sh.q = WeighSeq(w, ++at.s);
            while (sh.q.tiles == 0);  // (there is one, the line goes on)
          }
        }
      }
      sh.at = at;
      sh.nx = sh.q.q.rows * w.per;
      const int c0 = sh.q.c0(at.t);
      sh.pieces = sh.q.n + kWeTurn - c0;
      sh.c = c0 + (int)(u - at.tile);
      sh.count = (int)(min(at.tile + sh.pieces, line[1]) - u);
    }
    __syncthreads();
    const int base = sh.at.t * kWeTile, mine = min(sh.count, sh.q.n - sh.c);  // what is not the change to the tile
    auto column = [&](int i) { return (sh.c + i) * kPrTile; };
    // the queries of the i-th column tile, zeros where lse is not finite: asked for, and later written.  D / 8 lanes take a
    // row, a warp eight of them.
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kLoads = kPrTile / kWeWarps / kRows;
    const int qc = lane % kLanes, qr = kPrTile / kWeWarps * warp + lane / kLanes;
    uint4 raw[kLoads];
    float row_lse[kLoads];
    const uint16_t* const head = a.q + kv_row_offset(a.b, a.qs, sh.at.s, sh.q.q.row0, 0) + (int64_t)sh.at.h * w.per * a.qs.head + 8 * qc;
    const float* const lse = a.lse + kv_row_index(a.b, sh.at.s, sh.q.q.row0, 0) * a.q_heads + sh.at.h * w.per;
    auto ask = [&](int i_) {
      const int x = column(i_) + qr, i = x / w.per;
      int hq = x - i * w.per;
      const uint16_t* src = head + i * a.qs.row + hq * a.qs.head;
      const float* ls = lse + (int64_t)i * a.q_heads + hq;
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        raw[n] = make_uint4(0, 0, 0, 0);
        row_lse[n] = __int_as_float(0x7fffffff);
        if (x + n * kRows < sh.nx) {
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
      uint8_t* to = gen + kTileBytes * (2 + (i_ & 1)) + (qc / 8) * (kPrTile * 128);
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
          const float f = a.scale * kLog2e * back;
          if (fine && (fabsf(row_lse[n]) * kLog2e >= kKv8Coarse || !(fabsf(f) >= 0x1p-64f && fabsf(f) <= 0x1p64f))) sh_mode[i_ & 3].z = 1;
          float* col = reinterpret_cast<float*>(&sh_col[i_ & 3][r >> 1]);
          col[r & 1] = fine ? f : 0.0f;  // (the scale may be so large that the product is not finite)
          col[2 + (r & 1)] = fine ? -row_lse[n] * kLog2e : -__int_as_float(0x7f800000);
        }
      }
      if (tid < kPrTile) {
        const int x = column(i_) + tid;
        const int64_t p = sh.q.first + x / w.per;
        sh_seen[i_ & 3][tid] = x >= sh.nx || p < 0 ? 0 : (int)min(a.causal ? p + 1 : (int64_t)sh.q.len, (int64_t)sh.q.len);
      }
      if (tid < kWeTile / kPrTile) {
        const int low = base + tid * kPrTile, x0 = column(i_);
        const bool none = a.causal && sh.q.first + (x0 + kPrTile - 1) / w.per < low;
        const bool every = sh.q.first + x0 / w.per >= low + kPrTile - 1 || (!a.causal && sh.q.first >= 0);
        reinterpret_cast<uint32_t*>(&sh_mode[i_ & 3])[tid] = none ? kNothing : every ? kEvery : kSome;
        if (tid == 0) sh_mode[(i_ + 1) & 3].z = 0;  // (of three column tiles ago)
      }
    };
    if (mine > 0) {
      ask(0);
      // ---- the keys: a warp takes a block of 16 tokens
      {
        constexpr int kLanes = D / 16, kRows = 32 / kLanes;
        const int pos = base + 16 * warp, kc = lane % kLanes, kr = lane / kLanes;
        const int64_t pid = pos < sh.q.len ? kv_page(a.c, a.b, sh.at.s, pos >> a.c.page_shift) : -1;
        const uint8_t* blk = a.c.pages + pid * a.c.page_stride + sh.at.h * a.c.head_stride +
                             ((pos & (a.c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
#pragma unroll
        for (int i = 0; i < 16 / kRows; ++i) {
          const int r = i * kRows + kr, row = 16 * warp + r;
          uint4 v = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          if (pid >= 0) v = *reinterpret_cast<const uint4*>(blk + r * D + Geo::k_piece(r, kc) * 16);
          auto place = [&](int ch8) {
            return reinterpret_cast<uint4*>(gen + part * kTileBytes + (ch8 / 8) * (kPrTile * 128) + (row & (kPrTile - 1)) * 128 +
                                          ((ch8 % 8) ^ (row & 7)) * 16);
          };
          *place(2 * kc) = make_uint4(kv8_pair<0>(v.x), kv8_pair<1>(v.x), kv8_pair<0>(v.y), kv8_pair<1>(v.y));
          *place(2 * kc + 1) = make_uint4(kv8_pair<0>(v.z), kv8_pair<1>(v.z), kv8_pair<0>(v.w), kv8_pair<1>(v.w));
        }
        if (lane < 16) sh_step[16 * warp + lane] = pid >= 0 ? *reinterpret_cast<const float*>(blk + Geo::kParams) : 0.0f;
      }
      put(0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fence_before();
      __syncthreads();
      if (warp == 0) {
        fence_after();
        multiply(0, !(w.fail && blockIdx.x == 0 && u == line[0]));
      }
      if (mine > 1) ask(1);
    }

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
      if (!kv_wait(smem_addr(&done[b]), parity >> b & 1u, &sh_gone, w.err)) parity |= 4u;
      parity ^= 1u << b;
      fence_after();
      const uint32_t ts = tm + b * kWeTile + part * kPrTile + half * 64 + ((uint32_t)(quad * 32) << 16);
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
      const uint4 modes = sh_mode[i & 3];
      const uint32_t mode = part ? modes.y : modes.x;
      if (mode == kNothing) continue;
      if (modes.z)
        sum[0] = add2(sum[0], pair2(coarse_weights(w, sh, ts, x0 + half * 64, &sh_col[i & 3][half * 32], &sh_seen[i & 3][half * 64], base + token, ks), 0.0f));
      else if (mode == kEvery) consume(std::false_type());
      else consume(std::true_type());
    }
    float s0, s1;
    split2(add2(sum[0], sum[1]), s0, s1);
    if (half) sh_sum[token] = s0 + s1;
    fence_before();
    __syncthreads();
    // a token tile that is cut between CTAs: sums of a CTA's first stretch in slot 0, of its last in slot 1, and who
    // finishes the tile last adds them in order; sums of a CTA of which a wait gave up are NaN, and are added to nothing
    const bool whole = sh.count == sh.pieces;
    const int64_t tile = sh.at.tile, tile_end = tile + sh.pieces;
    if (!half) {
      const float all = gone() ? __int_as_float(0x7fffffff) : (s0 + s1) + sh_sum[token];
      if (!whole) w.parts[(int64_t)(2 * blockIdx.x + (u == line[0] ? 0 : 1)) * kWeTile + token] = all;
      else if (base + token < sh.q.len && all == all) add_mass(w, sh.at.s, sh.at.h, base + token, all);
    }
    if (!whole) {
      const int64_t total = line[2];
      const int n = weigh_ctas(total);
      const int c0 = (int)(((tile + 1) * n - 1) / total), c1 = (int)((tile_end * n - 1) / total);  // whose shares hold its ends
      __syncthreads();  // every thread's part is written: one release covers them
      if (tid == 0) sh_last = add_acq_rel(&w.counters[c0]);
      __syncthreads();
      if (sh_last == (unsigned)(c1 - c0)) {
        if (tid < kWeTile && base + tid < sh.q.len) {
          float sum_ = 0.0f;
#pragma unroll 8
          for (int y = c0; y <= c1; ++y)
            sum_ += __ldcg(w.parts + (int64_t)(2 * y + (y == c0 && tile != total * c0 / n ? 1 : 0)) * kWeTile + tid);
          if (sum_ == sum_) add_mass(w, sh.at.s, sh.at.h, base + tid, sum_);
        }
        if (tid == 0) w.counters[c0] = 0;  // for the next call
      }
    }
    u += sh.count;
    if (tid == 0) sh_mode[0].z = 0;
    __syncthreads();  // what this tile had in shared memory is the next one's
  }
  if (warp == 0) {
    fence_after();
    if (gone()) {  // products that nobody waited for end before their operands, their barriers and TMEM do
      commit(elect_leader(), &drained);
      mbar_drain(smem_addr(&drained), 0);
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(512));
  }
}

// From the scores that the single-token kernel wrote: a thread adds up the columns of four tokens (of one page).
constexpr int kScThreads = 256, kWeTokens = 4 * kScThreads;
__global__ void __launch_bounds__(kScThreads) kv8_weigh_scores_kernel(const __grid_constant__ WeighArgs w, const __grid_constant__ Kv8Scores scores,
                                                                      int ctas) {
  __shared__ float2 sh_col[kKv8Columns];
  const KvAttnArgs& a = w.a;
  const int h = blockIdx.x % a.c.heads, s = blockIdx.x / a.c.heads / ctas, z = blockIdx.x / a.c.heads % ctas;
  const KvSeq q = kv_seq(a.b, s);
  const int cols = min(q.rows * w.per, kKv8Columns), len = min(q.len, kv_capacity(a.c, a.b));
  if (q.rows == 0 || (int64_t)z * kWeTokens >= len) return;
  const int line = scores.base[s], width = scores.width, rounds = (len + kPrTile - 1) / kPrTile;
  if (line < 0) return;
  if ((int)threadIdx.x < cols) {
    const float2 ref = reference(w, kv_row_index(a.b, s, q.row0, threadIdx.x / w.per) * a.q_heads + h * w.per + threadIdx.x % w.per);
    sh_col[threadIdx.x] = adds(ref) ? ref : make_float2(0.0f, 0.0f);
  }
  __syncthreads();
  for (int64_t at = (int64_t)z * kWeTokens; at < len; at += (int64_t)ctas * kWeTokens) {
    const int pos = (int)at + 4 * threadIdx.x, n = min(len - pos, 4);
    const int64_t pid = n > 0 ? kv_page(a.c, a.b, s, pos >> a.c.page_shift) : -1;
    if (pid < 0) continue;
    float* mass = w.mass + (pid * a.c.heads + h) * a.c.page_size + (pos & (a.c.page_size - 1));
    const float4 had = *reinterpret_cast<const float4*>(mass);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int x = 0; x < cols; x += 4) {
      const int64_t round = line + (int64_t)(h * scores.ctiles + (x >> 4)) * rounds + pos / kPrTile;
      const float* y = scores.to + (round * kPrTile + (pos & (kPrTile - 1))) * width + (x & 15);
      float4 v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = *reinterpret_cast<const float4*>(y + t * width);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ref = x + i < cols ? sh_col[x + i] : make_float2(0.0f, 0.0f);
        if (ref.y == 0.0f) continue;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          sum[t] = fmaf(exp2_fast((i == 0 ? v[t].x : i == 1 ? v[t].y : i == 2 ? v[t].z : v[t].w) - ref.x), ref.y, sum[t]);
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
}

}  // namespace

cudaError_t moe::kv8_weigh(Kv8& kv, const KvAttnArgs& a, float* mass, const Kv8Scores& scores, cudaStream_t s) {
  WeighArgs w{a, mass, a.q_heads / a.c.heads, scores.refs, scores.refs_limit, scores.base, kv.parts(), kv.counters(), kv.err_dev, kv.fail_next};
  const int64_t cap = std::min<int64_t>((int64_t)a.b.table_pages << a.c.page_shift, 0x7ffff000);
  if (scores.base) {
    // a CTA for 1,024 tokens that the table could hold; of many, one that goes on to the next ones (an idle CTA takes 0.5 ns)
    const int64_t items = (int64_t)a.c.heads * a.b.batch;
    const int64_t ctas = std::min<int64_t>((cap + kWeTokens - 1) / kWeTokens, std::max<int64_t>(8192 / items, 1));
    if (items * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv8_weigh_scores_kernel<<<(unsigned)(items * ctas), kScThreads, 0, s>>>(w, scores, (int)ctas);
    const cudaError_t e = cudaGetLastError();
    const int64_t rounds = (cap + kPrTile - 1) / kPrTile;
    if (e != cudaSuccess || items * scores.ctiles <= scores.limit / rounds) return e;  // there was room for all of them
  }
  if ((int64_t)a.b.max_new * w.per > 0x7fffffff - kPrTile) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV8_DISPATCH(kv.d, {
    const size_t smem = std::max<size_t>(1024 + (size_t)4 * kPrTile * D * 2, 120 << 10);  // one CTA an SM, as many as TMEM holds
    const auto kernel = kv8_weigh_kernel<T, D>;
    e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e == cudaSuccess) {
      kernel<<<(unsigned)std::min(kv.sms, Kv8::kCounters), kWeThreads, smem, s>>>(w);
      e = cudaGetLastError();
    }
  });
  return e;
}
