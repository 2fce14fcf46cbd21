// Eviction from the 8-bit cache by accumulated weight: of every sequence and kv head the first and
// the last tokens and those of the largest mass stay, and move together.
//
// One cluster per (sequence, kv head), its CTAs sharing the tokens.
//   Choice: order-preserving 32-bit keys of the masses, kept in shared memory where they fit; the key
//   of the last token that is taken by three histograms of 11, 11 and 10 bits, added up over the
//   cluster through distributed shared memory; then one ordered pass counts, and one writes the kept
//   positions.
//   Moving: sixteen kept tokens make a new block, whose step is the largest of theirs.  A token moves
//   to a lower position or stays, so blocks are made in rounds, one per warp of the cluster: all of a
//   round have been read before any is written, and no later round reads what this one overwrites.  The
//   next round's words are asked for before this one's barrier is waited for.
//
// Measured (8 heads of 128 channels, caches whose tokens have not been moved before): 32 sequences of up to 4,608 tokens
// to 4,096 each 207 us (choice 28), 0.5 GB read and written; one of 131,072 to 65,536 232 us (choice 58), of which half the
// SMs have no part: the sixteen CTAs of a head's cluster share eight of them.  Bound by the rounds' chain of loads and
// by the turning of codes (50 us of either).
#include <cooperative_groups.h>

#include "kv8_internal.h"

using namespace moe;
namespace cg = cooperative_groups;

namespace {

constexpr int kEvThreads = 256, kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvKeys = 16384;  // that a CTA keeps in shared memory; of longer shares they are read again
constexpr int kEvMaxCluster = 16;

// Order-preserving key of a mass (-0 and +0 equal), NaN as -infinity.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) v = -__int_as_float(0x7f800000);
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Head {  // a sequence's kv head
  const Kv8EvictArgs& a;
  int s, h;
  __device__ __forceinline__ int64_t page(int j) const { return kv_page(a.c, a.b, s, j >> a.c.page_shift); }
  __device__ __forceinline__ int in_page(int j) const { return j & (a.c.page_size - 1); }
  __device__ __forceinline__ float* mass(int64_t pid, int j) const {
    return a.mass + (pid * a.c.heads + h) * a.c.page_size + in_page(j);
  }
  __device__ __forceinline__ uint8_t* block(int64_t pid, int j, int bytes) const {
    return a.c.pages + pid * a.c.page_stride + h * a.c.head_stride + (in_page(j) >> 4) * (int64_t)bytes;
  }
};

// Inclusive prefix sum of v over the CTA.
__device__ __forceinline__ int cta_scan(int v, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w)
    if (w < warp) v += sh[w];
  return v;
}

// What a token's codes of step s are multiplied with to become codes of step `to` >= s, so that a product rounded to a
// whole number in fp32 is u s / to to the nearest one; ties: the quotients' halves are to be told apart by turn_words.
//
// s / to itself, rounded, is wrong near halves, and these are not rare: steps are 127ths of 16-bit numbers, and the
// quotients of their codes halves of fractions with small denominators, but for a few 2^-24.  If some u s / to is within
// 2e-5 of a half, s / to is within 2e-5 / u of a fraction p / q with q <= 254, which is then the last of its continued
// fraction's convergents with such a q (and the only such fraction).  All quotients near halves then lie on the same
// side of them, s / to's side of p / q (mirrored for negative u): a ratio moved by 2^-20 that way rounds all of them
// rightly, and every other code, which is at least 1 / (2 q) from a half, as before.  Where s / to is p / q they are ties.
struct Ratio {
  float r;
  bool ties;  // and r is not exact
};
__device__ __forceinline__ Ratio ratio_of(float s, float to) {
  const float up = kv8_lift(to);
  s *= up;
  to *= up;
  if (!(s < to) || s == 0.0f) return {s < to ? 0.0f : 1.0f, false};
  const float r = __fdiv_rn(s, to);
  const uint32_t sb = __float_as_uint(s), tb = __float_as_uint(to);
  const int d = (int)(tb >> 23) - (int)(sb >> 23);
  if (d > 8) return {0.0f, false};  // below a half with every code
  // s / to = S / T in whole numbers of up to 24 and 32 bits
  const uint32_t S = (sb & 0x7fffffu) | 0x800000u, T = ((tb & 0x7fffffu) | 0x800000u) << d;
  uint32_t a = T, b = S, p0 = 1, q0 = 0, p = 0, q = 1;
  while (b != 0) {
    const uint32_t k = a / b, left = a - k * b;
    if (k > 254u || k * q + q0 > 254u) break;
    a = b;
    b = left;
    const uint32_t pn = k * p + p0, qn = k * q + q0;
    p0 = p;
    q0 = q;
    p = pn;
    q = qn;
  }
  const int over = (int)(S * q - p * T);  // below T / 254, so 32 bits tell it
  if (over == 0) return {r, fmaf(-r, to, s) != 0.0f};
  if ((uint32_t)abs(over) > (T >> 15)) return {r, false};
  return {fmaf(r, over > 0 ? 0x1p-20f : -0x1p-20f, r), false};
}

// Words of codes times their ratio.  ties: some lane's are (then rounded up and down, and the even one taken).
template <int N>
__device__ __forceinline__ void turn_words(const uint32_t (&w)[N], uint32_t (&o)[N], float ratio, bool ties) {
  if (__any_sync(0xffffffffu, ties)) {
    const float by = ties ? 0x1p-20f : 0.0f;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const float r = fmaf(ratio, side ? by : -by, ratio);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t x = kv8_scale(w[n], r);
        const uint32_t odd = (x & 0x01010101u) * 255u;
        o[n] = side ? (o[n] & odd) | (x & ~odd) : x;
      }
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) o[n] = kv8_scale(w[n], ratio);
}

template <int D>
__global__ void __launch_bounds__(kEvThreads, 2) kv8_evict_kernel(const __grid_constant__ Kv8EvictArgs a) {
  using Geo = Kv8Geom<D>;
  extern __shared__ uint32_t keys[];  // of this CTA's tokens
  __shared__ __align__(16) int hist[2][kEvBins];
  __shared__ int sh_scan[kEvWarps];
  __shared__ int sh_found[2];  // (the first CTA's) a bin, the count above it
  __shared__ int sh_gt[kEvWarps], sh_eq[kEvWarps];
  __shared__ int sh_count[2];  // this CTA's tokens above the last key, and equal to it
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / ctas;
  const Head head{a, item / a.c.heads, item % a.c.heads};
  int32_t* kept = a.kept + (int64_t)item * a.budget;
  const int len = min(max(a.b.lens[head.s], 0), kv_capacity(a.c, a.b));
  if (len <= a.budget) {  // stays as it is (the whole cluster leaves here)
    for (int j = rank * kEvThreads + tid; j < a.budget; j += ctas * kEvThreads) kept[j] = j < len ? j : -1;
    return;
  }
  const int lo_tok = (int)((int64_t)len * rank / ctas), n = (int)((int64_t)len * (rank + 1) / ctas) - lo_tok;
  const int last0 = len - a.last;  // from here on tokens always stay
  const bool held = n <= kEvKeys;
  auto read_key = [&](int x) {
    const int64_t pid = head.page(lo_tok + x);
    return pid >= 0 ? mass_key(*head.mass(pid, lo_tok + x)) : 0u;
  };
  if (held) {
    constexpr int kAtOnce = 8;
    for (int x0 = tid; x0 < n; x0 += kAtOnce * kEvThreads) {
      int64_t pid[kAtOnce];
      float m[kAtOnce];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) pid[y] = x0 + y * kEvThreads < n ? head.page(lo_tok + x0 + y * kEvThreads) : -1;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) m[y] = pid[y] >= 0 ? *head.mass(pid[y], lo_tok + x0 + y * kEvThreads) : 0.0f;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
        if (x0 + y * kEvThreads < n) keys[x0 + y * kEvThreads] = pid[y] >= 0 ? mass_key(m[y]) : 0u;
    }
  }
  auto key_of = [&](int x) { return held ? keys[x] : read_key(x); };

  // ---- the key of the last token that is taken by mass: bits from the top
  uint32_t prefix = 0;                     // the bits known so far
  int need = a.budget - a.first - a.last;  // tokens to take among those that agree with them
  const bool any = need > 0;
  int buf = 0;
  for (int level = 0; any && level < 3; ++level, buf ^= 1) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : kEvBins;
    for (int x = tid; x < kEvBins; x += kEvThreads) hist[buf][x] = 0;
    __syncthreads();
    for (int x = max(0, a.first - lo_tok) + tid; x < min(n, last0 - lo_tok); x += kEvThreads) {
      const uint32_t k = key_of(x);
      if (level == 0 || (k >> (shift + (level == 1 ? 11 : 10))) == prefix) atomicAdd(&hist[buf][(k >> shift) & (bins - 1)], 1);
    }
    if (ctas > 1) {  // the others' counts go to the first CTA's
      cluster.sync();
      int* to = cluster.map_shared_rank(&hist[buf][0], 0);
      for (int x = tid; rank && x < bins; x += kEvThreads)
        if (hist[buf][x]) atomicAdd(to + x, hist[buf][x]);
      cluster.sync();
    } else {
      __syncthreads();
    }
    if (rank == 0) {  // some bins a thread, from the top one down; the bin in which the count reaches `need`
      constexpr int kMine = kEvBins / kEvThreads;
      int mine[kMine], sum = 0;
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        mine[y] = hist[buf][kEvBins - 1 - (tid * kMine + y)];
        sum += mine[y];
      }
      int above = cta_scan(sum, sh_scan) - sum;
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        if (above < need && above + mine[y] >= need) {
          sh_found[0] = kEvBins - 1 - (tid * kMine + y);
          sh_found[1] = above;
        }
        above += mine[y];
      }
    }
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    const int* found = cluster.map_shared_rank(&sh_found[0], 0);
    const int bin = found[0], above = found[1];
    prefix = level == 0 ? (uint32_t)bin : prefix << (level == 1 ? 11 : 10) | (uint32_t)bin;
    need -= above;
  }
  __syncthreads();  // (the keys, where there were no histograms)
  // tokens above `prefix` are taken, and `need` of those equal to it, the lowest positions first; every
  // warp looks through a run of the CTA's tokens, 32 at a time
  const int run = (n + kEvThreads - 1) / kEvThreads * 32, w0 = min(warp * run, n), w1 = min(w0 + run, n);
  auto looks = [&](int x, bool& equal) {
    const int j = lo_tok + x;
    const bool in = x < w1, always = in && (j < a.first || j >= last0);
    const uint32_t k = in && any ? key_of(x) : 0u;
    equal = in && any && !always && k == prefix;
    return always || (in && any && k > prefix);
  };
  int gt = 0, eq = 0;
  for (int x = w0; x < w1; x += 32) {
    bool equal;
    gt += __popc(__ballot_sync(0xffffffffu, looks(x + lane, equal)));
    eq += __popc(__ballot_sync(0xffffffffu, equal));
  }
  if (lane == 0) {
    sh_gt[warp] = gt;
    sh_eq[warp] = eq;
  }
  __syncthreads();
  int gt_before = 0, eq_before = 0, gt_all = 0, eq_all = 0;
#pragma unroll
  for (int y = 0; y < kEvWarps; ++y) {
    if (y == warp) {
      gt_before = gt_all;
      eq_before = eq_all;
    }
    gt_all += sh_gt[y];
    eq_all += sh_eq[y];
  }
  if (tid == 0) {
    sh_count[0] = gt_all;
    sh_count[1] = eq_all;
  }
  cluster.sync();
  for (int z = 0; z < rank; ++z) {
    gt_before += *cluster.map_shared_rank(&sh_count[0], z);
    eq_before += *cluster.map_shared_rank(&sh_count[1], z);
  }
  {
    int at = gt_before + min(eq_before, need);
    const uint32_t below = (1u << lane) - 1u;
    for (int x = w0; x < w1; x += 32) {
      bool equal;
      const bool above = looks(x + lane, equal);
      const uint32_t eqs = __ballot_sync(0xffffffffu, equal);
      const bool take = above || (equal && eq_before + __popc(eqs & below) < need);
      const uint32_t takes = __ballot_sync(0xffffffffu, take);
      const int to = at + __popc(takes & below);
      if (take && to < a.budget) kept[to] = lo_tok + x + lane;  // (as many as that, unless mass is written to meanwhile)
      at += __popc(takes);
      eq_before += __popc(eqs);
    }
  }
  __threadfence();
  cluster.sync();

  // ---- moving
  const int blocks = (a.budget + 15) / 16, step = ctas * kEvWarps;
  constexpr int kLoads = D / 32;  // of 16 bytes a lane, keys and values each
  constexpr uint32_t kZero = 0x80808080u;
  // this warp's block of a round: the token that moves to place lane & 15, its page.  Positions are asked for three
  // rounds ahead, pages two, words one.
  int src, pid, next_src, next_pid, later;
  bool moves, next_moves;
  auto position = [&](int blk) {
    const int dst = blk * 16 + (lane & 15);
    return dst < a.budget ? __ldcg(kept + dst) : -1;
  };
  auto find = [&](int blk, int j) {  // j: the position as it was asked for (where mass was written to meanwhile: anything)
    const int dst = blk * 16 + (lane & 15);
    next_src = j >= dst && j < len ? j : -1;
    next_moves = __any_sync(0xffffffffu, next_src != dst) && blk < blocks;  // else it is what it is
    next_pid = next_src >= 0 ? (int)head.page(next_src) : -1;
  };
  auto advance = [&]() {
    src = next_src;
    pid = next_pid;
    moves = next_moves;
  };
  uint4 kw[kLoads], vw[kLoads][2], par;  // its words as they lie there, and the token's params
  float m;
  auto load = [&]() {
    par = make_uint4(0, 0, 0, 0);
    m = 0.0f;
    if (!moves) return;
    if (pid >= 0) {
      par = *reinterpret_cast<const uint4*>(head.block(pid, src, Geo::kBytes) + Geo::kParams);
      m = *head.mass(pid, src);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {  // keys: 16 channels of token t
      const int x = i * 32 + lane, t = x / (D / 16);
      const int p = __shfl_sync(0xffffffffu, pid, t), j = __shfl_sync(0xffffffffu, src, t);
      kw[i] = make_uint4(kZero, kZero, kZero, kZero);
      if (p >= 0)
        kw[i] = *reinterpret_cast<const uint4*>(head.block(p, j, Geo::kBytes) + (j & 15) * D + Geo::k_piece(j & 15, x % (D / 16)) * 16);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)  // values: 8 channels of the pairs that hold tokens 2 x and 2 x + 1
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int x = i * 32 + lane, t = x / (D / 8) * 2 + y;
        const int p = __shfl_sync(0xffffffffu, pid, t), j = __shfl_sync(0xffffffffu, src, t), from = (j & 15) >> 1;
        vw[i][y] = make_uint4(kZero, kZero, kZero, kZero);
        if (p >= 0)
          vw[i][y] = *reinterpret_cast<const uint4*>(head.block(p, j, Geo::kBytes) + Geo::kVOff + from * 2 * D +
                                                     Geo::v_piece(from, x % (D / 8)) * 16);
      }
  };
  const int mine = rank * kEvWarps + warp;
  later = position(mine);
  find(mine, later);
  later = position(mine + step);
  advance();
  load();
  find(mine + step, later);
  later = position(mine + 2 * step);
  for (int b0 = 0; b0 < blocks; b0 += step) {
    const int blk = b0 + mine;
    const bool moving = moves;
    const int64_t to_pid = moving ? head.page(blk * 16) : -1;
    uint4 ko[kLoads], vo[kLoads];
    float k_to = 0.0f, v_to = 0.0f;
    uint32_t marks = 0;
    int have = -1;
    float mass = 0.0f;
    if (moving) {
      const float ks = __uint_as_float(par.x), vs = __uint_as_float(par.y);
      have = src;
      mass = m;
      marks = ((par.z >> (src & 15)) & 1u) | ((par.z >> (16 + (src & 15))) & 1u) << 16;
      k_to = ks;
      v_to = vs;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        k_to = fmaxf(k_to, __shfl_xor_sync(0xffffffffu, k_to, o));
        v_to = fmaxf(v_to, __shfl_xor_sync(0xffffffffu, v_to, o));
      }
      // what the tokens' codes are multiplied with: the keys' in lanes 0 to 15, the values' in 16 to 31
      const Ratio ratio = ratio_of(lane < 16 ? ks : vs, lane < 16 ? k_to : v_to);
      if (__all_sync(0xffffffffu, ratio.r == 1.0f)) {  // nothing to turn: of one step, all of them
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ko[i] = kw[i];
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int t = (i * 32 + lane) / (D / 16);
          const uint32_t w[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
          uint32_t o[4];
          turn_words(w, o, __shfl_sync(0xffffffffu, ratio.r, t), __shfl_sync(0xffffffffu, (int)ratio.ties, t));
          ko[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint32_t o[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = (i * 32 + lane) / (D / 8) * 2 + y;
          const uint32_t sel = __shfl_sync(0xffffffffu, src, t) & 1 ? 0x7531 : 0x6420;  // the token's byte of every pair
          const uint32_t w[2] = {__byte_perm(vw[i][y].x, vw[i][y].y, sel), __byte_perm(vw[i][y].z, vw[i][y].w, sel)};
          turn_words(w, o[y], __shfl_sync(0xffffffffu, ratio.r, 16 + t), __shfl_sync(0xffffffffu, (int)ratio.ties, 16 + t));
        }
        vo[i] = make_uint4(__byte_perm(o[0][0], o[1][0], 0x5140), __byte_perm(o[0][0], o[1][0], 0x7362),
                           __byte_perm(o[0][1], o[1][1], 0x5140), __byte_perm(o[0][1], o[1][1], 0x7362));
      }
    }
    auto token = cluster.barrier_arrive();  // this warp has read its part of the round
    advance();
    load();
    find(blk + 2 * step, later);
    later = position(blk + 3 * step);
    cluster.barrier_wait(std::move(token));
    if (to_pid >= 0) {
      uint8_t* to = head.block(to_pid, blk * 16, Geo::kBytes);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int x = i * 32 + lane, t = x / (D / 16), pair = x / (D / 8);
        *reinterpret_cast<uint4*>(to + t * D + Geo::k_piece(t, x % (D / 16)) * 16) = ko[i];
        *reinterpret_cast<uint4*>(to + Geo::kVOff + pair * 2 * D + Geo::v_piece(pair, x % (D / 8)) * 16) = vo[i];
      }
      const uint32_t bits_k = __ballot_sync(0xffffffffu, lane < 16 && (marks & 1u));
      const uint32_t bits_v = __ballot_sync(0xffffffffu, lane < 16 && (marks >> 16));
      if (lane == 0)
        *reinterpret_cast<uint4*>(to + Geo::kParams) =
            make_uint4(__float_as_uint(k_to), __float_as_uint(v_to), bits_k | bits_v << 16, 0);
      if (lane < 16 && have >= 0) *head.mass(to_pid, blk * 16 + lane) = mass;
    }
  }
}

template <int D>
cudaError_t evict(const Kv8EvictArgs& a, int ctas, cudaStream_t s) {
  const auto kernel = kv8_evict_kernel<D>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kEvKeys * sizeof(uint32_t));
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a.b.batch * a.c.heads * ctas));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = kEvKeys * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t moe::kv8_evict(const Kv8& kv, const Kv8EvictArgs& a, cudaStream_t s) {
  const int64_t items = (int64_t)a.b.batch * a.c.heads, cap = (int64_t)a.b.table_pages << a.c.page_shift;
  int ctas = kEvMaxCluster;
  // as many as two a multiprocessor hold at once, and as have some tokens each.  Measured, one sequence of 131,072
  // tokens, 8 heads: 16 CTAs of 256 threads 232 us, 16 of 512 (of which half the clusters wait for the others) 254, 8 of
  // 512 236, 8 of 256 371.
  while (ctas > 1 && (items * ctas > 2 * kv.sms || ctas * 1024 > cap)) ctas >>= 1;
  if (items * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return kv.d.head_dim == 64 ? evict<64>(a, ctas, s) : evict<128>(a, ctas, s);
}
