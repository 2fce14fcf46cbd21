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
#include <cooperative_groups.h>

#include "kv8_internal.h"

using namespace moe;
namespace cg = cooperative_groups;

namespace {

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
template <int kEvWarps>
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

// Words of a token's codes, of a step s that is `ratio` (rounded) times the new one, `to`; the token's other words are
// in the lanes of `group`, with the same numbers.
//
// Of one token, the quotients u s / to that are near a half are all near ties of one fraction: s / to is then within
// 2e-5 / u of a p / q with q <= 254, and two such fractions are further apart.  So they lie on the same side of their
// half (mirrored for negative u), and one of them, settled exactly, says on which: a ratio moved by 2^-20 that way rounds
// all of them rightly, and every other code, which is at least 1 / (2 q) away from a half, as before.  Where s / to is
// that fraction itself the ties are even ones: right already if ratio is exact, else settled one by one.
template <int N>
__device__ __forceinline__ void turn_words(const uint32_t (&w)[N], uint32_t (&o)[N], float s, float to, float ratio, uint32_t group) {
  if (__all_sync(0xffffffffu, s == to)) {
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = w[n];
    return;
  }
  uint32_t near = 0;  // a bit per byte, the first one's the highest
#pragma unroll
  for (int n = 0; n < N; ++n) o[n] = kv8_turn(w[n], ratio, near);
  const uint32_t votes = __ballot_sync(0xffffffffu, near != 0);
  if (votes == 0) return;
  float side = 0.0f;
  if (near) {
    const int at = 4 * N - 1 - (31 - __clz(near));
    uint32_t x = w[0];
#pragma unroll
    for (int n = 1; n < N; ++n) x = at / 4 == n ? w[n] : x;
    const float u = (float)((int)((x >> (8 * (at & 3))) & 0xffu) - 128), half = floorf(u * ratio) + 0.5f;
    const float p = u * s, q = half * to, over = (p - q) + (fmaf(u, s, -p) - fmaf(half, to, -q));
    side = over == 0.0f ? 0.0f : (over > 0.0f) == (u > 0.0f) ? 0x1p-20f : -0x1p-20f;
  }
  const uint32_t mine = votes & group;
  side = __shfl_sync(0xffffffffu, side, mine ? __ffs(mine) - 1 : 0);
  if (mine && side != 0.0f) {
    const float moved = fmaf(ratio, side, ratio);
    uint32_t unused = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = kv8_turn(w[n], moved, unused);
  } else if (near && fmaf(-ratio, to, s) != 0.0f) {
#pragma unroll 1
    for (; near; near &= near - 1) {
      const int at = 4 * N - __ffs(near), shift = 8 * (at & 3);
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (at / 4 == n) o[n] = (o[n] & ~(0xffu << shift)) | kv8_settle_byte(w[n], at & 3, s, to, ratio) << shift;
    }
  }
}

template <int D, int kEvThreads>
__global__ void __launch_bounds__(kEvThreads, 512 / kEvThreads) kv8_evict_kernel(const __grid_constant__ Kv8EvictArgs a) {
  using Geo = Kv8Geom<D>;
  constexpr int kEvWarps = kEvThreads / 32;
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
      int above = cta_scan<kEvWarps>(sum, sh_scan) - sum;
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
      // what every token's codes are multiplied with
      const float up_k = kv8_lift(k_to), up_v = kv8_lift(v_to), kt = k_to * up_k, vt = v_to * up_v;
      const float kr = kt > 0.0f ? __fdiv_rn(ks * up_k, kt) : 0.0f, vr = vt > 0.0f ? __fdiv_rn(vs * up_v, vt) : 0.0f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int t = (i * 32 + lane) / (D / 16);
        const uint32_t w[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
        uint32_t o[4];
        turn_words(w, o, __shfl_sync(0xffffffffu, ks * up_k, t), kt, __shfl_sync(0xffffffffu, kr, t),
                   ((1u << (D / 16)) - 1u) << (lane & ~(D / 16 - 1)));
        ko[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint32_t o[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = (i * 32 + lane) / (D / 8) * 2 + y;
          const uint32_t sel = __shfl_sync(0xffffffffu, src, t) & 1 ? 0x7531 : 0x6420;  // the token's byte of every pair
          const uint32_t w[2] = {__byte_perm(vw[i][y].x, vw[i][y].y, sel), __byte_perm(vw[i][y].z, vw[i][y].w, sel)};
          turn_words(w, o[y], __shfl_sync(0xffffffffu, vs * up_v, t), vt, __shfl_sync(0xffffffffu, vr, t),
                     ((1u << (D / 8)) - 1u) << (lane & ~(D / 8 - 1)));
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

template <int D, int Threads>
cudaError_t evict(const Kv8EvictArgs& a, int ctas, cudaStream_t s) {
  const auto kernel = kv8_evict_kernel<D, Threads>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kEvKeys * sizeof(uint32_t));
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a.b.batch * a.c.heads * ctas));
  cfg.blockDim = dim3(Threads);
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
  // as many as two a multiprocessor hold at once, and as have some tokens each
  while (ctas > 1 && (items * ctas > 2 * kv.sms || ctas * 1024 > cap)) ctas >>= 1;
  if (items * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const bool wide = items * ctas <= kv.sms;  // a multiprocessor each: twice the warps
  if (kv.d.head_dim == 64) return wide ? evict<64, 512>(a, ctas, s) : evict<64, 256>(a, ctas, s);
  return wide ? evict<128, 512>(a, ctas, s) : evict<128, 256>(a, ctas, s);
}
