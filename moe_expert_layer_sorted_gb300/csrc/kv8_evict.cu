// Eviction from the 8-bit cache by accumulated weight: of every sequence and kv head the first and
// the last tokens and those of the largest mass stay, and move together.
//
// Choice: one cluster per (sequence, kv head), its CTAs sharing the tokens.  Order-preserving 32-bit keys of the masses,
//   kept in shared memory where they fit; the key of the last token that is taken by three histograms of 11, 11 and 10
//   bits, added up over the cluster through distributed shared memory; then one ordered pass counts, and one writes the
//   kept positions.
// Moving: one cluster for the keys and one for the values of a (sequence, kv head), which share no byte that either
//   writes.  Sixteen kept tokens make a new block, whose step is the largest of theirs.  A token moves to a lower
//   position or stays, so blocks are made in rounds, one per warp of the cluster: all of a round have been read before
//   any is written, and no later round reads what this one overwrites.  What later rounds need may then be read as early
//   as one likes: asynchronous copies bring it to shared memory a round ahead, and the barrier of a round runs while
//   its codes are turned.
//
// Measured (8 heads of 128 channels, caches whose tokens have not been moved before): 32 sequences of up to 4,608 tokens
// to 4,096 each 106 us (choice 21), 0.5 GB read and written; one of 131,072 to 65,536 161 us (choice 33).  Keys and values
// by the same warps: 207 and 232; rings of three rounds and two CTAs an SM: 117 and 167.  Bound by the chain of a block (ratios,
// 10 us and 20, and turning, 10 and 17) at 24 warps an SM, and for one sequence by the SMs that sixteen clusters leave idle.
#include <cooperative_groups.h>

#include "kv8_internal.h"

using namespace moe;
namespace cg = cooperative_groups;

namespace {

constexpr int kChThreads = 512, kChWarps = kChThreads / 32;  // that choose
constexpr int kMvThreads = 256, kMvWarps = kMvThreads / 32;  // that move
constexpr int kEvBins = 2048;
constexpr int kEvKeys = 16384;  // that a CTA keeps in shared memory; of longer shares they are read again
constexpr int kEvMaxCluster = 16;
constexpr int kMvStages = 2;  // rounds in a ring
constexpr int kMvPerSm = 3;  // CTAs that move tokens

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
  for (int w = 0; w < kChWarps; ++w)
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
  if (s * 256.0f < to) return {0.0f, false};  // below a half with every code
  const float r = __fdiv_rn(s, to);
  // Euclid's steps on to and s: whole multiples of s's last place of up to 24 bits, so every remainder is exact.  The
  // remainder is also how far s q is from to p, on the one side and the other in turn.
  float a = to, b = s, q0 = 0.0f, q = 1.0f, side = 0x1p-20f;
  while (b != 0.0f) {
    float k = (__fdividef(a, b) - 0.5f + 12582912.0f) - 12582912.0f, left = fmaf(-k, b, a);
    if (left < 0.0f) left = fmaf(-(k -= 1.0f), b, a);
    if (left >= b) left = fmaf(-(k += 1.0f), b, a);
    const float qn = fmaf(k, q, q0);
    if (qn > 254.0f) break;
    a = b;
    b = left;
    q0 = q;
    q = qn;
    side = -side;
  }
  if (b == 0.0f) return {r, fmaf(-r, to, s) != 0.0f};
  if (b > to * 0x1p-15f) return {r, false};
  return {fmaf(r, side, r), false};
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

__global__ void __launch_bounds__(kChThreads, 2) kv8_choose_kernel(const __grid_constant__ Kv8EvictArgs a) {
  extern __shared__ uint32_t keys[];  // of this CTA's tokens
  __shared__ __align__(16) int hist[2][kEvBins];
  __shared__ int sh_scan[kChWarps];
  __shared__ int sh_found[2];  // (the first CTA's) a bin, the count above it
  __shared__ int sh_gt[kChWarps], sh_eq[kChWarps];
  __shared__ int sh_count[2];  // this CTA's tokens above the last key, and equal to it
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / ctas;
  const Head head{a, item / a.c.heads, item % a.c.heads};
  int32_t* kept = a.kept + (int64_t)item * a.budget;
  const int len = min(max(a.b.lens[head.s], 0), kv_capacity(a.c, a.b));
  if (len <= a.budget) {  // stays as it is (the whole cluster leaves here)
    for (int j = rank * kChThreads + tid; j < a.budget; j += ctas * kChThreads) kept[j] = j < len ? j : -1;
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
    for (int x0 = tid; x0 < n; x0 += kAtOnce * kChThreads) {
      int64_t pid[kAtOnce];
      float m[kAtOnce];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) pid[y] = x0 + y * kChThreads < n ? head.page(lo_tok + x0 + y * kChThreads) : -1;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y) m[y] = pid[y] >= 0 ? *head.mass(pid[y], lo_tok + x0 + y * kChThreads) : 0.0f;
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
        if (x0 + y * kChThreads < n) keys[x0 + y * kChThreads] = pid[y] >= 0 ? mass_key(m[y]) : 0u;
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
    for (int x = tid; x < kEvBins; x += kChThreads) hist[buf][x] = 0;
    __syncthreads();
    for (int x = max(0, a.first - lo_tok) + tid; x < min(n, last0 - lo_tok); x += kChThreads) {
      const uint32_t k = key_of(x);
      if (level == 0 || (k >> (shift + (level == 1 ? 11 : 10))) == prefix) atomicAdd(&hist[buf][(k >> shift) & (bins - 1)], 1);
    }
    if (ctas > 1) {  // the others' counts go to the first CTA's
      cluster.sync();
      int* to = cluster.map_shared_rank(&hist[buf][0], 0);
      for (int x = tid; rank && x < bins; x += kChThreads)
        if (hist[buf][x]) atomicAdd(to + x, hist[buf][x]);
      cluster.sync();
    } else {
      __syncthreads();
    }
    if (rank == 0) {  // some bins a thread, from the top one down; the bin in which the count reaches `need`
      constexpr int kMine = kEvBins / kChThreads;
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
  const int run = (n + kChThreads - 1) / kChThreads * 32, w0 = min(warp * run, n), w1 = min(w0 + run, n);
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
  for (int y = 0; y < kChWarps; ++y) {
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
  cluster.sync();  // no CTA ends while another reads its counts
}

__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
// Bytes of a round in a warp's ring: positions, steps, marks and masses of sixteen tokens, and their values' words.
template <int D>
constexpr int kMvStage = 256 + 32 * D;

// The keys' or the values' codes and steps of a sequence's head, and with the keys the masses.
template <int D, bool kValues>
__device__ __forceinline__ void move_tokens(const Kv8EvictArgs& a, cg::cluster_group& cluster, int item) {
  using Geo = Kv8Geom<D>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const Head head{a, item / a.c.heads, item % a.c.heads};
  const int32_t* kept = a.kept + (int64_t)item * a.budget;
  const int len = min(max(a.b.lens[head.s], 0), kv_capacity(a.c, a.b));
  if (len <= a.budget) return;  // (the whole cluster)
  const int blocks = (a.budget + 15) / 16, step = ctas * kMvWarps;
  constexpr int kLoads = kValues ? D / 16 : D / 32;  // of 16 bytes a lane
  constexpr uint32_t kZero = 0x80808080u;
  constexpr int kStep = Geo::kParams + (kValues ? 4 : 0), kMark = Geo::kParams + (kValues ? 10 : 8);
  // Sources are copied into a ring of the warp's: words as they lie there, every lane's own, and of the sixteen tokens
  // the position, step, marks and mass.  Positions are asked for two rounds before that, pages one.
  extern __shared__ __align__(16) uint8_t ring_raw[];
  constexpr int kStage = kMvStage<D>;
  uint8_t* ring = ring_raw + warp * kMvStages * kStage;
  int next_src, next_pid, later, next_blk = rank * kMvWarps + warp;
  auto position = [&](int blk) {
    const int dst = blk * 16 + (lane & 15);
    return dst < a.budget ? __ldg(kept + dst) : -1;
  };
  auto find = [&]() {  // the token that moves to place lane & 15 of next_blk, its page
    const int dst = next_blk * 16 + (lane & 15);
    next_src = later >= dst && later < len ? later : -1;  // (where mass was written to meanwhile, `later` is anything)
    next_pid = next_src >= 0 ? (int)head.page(next_src) : -1;
  };
  auto moving = [&](int blk, int src) {  // else it is what it is
    return __any_sync(0xffffffffu, src != blk * 16 + (lane & 15)) && blk < blocks;
  };
  // Keys: 16 channels of a token; values: 8 channels of the pairs that hold tokens 2 x and 2 x + 1, one after the other
  auto fetch = [&](int stage) {
    uint8_t* to = ring + stage * kStage;
    if (lane < 16) reinterpret_cast<int*>(to)[lane] = next_src;
    if (moving(next_blk, next_src)) {
      // where the token's block lies, a multiple of 16, and the token's place in it
      const int64_t block = next_pid >= 0 ? head.block(next_pid, next_src, Geo::kBytes) - a.c.pages : -16;
      const uint32_t lo = (uint32_t)block | (next_src & 15), hi = (uint32_t)(block >> 32);
      if (lane < 16) {
        uint32_t* par = reinterpret_cast<uint32_t*>(to) + 16 + lane;
        if (next_pid >= 0) {
          const uint8_t* from = a.c.pages + block + Geo::kParams;
          copy4(par, from + (kValues ? 4 : 0));
          copy4(par + 16, from + 8);
          if constexpr (!kValues) copy4(par + 32, head.mass(next_pid, next_src));
        } else {
          par[0] = par[16] = par[32] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int x = (kValues ? i / 2 : i) * 32 + lane, piece = x % (kValues ? D / 8 : D / 16);
        const int t = kValues ? x / (D / 8) * 2 + i % 2 : x / (D / 16);
        const uint32_t l = __shfl_sync(0xffffffffu, lo, t), h = __shfl_sync(0xffffffffu, hi, t);
        uint4* dst = reinterpret_cast<uint4*>(to + 256) + i * 32 + lane;
        if ((int)h >= 0) {
          const int row = kValues ? (l & 15u) >> 1 : l & 15u;
          const int at = kValues ? Geo::kVOff + row * 2 * D + Geo::v_piece(row, piece) * 16 : row * D + Geo::k_piece(row, piece) * 16;
          copy16(dst, a.c.pages + ((int64_t)h << 32 | (l & ~15u)) + at);
        } else {
          *dst = make_uint4(kZero, kZero, kZero, kZero);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next_blk += step;
    find();
    later = position(next_blk + step);
  };
  later = position(next_blk);
  find();
  later = position(next_blk + step);
#pragma unroll 1
  for (int y = 0; y < kMvStages - 1; ++y) fetch(y);
  int stage = 0;
  for (int b0 = 0; b0 < blocks; b0 += step) {
    const int blk = b0 + rank * kMvWarps + warp;
    asm volatile("cp.async.wait_group %0;" ::"n"(kMvStages - 2) : "memory");
    __syncwarp();
    // This warp has its part of the round: nothing is handed over but that, so the barrier does not wait for its writes.
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    fetch(stage == 0 ? kMvStages - 1 : stage - 1);  // (the one before this)
    const uint8_t* from = ring + stage * kStage;
    const int src = reinterpret_cast<const int*>(from)[lane & 15];
    const int64_t to_pid = moving(blk, src) ? head.page(blk * 16) : -1;
    uint4 out[D / 32];
    float s_new = 0.0f;
    bool marked = false;
    if (to_pid >= 0) {
      const uint32_t* par = reinterpret_cast<const uint32_t*>(from) + 16 + (lane & 15);
      const uint4* words = reinterpret_cast<const uint4*>(from + 256) + lane;
      const float s_old = __uint_as_float(par[0]);
      marked = (par[16] >> ((kValues ? 16 : 0) + (src & 15))) & 1u;
      s_new = s_old;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) s_new = fmaxf(s_new, __shfl_xor_sync(0xffffffffu, s_new, o));
      const Ratio ratio = ratio_of(s_old, s_new);  // what the codes of token lane & 15 are multiplied with
      if constexpr (!kValues) {
        if (__all_sync(0xffffffffu, ratio.r == 1.0f)) {  // nothing to turn: of one step, all of them
#pragma unroll
          for (int i = 0; i < kLoads; ++i) out[i] = words[32 * i];
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int t = (i * 32 + lane) / (D / 16);
            const uint4 v = words[32 * i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
            turn_words(w, o, __shfl_sync(0xffffffffu, ratio.r, t), __shfl_sync(0xffffffffu, (int)ratio.ties, t));
            out[i] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[2][2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 v = words[32 * (2 * i + y)];
            const int t = (i * 32 + lane) / (D / 8) * 2 + y;
            const uint32_t sel = __shfl_sync(0xffffffffu, src, t) & 1 ? 0x7531 : 0x6420;  // the token's byte of every pair
            const uint32_t w[2] = {__byte_perm(v.x, v.y, sel), __byte_perm(v.z, v.w, sel)};
            turn_words(w, o[y], __shfl_sync(0xffffffffu, ratio.r, t), __shfl_sync(0xffffffffu, (int)ratio.ties, t));
          }
          out[i] = make_uint4(__byte_perm(o[0][0], o[1][0], 0x5140), __byte_perm(o[0][0], o[1][0], 0x7362),
                              __byte_perm(o[0][1], o[1][1], 0x5140), __byte_perm(o[0][1], o[1][1], 0x7362));
        }
      }
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (to_pid >= 0) {
      uint8_t* to = head.block(to_pid, blk * 16, Geo::kBytes);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int x = i * 32 + lane, row = x / (kValues ? D / 8 : D / 16), piece = x % (kValues ? D / 8 : D / 16);
        const int at = kValues ? Geo::kVOff + row * 2 * D + Geo::v_piece(row, piece) * 16 : row * D + Geo::k_piece(row, piece) * 16;
        *reinterpret_cast<uint4*>(to + at) = out[i];
      }
      const uint32_t marks = __ballot_sync(0xffffffffu, lane < 16 && marked);
      if (lane == 0) {
        *reinterpret_cast<float*>(to + kStep) = s_new;
        *reinterpret_cast<uint16_t*>(to + kMark) = (uint16_t)marks;
        if constexpr (!kValues) *reinterpret_cast<uint32_t*>(to + Geo::kParams + 12) = 0;
      }
      if constexpr (!kValues)
        if (lane < 16 && src >= 0) *head.mass(to_pid, blk * 16 + lane) = reinterpret_cast<const float*>(from)[48 + lane];
    }
    stage = stage + 1 == kMvStages ? 0 : stage + 1;
  }
}

// Clusters of the values first (they have more to do), then those of the keys: the two share no byte that either writes.
template <int D>
__global__ void __launch_bounds__(kMvThreads, kMvPerSm) kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int item = blockIdx.x / cluster.num_blocks(), items = a.b.batch * a.c.heads;
  if (item < items) move_tokens<D, true>(a, cluster, item);
  else move_tokens<D, false>(a, cluster, item - items);
}

using Kernel = void (*)(Kv8EvictArgs);

// Calls f with the launch of `clusters` clusters.
template <typename F>
cudaError_t with_launch(Kernel kernel, int64_t clusters, int ctas, int threads, size_t smem, cudaStream_t s, F f) {
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(clusters * ctas));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return f(cfg);
}

}  // namespace

cudaError_t moe::kv8_evict(const Kv8& kv, const Kv8EvictArgs& a, cudaStream_t s) {
  const int64_t items = (int64_t)a.b.batch * a.c.heads, cap = (int64_t)a.b.table_pages << a.c.page_shift;
  // to choose: as many CTAs as two a multiprocessor hold at once, and as have some tokens each
  int choose = kEvMaxCluster;
  while (choose > 1 && (items * choose > 2 * kv.sms || choose * 1024 > cap)) choose >>= 1;
  // to move: as many as have a block for each warp, and as let all clusters run at once (the parts of the chip that a
  // cluster has to lie in are not of one size, so the driver is asked, once a cache); where clusters outnumber what
  // runs at once, enough for some waves, since those of the values take longer.  Measured: 32 sequences of up to 4,608
  // tokens, 8 heads, 512 clusters of one CTA 160 us, of two 117, of four 110; one of 131,072, 16 clusters of 16 CTAs, of
  // which some wait for others, 187, of as many as all run 178.
  const Kernel mover = kv.d.head_dim == 64 ? kv8_move_kernel<64> : kv8_move_kernel<128>;
  const size_t ring = kMvWarps * kMvStages * (kv.d.head_dim == 64 ? kMvStage<64> : kMvStage<128>);
  const bool waves = 2 * items > kMvPerSm * kv.sms;
  int move = kEvMaxCluster;
  for (; move > 1; --move) {
    if (2 * items * move > (waves ? 14 : kMvPerSm) * kv.sms || move * kMvWarps * 16 > a.budget) continue;
    if (waves) break;
    int& fit = kv.move_clusters[move];
    if (fit < 0) {
      const cudaError_t e = with_launch(mover, 1, move, kMvThreads, ring, s, [&](const cudaLaunchConfig_t& cfg) {
        return cudaOccupancyMaxActiveClusters(&fit, mover, &cfg);
      });
      if (e != cudaSuccess) return e;
    }
    if (fit >= 2 * items) break;
  }
  if (items * choose > 0x7fffffff || 2 * items * move > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const cudaError_t e = with_launch(kv8_choose_kernel, items, choose, kChThreads, kEvKeys * sizeof(uint32_t), s,
                                    [&](const cudaLaunchConfig_t& cfg) { return cudaLaunchKernelEx(&cfg, kv8_choose_kernel, a); });
  if (e != cudaSuccess) return e;
  return with_launch(mover, 2 * items, move, kMvThreads, ring, s,
                     [&](const cudaLaunchConfig_t& cfg) { return cudaLaunchKernelEx(&cfg, mover, a); });
}
