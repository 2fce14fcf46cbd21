// Eviction from the 8-bit cache by accumulated weight: of every sequence and kv head the first and
// the last tokens and those of the largest mass stay, and move together.
//
// One cluster per (sequence, kv head), its CTAs sharing the tokens.
//   Choice: order-preserving 32-bit keys of the masses; the key of the last token that is taken by
//   three histograms of 11, 11 and 10 bits, added up over the cluster through distributed shared
//   memory; then one ordered pass counts, and one writes the kept positions.
//   Moving: sixteen kept tokens make a new block, whose step is the largest of theirs.  A token moves
//   to a lower position or stays, so blocks are made in rounds, one per warp of the cluster: all of a
//   round are in registers before any is written, and no later round reads what this one overwrites.
#include <cooperative_groups.h>

#include "kv8_internal.h"

using namespace moe;
namespace cg = cooperative_groups;

namespace {

constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 8;

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

// Codes of a word (u + 128 in each byte) of a step that is `ratio` = s / to times the new one, turned.
__device__ __forceinline__ uint32_t turn_word(uint32_t word, float ratio, float s, float to) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u = kv8_code(word, i), y = u * ratio, lo = floorf(y);
    float z = rintf(y);
    if (fabsf(y - lo - 0.5f) < 1e-3f) {  // near a half: by what is left above it, exact in fp64
      const double over = (double)u * (double)s - ((double)lo + 0.5) * (double)to;
      z = over > 0.0 ? lo + 1.0f : over < 0.0 ? lo : 2.0f * rintf(0.5f * (lo + 0.5f));
    }
    out |= (__float_as_uint(z + 12583040.0f) & 0xffu) << (8 * i);
  }
  return out;
}

template <int D>
__global__ void __launch_bounds__(kEvThreads) kv8_evict_kernel(const __grid_constant__ Kv8EvictArgs a) {
  using Geo = Kv8Geom<D>;
  __shared__ int hist[2][kEvBins];
  __shared__ int sh_scan[kEvWarps];
  __shared__ int sh_bin, sh_above;
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
  const int lo_tok = (int)((int64_t)len * rank / ctas), hi_tok = (int)((int64_t)len * (rank + 1) / ctas);
  const int last0 = len - a.last;  // from here on tokens always stay
  auto key_of = [&](int j) {
    const int64_t pid = head.page(j);
    return pid >= 0 ? mass_key(*head.mass(pid, j)) : 0u;
  };

  // ---- the key of the last token that is taken by mass: bits from the top
  uint32_t prefix = 0;                    // the bits known so far
  int need = a.budget - a.first - a.last;  // tokens to take among those that agree with them
  const bool any = need > 0;
  int buf = 0;
  for (int level = 0; any && level < 3; ++level, buf ^= 1) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : kEvBins;
    for (int x = tid; x < kEvBins; x += kEvThreads) hist[buf][x] = 0;
    __syncthreads();
    for (int j = max(lo_tok, a.first) + tid; j < min(hi_tok, last0); j += kEvThreads) {
      const uint32_t k = key_of(j);
      if (level == 0 || (k >> (shift + (level == 1 ? 11 : 10))) == prefix) atomicAdd(&hist[buf][(k >> shift) & (bins - 1)], 1);
    }
    cluster.sync();
    // totals of four bins a thread, from the top one down; the bin in which the count reaches `need`
    int mine[kEvBins / kEvThreads], sum = 0;
#pragma unroll
    for (int y = 0; y < kEvBins / kEvThreads; ++y) {
      const int bin = kEvBins - 1 - (tid * (kEvBins / kEvThreads) + y);
      mine[y] = 0;
      for (int z = 0; z < ctas; ++z) mine[y] += *cluster.map_shared_rank(&hist[buf][bin], z);
      sum += mine[y];
    }
    int above = cta_scan(sum, sh_scan) - sum;
#pragma unroll
    for (int y = 0; y < kEvBins / kEvThreads; ++y) {
      if (above < need && above + mine[y] >= need) {
        sh_bin = kEvBins - 1 - (tid * (kEvBins / kEvThreads) + y);
        sh_above = above;
      }
      above += mine[y];
    }
    __syncthreads();
    prefix = level == 0 ? (uint32_t)sh_bin : prefix << (level == 1 ? 11 : 10) | (uint32_t)sh_bin;
    need -= sh_above;
  }
  // tokens above `prefix` are taken, and `need` of those equal to it, the lowest positions first
  auto takes = [&](int j, uint32_t k, bool& equal) {
    const bool always = j < a.first || j >= last0;
    equal = any && !always && k == prefix;
    return always || (any && k > prefix);
  };
  // every thread takes a run of the CTA's tokens
  const int run = (hi_tok - lo_tok + kEvThreads - 1) / kEvThreads;
  const int b = min(lo_tok + tid * run, hi_tok), e = min(b + run, hi_tok);
  int gt = 0, eq = 0;
  for (int j = b; j < e; ++j) {
    bool equal;
    gt += takes(j, key_of(j), equal);
    eq += equal;
  }
  const int eq_upto = cta_scan(eq, sh_scan), gt_upto = cta_scan(gt, sh_scan);
  if (tid == kEvThreads - 1) {
    sh_count[0] = gt_upto;
    sh_count[1] = eq_upto;
  }
  cluster.sync();
  int gt_before = 0, eq_before = 0;
  for (int z = 0; z < rank; ++z) {
    gt_before += *cluster.map_shared_rank(&sh_count[0], z);
    eq_before += *cluster.map_shared_rank(&sh_count[1], z);
  }
  {
    int e_rank = eq_before + eq_upto - eq;                           // equal tokens before this run
    int at = gt_before + gt_upto - gt + min(e_rank, need);           // kept ones
    for (int j = b; j < e; ++j) {
      bool equal;
      const bool take = takes(j, key_of(j), equal) || (equal && e_rank < need);
      e_rank += equal;
      if (take && at < a.budget) kept[at++] = j;  // (as many as that, unless mass is written to meanwhile)
    }
  }
  __threadfence();
  cluster.sync();

  // ---- moving
  const int blocks = (a.budget + 15) / 16, step = ctas * kEvWarps;
  constexpr int kLoads = D / 32;  // of 16 bytes a lane, keys and values each
  for (int b0 = 0; b0 < blocks; b0 += step) {
    const int blk = b0 + rank * kEvWarps + warp;
    uint4 kw[kLoads], vw[kLoads];
    float ks = 0.0f, vs = 0.0f, m = 0.0f;  // lane t < 16: of the token that moves to place t
    uint32_t marks = 0;
    int src = -1;
    int64_t pid = -1, to_pid = -1;
    bool moves = false;
    float k_to = 0.0f, v_to = 0.0f;
    if (blk < blocks) {
      const int dst = blk * 16 + (lane & 15);
      src = dst < a.budget ? __ldcg(kept + dst) : -1;
      moves = __any_sync(0xffffffffu, src != dst);  // else it is what it is
      to_pid = head.page(blk * 16);
      if (moves) {
        if (src >= 0) pid = head.page(src);
        if (pid >= 0) {
          const uint8_t* from = head.block(pid, src, Geo::kBytes);
          const uint4 par = *reinterpret_cast<const uint4*>(from + Geo::kParams);
          ks = __uint_as_float(par.x);
          vs = __uint_as_float(par.y);
          marks = ((par.z >> (src & 15)) & 1u) | ((par.z >> (16 + (src & 15))) & 1u) << 16;
          m = *head.mass(pid, src);
        }
        k_to = ks;
        v_to = vs;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          k_to = fmaxf(k_to, __shfl_xor_sync(0xffffffffu, k_to, o));
          v_to = fmaxf(v_to, __shfl_xor_sync(0xffffffffu, v_to, o));
        }
        auto turn4 = [&](uint4 x, float s, float to) {
          const float ratio = to > 0.0f ? __fdiv_rn(s, to) : 0.0f;
          return make_uint4(turn_word(x.x, ratio, s, to), turn_word(x.y, ratio, s, to), turn_word(x.z, ratio, s, to),
                            turn_word(x.w, ratio, s, to));
        };
        const uint4 zero = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {  // keys: 16 channels of token t
          const int x = i * 32 + lane, t = x / (D / 16);
          const int64_t p = __shfl_sync(0xffffffffu, pid, t);
          const int j = __shfl_sync(0xffffffffu, src, t);
          const float s = __shfl_sync(0xffffffffu, ks, t);
          kw[i] = zero;
          if (p >= 0) {
            kw[i] = *reinterpret_cast<const uint4*>(head.block(p, j, Geo::kBytes) + (j & 15) * D + Geo::k_piece(j & 15, x % (D / 16)) * 16);
            if (s != k_to) kw[i] = turn4(kw[i], s, k_to);
          }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {  // values: 8 channels of the tokens 2 x and 2 x + 1
          const int x = i * 32 + lane, pair = x / (D / 8);
          uint2 half[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int t = 2 * pair + y;
            const int64_t p = __shfl_sync(0xffffffffu, pid, t);
            const int j = __shfl_sync(0xffffffffu, src, t);
            const float s = __shfl_sync(0xffffffffu, vs, t);
            half[y] = make_uint2(0x80808080u, 0x80808080u);
            if (p >= 0) {
              const int from = (j & 15) >> 1;
              const uint4 v = *reinterpret_cast<const uint4*>(head.block(p, j, Geo::kBytes) + Geo::kVOff + from * 2 * D +
                                                              Geo::v_piece(from, x % (D / 8)) * 16);
              const uint32_t sel = j & 1 ? 0x7531 : 0x6420;  // the token's byte of every pair
              half[y] = make_uint2(__byte_perm(v.x, v.y, sel), __byte_perm(v.z, v.w, sel));
              if (s != v_to) {
                const float ratio = v_to > 0.0f ? __fdiv_rn(s, v_to) : 0.0f;
                half[y] = make_uint2(turn_word(half[y].x, ratio, s, v_to), turn_word(half[y].y, ratio, s, v_to));
              }
            }
          }
          vw[i] = make_uint4(__byte_perm(half[0].x, half[1].x, 0x5140), __byte_perm(half[0].x, half[1].x, 0x7362),
                             __byte_perm(half[0].y, half[1].y, 0x5140), __byte_perm(half[0].y, half[1].y, 0x7362));
        }
      }
    }
    cluster.sync();  // everything of the round has been read
    if (moves && to_pid >= 0) {
      uint8_t* to = head.block(to_pid, blk * 16, Geo::kBytes);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int x = i * 32 + lane, t = x / (D / 16), pair = x / (D / 8);
        *reinterpret_cast<uint4*>(to + t * D + Geo::k_piece(t, x % (D / 16)) * 16) = kw[i];
        *reinterpret_cast<uint4*>(to + Geo::kVOff + pair * 2 * D + Geo::v_piece(pair, x % (D / 8)) * 16) = vw[i];
      }
      const uint32_t bits_k = __ballot_sync(0xffffffffu, lane < 16 && (marks & 1u));
      const uint32_t bits_v = __ballot_sync(0xffffffffu, lane < 16 && (marks >> 16));
      if (lane == 0)
        *reinterpret_cast<uint4*>(to + Geo::kParams) =
            make_uint4(__float_as_uint(k_to), __float_as_uint(v_to), bits_k | bits_v << 16, 0);
      if (lane < 16 && src >= 0) *head.mass(to_pid, blk * 16 + lane) = m;
    }
  }
}

template <int D>
cudaError_t evict(const Kv8EvictArgs& a, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a.b.batch * a.c.heads * ctas));
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_evict_kernel<D>, a);
}

}  // namespace

cudaError_t moe::kv8_evict(const Kv8& kv, const Kv8EvictArgs& a, cudaStream_t s) {
  const int64_t items = (int64_t)a.b.batch * a.c.heads;
  int ctas = kEvMaxCluster;
  while (ctas > 1 && items * ctas > 2 * kv.sms) ctas >>= 1;  // as many as two a multiprocessor hold at once
  if (items * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return kv.d.head_dim == 64 ? evict<64>(a, ctas, s) : evict<128>(a, ctas, s);
}
