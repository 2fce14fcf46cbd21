// Choice of the pages a query attends to.  Per row and kv head, with qs the
// sum of the group's query heads (ascending, fp32) and M, m the page's bounds,
//     score(page) = sum over d of max(qs[d] M[d], qs[d] m[d]),
// an upper bound of qs . k over the page's keys.  The summation order is fixed
// (adjacent pairs, level by level), so that the choice is the same on every
// run and can be checked to the bit.  The first and the last pages are always
// taken, then the highest scores, ties to the lower page; a NaN score counts
// as minus infinity.
//
// Scoring streams the bounds (2 D values per page and head); picking works on
// the scores' order-preserving keys: the value of the last key that is taken by
// bisection, then one ordered pass.  Rows with few pages do both in one CTA per
// row and head (keys in shared memory); otherwise the pages of a row are spread
// over CTAs first and a second kernel picks.
//
// Measured, 16 rows of contexts up to 131,072 (pages of 64, 8 kv heads of 128
// channels): scores 27 us for 104 MB of bounds, 3.8 TB/s, at 48 % of the issue
// slots: every CTA starts with the chain length -> page numbers -> bounds, and the
// some 800 that have pages are just above the 760 that the SMs hold at once (16, 32
// and 64 pages a CTA are within 1 us of each other);
// choice 8 us, one CTA a row and head, a barrier a step of the bisection: latency.
// One row of 6,001 tokens, with the attention over its 16 pages: 16.4 us.
#include "kv_internal.h"

using namespace moe;

namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelPages = 32;     // pages per scoring CTA
constexpr int kSelHeads = 16;     // kv heads per scoring CTA
constexpr uint32_t kAlways = 0xffffffffu;  // above the key of +infinity

// Order-preserving key of a score (-0 and +0 equal), NaN as -infinity.
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) v = -__int_as_float(0x7f800000);
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct Row {
  int s, i;
  KvSeq q;
  int pages;  // pages the row sees
};
__device__ __forceinline__ Row row_of(const KvSelectArgs& a, int64_t r) {
  Row w;
  w.s = (int)(r / a.b.max_new);
  w.i = (int)(r % a.b.max_new);
  w.q = kv_seq(a.b, w.s);
  const int64_t pos = min((int64_t)w.q.len - w.q.rows + w.i, (int64_t)kv_capacity(a.c, a.b) - 1);
  w.pages = w.i >= w.q.rows || pos < 0 ? 0 : (int)(pos >> a.c.page_shift) + 1;
  return w;
}

// qs[8 o ..] of one head, eight channels.
template <typename T, int D>
__device__ __forceinline__ void head_sum(const KvSelectArgs& a, const Row& w, int h, int o, float* qs) {
  const int per = a.q_heads / a.c.heads;
  const uint16_t* src = a.q + kv_row_offset(a.b, a.qs, w.s, w.q.row0, w.i) + (int64_t)h * per * a.qs.head + 8 * o;
  float v[8];
#pragma unroll 8
  for (int x = 0; x < per; ++x) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(src + x * a.qs.head));
    const uint32_t c[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = x ? __fadd_rn(v[2 * e], KvType<T>::lo(c[e])) : KvType<T>::lo(c[e]);
      v[2 * e + 1] = x ? __fadd_rn(v[2 * e + 1], KvType<T>::hi(c[e])) : KvType<T>::hi(c[e]);
    }
  }
  *reinterpret_cast<float4*>(qs + 8 * o) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(qs + 8 * o + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// A lane's part (eight channels) of a page's score: three levels of the sum's tree.
template <typename T, int D>
__device__ __forceinline__ float score_part(const float* qs, uint4 hi, uint4 lo) {
  const int l = threadIdx.x % (D / 8);
  const float4 q0 = *reinterpret_cast<const float4*>(qs + 8 * l), q1 = *reinterpret_cast<const float4*>(qs + 8 * l + 4);
  const float q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, o[4] = {lo.x, lo.y, lo.z, lo.w};
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = max_nan(__fmul_rn(q[2 * e], KvType<T>::lo(h[e])), __fmul_rn(q[2 * e], KvType<T>::lo(o[e])));
    v[2 * e + 1] = max_nan(__fmul_rn(q[2 * e + 1], KvType<T>::hi(h[e])), __fmul_rn(q[2 * e + 1], KvType<T>::hi(o[e])));
  }
  return __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3])),
                   __fadd_rn(__fadd_rn(v[4], v[5]), __fadd_rn(v[6], v[7])));
}

// Keys of pages [j0, j1) and heads [h0, h1) of a row: D / 8 lanes take a page of every
// kSelThreads / (D / 8), and of it four heads at once (HEADS), or they take one head (h0)
// of four pages at once.  ids: [page - j0] page numbers, -1 where there is none; qs:
// [head - h0][D]; keys[(head - h0) * stride + page - j0].
template <typename T, int D, bool HEADS>
__device__ __forceinline__ void score_pages(const KvSelectArgs& a, const Row& w, int j0, int j1, int h0, int h1,
                                            const int32_t* ids, const float* qs, uint32_t* keys, int64_t stride) {
  constexpr int L = D / 8, kGroups = kSelThreads / L, kAtOnce = 4;
  const int l = threadIdx.x % L, grp = threadIdx.x / L, nh = HEADS ? h1 - h0 : 1, np = j1 - j0;
  for (int p0 = 0; p0 < np; p0 += kGroups * (HEADS ? 1 : kAtOnce)) {  // every lane goes round: lanes of a group shuffle
    for (int x0 = 0; x0 < nh; x0 += kAtOnce) {
      uint4 hi[kAtOnce], lo[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {  // what is out of range or in no page reads something, and is not used
        const int p = min(p0 + grp + (HEADS ? 0 : x * kGroups), np - 1), h = HEADS ? min(x0 + x, nh - 1) : 0;
        const uint4* ends = reinterpret_cast<const uint4*>(a.c.bounds + ((int64_t)max(ids[p], 0) * a.c.heads + h0 + h) * (2 * D));
        hi[x] = __ldg(ends + l);
        lo[x] = __ldg(ends + L + l);
      }
      float s[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) s[x] = score_part<T, D>(qs + (HEADS ? min(x0 + x, nh - 1) : 0) * D, hi[x], lo[x]);
      // the tree's next levels pair neighbouring lanes; in the first two every lane keeps one of
      // two units and gives the other away, so that lane l ends with unit l % 4
      const bool odd = l & 1, upper = l & 2;
      float s0 = odd ? s[1] : s[0], s1 = odd ? s[3] : s[2];
      s0 = __fadd_rn(s0, __shfl_xor_sync(0xffffffffu, odd ? s[0] : s[1], 1));
      s1 = __fadd_rn(s1, __shfl_xor_sync(0xffffffffu, odd ? s[2] : s[3], 1));
      float sum = upper ? s1 : s0;
      sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, upper ? s0 : s1, 2));
#pragma unroll
      for (int x = 4; x < L; x <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, x));
      const int p = p0 + grp + (HEADS ? 0 : l * kGroups), h = HEADS ? x0 + l : 0, j = j0 + p;
      if (l < kAtOnce && p < np && h < nh)
        keys[h * stride + p] = j < a.first || j >= w.pages - a.last
                                   ? kAlways
                                   : score_key(ids[p] >= 0 ? sum : -__int_as_float(0x7f800000));
    }
  }
}

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
  for (int w = 0; w < kSelWarps; ++w)
    if (w < warp) v += sh[w];
  return v;
}

// The list of a row and head from its n > budget keys.  KEYS > 0: every thread holds
// the keys tid, tid + 256, ... in registers (n <= 256 KEYS); 0: they are read each time.
template <int KEYS>
__device__ __forceinline__ void pick(const KvSelectArgs& a, const uint32_t* keys, int n, int32_t* out) {
  __shared__ uint32_t sh_lo[kSelWarps], sh_hi[kSelWarps];
  __shared__ int sh_cnt[2][kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t held[KEYS > 0 ? KEYS : 1];  // kAlways and the places past n as 0: below every key that counts
  if constexpr (KEYS > 0) {
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      const int j = tid + x * kSelThreads;
      held[x] = j < n ? keys[j] : 0u;
      if (held[x] == kAlways) held[x] = 0u;
    }
  }
  int need = a.budget - a.first - a.last;  // pages to take by score
  uint32_t tau = kAlways - 1;              // keys above are taken, and `need` of those equal, lowest pages first
  if (need > 0) {
    uint32_t lo = kAlways, hi = 0;  // of the keys that count
    auto widen = [&](uint32_t k) {
      if (k != 0u && k != kAlways) {
        lo = min(lo, k);
        hi = max(hi, k);
      }
    };
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int x = 0; x < KEYS; ++x) widen(held[x]);
    } else {
      for (int j = tid; j < n; j += kSelThreads) widen(keys[j]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      sh_lo[warp] = lo;
      sh_hi[warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      lo = min(lo, sh_lo[w]);
      hi = max(hi, sh_hi[w]);
    }
    // at least `need` keys are >= lo, fewer are > hi; above: how many are > hi
    int above = 0;
    for (int it = 0; lo < hi; it ^= 1) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      int c = 0;
      if constexpr (KEYS > 0) {
#pragma unroll
        for (int x = 0; x < KEYS; ++x) c += held[x] >= mid;
      } else {
#pragma unroll 4
        for (int j = tid; j < n; j += kSelThreads) {
          const uint32_t k = keys[j];
          c += k >= mid && k != kAlways;
        }
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) sh_cnt[it][warp] = c;  // two buffers: one barrier per step
      __syncthreads();
      c = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) c += sh_cnt[it][w];
      if (c >= need) {
        lo = mid;
        if (c == need) {  // exactly the keys from mid on
          above = need;
          hi = lo = mid - 1;
        }
      } else {
        hi = mid - 1;
        above = c;
      }
    }
    tau = lo;
    need -= above;
  }
  // every thread takes a run of pages: ranks of the keys equal to tau, then places in the list
  const int run = (n + kSelThreads - 1) / kSelThreads;
  const int b = min(tid * run, n), e = min(b + run, n);
  int eq = 0, gt = 0;
  for (int j = b; j < e; ++j) {
    const uint32_t k = keys[j];
    eq += k == tau;
    gt += k > tau;
  }
  int rank = cta_scan(eq, sh_cnt[0]) - eq;
  const int taken = gt + min(eq, max(need - rank, 0));
  int at = cta_scan(taken, sh_cnt[1]) - taken;
  for (int j = b; j < e; ++j) {
    const uint32_t k = keys[j];
    if (k > tau || (k == tau && rank++ < need)) out[at++] = j;
  }
}

__device__ __forceinline__ int32_t* list_of(const KvSelectArgs& a, const Row& w, int h) {
  return a.out + (kv_row_index(a.b, w.s, w.q.row0, w.i) * a.c.heads + h) * a.budget;
}
// All pages, where they are no more than the budget.
__device__ __forceinline__ void list_all(const KvSelectArgs& a, const Row& w, int32_t* out) {
  for (int x = threadIdx.x; x < a.budget; x += kSelThreads) out[x] = x < w.pages ? x : -1;
}

// One CTA per (row, head): scores and choice.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ KvSelectArgs a) {
  __shared__ __align__(16) float qs[D];
  __shared__ uint32_t keys[kKvSelOwn];
  __shared__ int32_t ids[kKvSelOwn];
  const int h = blockIdx.x % a.c.heads;
  const Row w = row_of(a, blockIdx.x / a.c.heads);
  if (w.i >= w.q.rows) return;
  int32_t* out = list_of(a, w, h);
  if (w.pages <= a.budget) return list_all(a, w, out);
  for (int j = threadIdx.x; j < w.pages; j += kSelThreads) ids[j] = (int32_t)kv_page(a.c, a.b, w.s, j);
  if (threadIdx.x < D / 8) head_sum<T, D>(a, w, h, threadIdx.x, qs);
  __syncthreads();
  score_pages<T, D, false>(a, w, 0, w.pages, h, h + 1, ids, qs, keys, 0);
  __syncthreads();
  pick<kKvSelOwn / kSelThreads>(a, keys, w.pages, out);
}

// Scores: one CTA per (row, kSelPages pages, kSelHeads heads).
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) kv_score_kernel(const __grid_constant__ KvSelectArgs a, int64_t first_row,
                                                               int chunks, uint32_t* __restrict__ keys) {
  __shared__ __align__(16) float qs[kSelHeads * D];
  __shared__ int32_t ids[kSelPages];
  static_assert(kSelPages <= kSelThreads, "one page number per thread");
  const int64_t r = blockIdx.x / chunks;
  const Row w = row_of(a, first_row + r);
  const int j0 = blockIdx.x % chunks * kSelPages, j1 = min(j0 + kSelPages, w.pages);
  if (w.pages <= a.budget || j0 >= j1) return;
  const int h0 = blockIdx.y * kSelHeads, h1 = min(h0 + kSelHeads, a.c.heads);
  if (threadIdx.x < j1 - j0) ids[threadIdx.x] = (int32_t)kv_page(a.c, a.b, w.s, j0 + threadIdx.x);
  for (int x = threadIdx.x; x < (h1 - h0) * (D / 8); x += kSelThreads)
    head_sum<T, D>(a, w, h0 + x / (D / 8), x % (D / 8), qs + x / (D / 8) * D);
  __syncthreads();
  score_pages<T, D, true>(a, w, j0, j1, h0, h1, ids, qs, keys + (r * a.c.heads + h0) * a.b.table_pages + j0, a.b.table_pages);
}
// ... and the choice: one CTA per (row, head).
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads) kv_pick_kernel(const __grid_constant__ KvSelectArgs a, int64_t first_row,
                                                              const uint32_t* __restrict__ keys) {
  const int h = blockIdx.x % a.c.heads;
  const Row w = row_of(a, first_row + blockIdx.x / a.c.heads);
  if (w.i >= w.q.rows) return;
  if (w.pages <= a.budget) return list_all(a, w, list_of(a, w, h));
  pick<KEYS>(a, keys + (int64_t)blockIdx.x * a.b.table_pages, w.pages, list_of(a, w, h));
}

template <typename T, int D>
cudaError_t select(Kv& kv, const KvSelectArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.b.batch * a.b.max_new;
  if (a.b.table_pages <= kKvSelOwn) {
    if (rows * a.c.heads > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv_select_kernel<T, D><<<(unsigned)(rows * a.c.heads), kSelThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  uint32_t* keys = reinterpret_cast<uint32_t*>(kv.ws);
  const int chunks = (a.b.table_pages + kSelPages - 1) / kSelPages;
  const int64_t step = std::min<int64_t>((int64_t)(Kv::kScoreBytes / 4) / ((int64_t)a.c.heads * a.b.table_pages),
                                         0x7fffffff / std::max(chunks, a.c.heads));
  const unsigned head_tiles = (unsigned)((a.c.heads + kSelHeads - 1) / kSelHeads);
  for (int64_t r = 0; r < rows; r += step) {  // as many rows at a time as the workspace holds scores for
    const int64_t n = std::min(step, rows - r);
    kv_score_kernel<T, D><<<dim3((unsigned)(n * chunks), head_tiles), kSelThreads, 0, s>>>(a, r, chunks, keys);
    // keys in registers / read again each step (us, 1 and 16 rows): tables of 1,024 pages 10.7 / 11.7,
    // 16.5 / 17.9; of 4,096 13.5 / 18.5, 56.8 / 63.9.  32 keys a thread cost tables of 1,024 2.8 us
    // (and would take 11.6 off 34.1 at 8,192 pages).
    const auto pick_kernel = a.b.table_pages <= 16 * kSelThreads ? kv_pick_kernel<16> : kv_pick_kernel<0>;
    pick_kernel<<<(unsigned)(n * a.c.heads), kSelThreads, 0, s>>>(a, r, keys);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t moe::kv_select(Kv& kv, const KvSelectArgs& a, cudaStream_t s) {
  if (kv.d.dtype == MOE_KV_BF16)
    return kv.d.head_dim == 128 ? select<__nv_bfloat16, 128>(kv, a, s) : select<__nv_bfloat16, 64>(kv, a, s);
  return kv.d.head_dim == 128 ? select<__half, 128>(kv, a, s) : select<__half, 64>(kv, a, s);
}
