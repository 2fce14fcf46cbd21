// Choice of the pages a query attends to.  Per row and kv head, with qs the
// sum of the group's query heads (ascending, fp32) and M, m the page's bounds,
//     score(page) = sum over d of max(qs[d] M[d], qs[d] m[d]),
// an upper bound of qs . k over the page's keys.  The summation order is fixed
// (adjacent pairs, level by level), so that the choice is the same on every
// run and can be checked to the bit.  The first and the last pages are always
// taken, then the highest scores, ties to the lower page; a NaN score counts
// as minus infinity.
#include "kv_internal.h"

using namespace moe;

namespace {

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

// One CTA of 256 threads per (row, head) of the rows first_row ..: scores into
// keys, the budget-th largest key by four 8-bit radix passes, then the list in
// ascending page order.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_select_kernel(KvSelectArgs a, int64_t first_row, uint32_t* keys_all) {
  constexpr int C = D / 32;  // channels per lane
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int wsum[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.c.heads;
  const int64_t r = first_row + blockIdx.x / a.c.heads;
  const int s = (int)(r / a.b.max_new), i = (int)(r % a.b.max_new);
  const KvSeq q = kv_seq(a.b, s);
  if (i >= q.rows) return;
  const int64_t pos = min((int64_t)q.len - q.rows + i, (int64_t)kv_capacity(a.c, a.b) - 1);
  const int n = pos < 0 ? 0 : (int)(pos >> a.c.page_shift) + 1;  // pages the row sees
  int32_t* out = a.out + (kv_row_index(a.b, s, q.row0, i) * a.c.heads + h) * a.budget;
  if (n <= a.budget) {
    for (int x = tid; x < a.budget; x += 256) out[x] = x < n ? x : -1;
    return;
  }
  uint32_t* keys = keys_all + (int64_t)blockIdx.x * a.b.table_pages;
  const int per = a.q_heads / a.c.heads;
  const uint16_t* qr = a.q + kv_row_offset(a.b, a.qs, s, q.row0, i) + (int64_t)h * per * a.qs.head + C * lane;
  float qs[C];
#pragma unroll
  for (int c = 0; c < C; ++c) qs[c] = KvType<T>::to_f(qr[c]);
  for (int x = 1; x < per; ++x)
#pragma unroll
    for (int c = 0; c < C; ++c) qs[c] = __fadd_rn(qs[c], KvType<T>::to_f(qr[x * a.qs.head + c]));
  for (int j = warp; j < n; j += 8) {
    uint32_t key = kAlways;
    if (j >= a.first && j < n - a.last) {
      float sc = -__int_as_float(0x7f800000);
      const int64_t pid = kv_page(a.c, a.b, s, j);
      if (pid >= 0) {
        const uint16_t* ends = a.c.bounds + (pid * a.c.heads + h) * (2 * D) + C * lane;
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
          v[c] = max_nan(__fmul_rn(qs[c], KvType<T>::to_f(ends[c])), __fmul_rn(qs[c], KvType<T>::to_f(ends[D + c])));
#pragma unroll
        for (int st = 1; st < C; st <<= 1)
#pragma unroll
          for (int c = 0; c < C; c += 2 * st) v[c] = __fadd_rn(v[c], v[c + st]);
        sc = v[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sc = __fadd_rn(sc, __shfl_xor_sync(0xffffffffu, sc, o));
      }
      key = score_key(sc);
    }
    if (lane == 0) keys[j] = key;
  }
  if (tid == 0) {
    sh_prefix = 0;
    sh_need = (uint32_t)a.budget;
  }
  __syncthreads();
  for (int shift = 24; shift >= 0; shift -= 8) {  // the budget-th largest key, byte by byte
    hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = sh_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = tid; j < n; j += 256)
      if ((keys[j] & mask) == prefix) atomicAdd(&hist[(keys[j] >> shift) & 255u], 1u);
    __syncthreads();
    if (tid == 0) {
      uint32_t need = sh_need;
      int bin = 255;
      while (bin > 0 && hist[bin] < need) need -= hist[bin--];
      sh_prefix = prefix | (uint32_t)bin << shift;
      sh_need = need;
    }
    __syncthreads();
  }
  const uint32_t tau = sh_prefix;
  int left = (int)sh_need, done = 0;  // keys equal to tau still to take; entries written
  for (int base = 0; base < n; base += 256) {
    const int j = base + tid;
    const uint32_t key = j < n ? keys[j] : 0u;
    const bool eq = j < n && key == tau;
    const uint32_t beq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) wsum[0][warp] = __popc(beq);
    __syncthreads();
    int before = __popc(beq & ((1u << lane) - 1u)), all = 0;
    for (int x = 0; x < 8; ++x) {
      before += x < warp ? wsum[0][x] : 0;
      all += wsum[0][x];
    }
    const bool take = j < n && (key > tau || (eq && before < left));
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) wsum[1][warp] = __popc(bt);
    __syncthreads();
    int at = done + __popc(bt & ((1u << lane) - 1u)), sum = 0;
    for (int x = 0; x < 8; ++x) {
      at += x < warp ? wsum[1][x] : 0;
      sum += wsum[1][x];
    }
    if (take) out[at] = j;
    done += sum;
    left = max(left - all, 0);
  }
}

}  // namespace

cudaError_t moe::kv_select(Kv& kv, const KvSelectArgs& a, cudaStream_t s) {
  const int64_t per_row = (int64_t)a.c.heads * a.b.table_pages;  // keys
  const int64_t rows = (int64_t)a.b.batch * a.b.max_new;
  const int64_t step = std::min<int64_t>((int64_t)(Kv::kScoreBytes / 4) / per_row, 0x7fffffff / a.c.heads);
  for (int64_t r = 0; r < rows; r += step) {
    const unsigned ctas = (unsigned)(std::min(step, rows - r) * a.c.heads);
    KV_DISPATCH(kv.d, {
      kv_select_kernel<T, D><<<ctas, 256, 0, s>>>(a, r, reinterpret_cast<uint32_t*>(kv.ws));
    });
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
