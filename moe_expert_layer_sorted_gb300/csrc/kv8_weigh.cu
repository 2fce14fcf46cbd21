// The weight of every token: after an attention, the softmax weights of its rows, summed over the
// rows and query heads that see the token, are added to the token's mass.
//
// With lse from the attention a weight is 2^(y - lse log2 e), y the score in log2 units as the
// attention computes it, so that a token's sum needs its keys and the queries alone: one warp per
// block of 16 tokens and kv head holds the codes as the rows of mma.m16n8k16 and walks over the
// columns (row, query head), eight at a time.  A token's sum is one lane's and its neighbours', in
// the order of the columns: no atomics.
#include "kv8_internal.h"

using namespace moe;

namespace {

#include "device_common.cuh"
#include "kv_operand.cuh"
#include "kv_rounds.cuh"

template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_weigh_kernel(const __grid_constant__ KvAttnArgs a, float* __restrict__ mass, int chunks) {
  using Geo = Kv8Geom<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int h = blockIdx.x % a.c.heads, per = a.q_heads / a.c.heads;
  const int s = blockIdx.x / a.c.heads / chunks;
  const KvSeq q = kv_seq(a.b, s);
  const int pos = (blockIdx.x / a.c.heads % chunks * 8 + warp) * 16;
  if (pos >= min(q.len, kv_capacity(a.c, a.b)) || q.rows == 0) return;
  const int64_t pid = kv_page(a.c, a.b, s, pos >> a.c.page_shift);
  if (pid < 0) return;
  const int off = pos & (a.c.page_size - 1);
  const uint8_t* blk = a.c.pages + pid * a.c.page_stride + h * a.c.head_stride + (off >> 4) * (int64_t)Geo::kBytes;
  uint32_t kf[D / 4];  // the codes as operand: D / 16 steps of four registers
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t lo[4], hi[4];
    load_words(lo, blk + r * D + Geo::k_piece(r, c + 4 * i) * 16);
    load_words(hi, blk + (r + 8) * D + Geo::k_piece(r, c + 4 * i) * 16);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      kf[16 * i + 4 * w] = kv8_pair<0>(lo[w]);
      kf[16 * i + 4 * w + 1] = kv8_pair<0>(hi[w]);
      kf[16 * i + 4 * w + 2] = kv8_pair<1>(lo[w]);
      kf[16 * i + 4 * w + 3] = kv8_pair<1>(hi[w]);
    }
  }
  const float ks = *reinterpret_cast<const float*>(blk + Geo::kParams);
  const int64_t first = (int64_t)q.len - q.rows;  // position of row 0
  const int64_t skip = a.causal ? max((int64_t)pos - first, (int64_t)0) : max(-first, (int64_t)0);  // rows that see nothing of the block
  const int64_t cols = (int64_t)q.rows * per;
  float sum[2] = {0.0f, 0.0f};  // of tokens r and r + 8, columns 2 c, 2 c + 1 of each eight
  for (int64_t x0 = skip * per / 8 * 8; x0 < cols; x0 += 8) {
    const int64_t x = x0 + r;
    const bool real = x < cols;
    const int i = real ? (int)(x / per) : 0, hq = h * per + (real ? (int)(x % per) : 0);
    const uint16_t* src = a.q + kv_row_offset(a.b, a.qs, s, q.row0, i) + (int64_t)hq * a.qs.head;
    uint4 raw[D / 32];
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      raw[w] = real ? *reinterpret_cast<const uint4*>(src + (c + 4 * (w / 2)) * 16 + w % 2 * 8) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = max(top, max(__float_as_uint(fabsf(KvType<T>::lo(v[e]))), __float_as_uint(fabsf(KvType<T>::hi(v[e])))));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int ex = (int)(top >> 23) - 127;
    const int by = top == 0u || ex > 127 ? 0 : min(max(14 - ex, -113), 113);
    const float up = pow2(by);
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
      uint32_t f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = KvType<__half>::pack(KvType<T>::lo(v[e]) * up, KvType<T>::hi(v[e]) * up);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int k = 8 * w + 2 * e;
        mma_f16(y, kf[k], kf[k + 1], kf[k + 2], kf[k + 3], f[e], f[e + 1]);
      }
    }
    // column x's factor, lse in log2 units (NaN: its weights are not counted) and what it sees
    const float back = a.scale * 1.4426950408889634f * pow2(-by);
    const float ls = real ? a.lse[kv_row_index(a.b, s, q.row0, i) * a.q_heads + hq] : __int_as_float(0x7fffffff);
    const float off2 = fabsf(ls) < __int_as_float(0x7f800000) ? ls * 1.4426950408889634f : __int_as_float(0x7fffffff);
    const int64_t p = first + i;
    const int see = !real || p < 0 ? 0 : (int)min(a.causal ? p + 1 : (int64_t)q.len, (int64_t)0x7fffffff);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e)), o = __shfl_sync(0xffffffffu, off2, 4 * (2 * c + e));
      const int n = __shfl_sync(0xffffffffu, see, 4 * (2 * c + e));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float w = exp2_fast(y[2 * t + e] * f * ks - o);
        if (pos + r + 8 * t < n && o == o) sum[t] += w;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 1);
    sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 2);
    if (c == 0 && pos + r + 8 * t < q.len) mass[(pid * a.c.heads + h) * a.c.page_size + off + r + 8 * t] += sum[t];
  }
}

}  // namespace

cudaError_t moe::kv8_weigh(Kv8& kv, const KvAttnArgs& a, float* mass, cudaStream_t s) {
  const int64_t chunks = (((int64_t)a.b.table_pages << a.c.page_shift) + 127) / 128;
  const int64_t ctas = chunks * a.c.heads * a.b.batch;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV8_DISPATCH(kv.d, {
    kv8_weigh_kernel<T, D><<<(unsigned)ctas, 256, 0, s>>>(a, mass, (int)chunks);
    e = cudaGetLastError();
  });
  return e;
}
