// Attention over the 4-bit key/value cache, o = softmax(scale q k^T) v: one
// warp per (row, query head), the online softmax over the tokens it may see.
#include "kv_internal.h"

using namespace moe;

namespace {

template <typename T, int D, int G>
__global__ void __launch_bounds__(128) kv_attention_kernel(KvAttnArgs a) {
  using Geo = KvGeom<D, G>;
  constexpr int kWords = D / 8, kTok = 32 / kWords;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int hq = (int)(unit % a.q_heads);
  const int64_t r = unit / a.q_heads;
  if (r >= (int64_t)a.b.batch * a.b.max_new) return;
  const int s = (int)(r / a.b.max_new), i = (int)(r % a.b.max_new);
  const KvSeq q = kv_seq(a.b, s);
  if (i >= q.rows) return;
  const int h = hq / (a.q_heads / a.c.heads);
  const int64_t pos = (int64_t)q.len - q.rows + i;
  int64_t seen = a.causal ? pos + 1 : (int64_t)q.len;
  seen = min(max(seen, (int64_t)0), (int64_t)kv_capacity(a.c, a.b));
  const int w = lane % kWords, g = 8 * w / G;
  float qf[8], o[8], m = -__int_as_float(0x7f800000), l = 0.0f;
  const uint4 raw = *reinterpret_cast<const uint4*>(a.q + kv_row_offset(a.b, a.qs, s, q.row0, i) + hq * a.qs.head + 8 * w);
  const uint32_t r4[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    qf[2 * e] = KvType<T>::lo(r4[e]);
    qf[2 * e + 1] = KvType<T>::hi(r4[e]);
    o[2 * e] = o[2 * e + 1] = 0.0f;
  }
  const int64_t row = kv_row_index(a.b, s, q.row0, i);
  const int32_t* sel = a.sel ? a.sel + (row * a.c.heads + h) * a.budget : nullptr;
  const int64_t pages = sel ? a.budget : (seen + a.c.page_size - 1) >> a.c.page_shift;
  for (int64_t n = 0; n < pages; ++n) {
    const int64_t j = sel ? sel[n] : n;
    if (j < 0 || j << a.c.page_shift >= seen) continue;
    const int64_t pid = kv_page(a.c, a.b, s, (int)j);
    if (pid < 0) continue;
    const uint8_t* base = a.c.pages + pid * a.c.page_stride + h * a.c.head_stride;
    const int count = (int)min((int64_t)a.c.page_size, seen - (j << a.c.page_shift));
    for (int t0 = 0; t0 < count; t0 += kTok) {
      const int off = t0 + lane / kWords, t = off & 15;
      const uint8_t* blk = base + (off >> 4) * Geo::kBytes;
      const uint32_t kw = reinterpret_cast<const uint32_t*>(blk + t * Geo::kRow)[Geo::k_word(w)];
      const uint32_t kp = reinterpret_cast<const uint32_t*>(blk + Geo::kKPar + t * Geo::kParRow)[g];
      float sc = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sc = fmaf(qf[e], fmaf(KvType<T>::lo(kp), kv_code(kw, e), KvType<T>::hi(kp)), sc);
#pragma unroll
      for (int x = 1; x < kWords; x <<= 1) sc += __shfl_xor_sync(0xffffffffu, sc, x);
      if (off < count) {
        sc *= a.scale;
        const float mn = fmaxf(m, sc), fix = m == mn ? 1.0f : expf(m - mn), p = expf(sc - mn);
        const uint32_t vw = kv_v_codes<D, G>(
            reinterpret_cast<const uint32_t*>(blk + Geo::kVOff + kv_v_row(t) * Geo::kRow), w, kv_v_flip<D>(t));
        const uint32_t vp = reinterpret_cast<const uint32_t*>(blk + Geo::kVPar + t * Geo::kParRow)[g];
        l = l * fix + p;
        m = mn;
  #pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = fmaf(p, fmaf(KvType<T>::lo(vp), kv_code(vw, e), KvType<T>::hi(vp)), o[e] * fix);
      }
      __syncwarp();
    }
  }
#pragma unroll
  for (int x = kWords; x < 32; x <<= 1) {  // join the tokens' parts
    const float m2 = __shfl_xor_sync(0xffffffffu, m, x), l2 = __shfl_xor_sync(0xffffffffu, l, x);
    const float mn = fmaxf(m, m2);
    const float f1 = l > 0.0f ? expf(m - mn) : (l == l ? 0.0f : l), f2 = l2 > 0.0f ? expf(m2 - mn) : (l2 == l2 ? 0.0f : l2);
    l = l * f1 + l2 * f2;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f1 + __shfl_xor_sync(0xffffffffu, o[e], x) * f2;
    m = mn;
  }
  if (lane < kWords) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is zero
    *reinterpret_cast<uint4*>(a.out + kv_row_offset(a.b, a.os, s, q.row0, i) + hq * a.os.head + 8 * w) =
        make_uint4(KvType<T>::pack(o[0] * inv, o[1] * inv), KvType<T>::pack(o[2] * inv, o[3] * inv),
                   KvType<T>::pack(o[4] * inv, o[5] * inv), KvType<T>::pack(o[6] * inv, o[7] * inv));
    if (a.lse && lane == 0) a.lse[row * a.q_heads + hq] = l == 0.0f ? -__int_as_float(0x7f800000) : m + logf(l);
  }
}

}  // namespace

cudaError_t moe::kv_attention(Kv& kv, const KvAttnArgs& a, cudaStream_t s) {
  if (a.sel || (int64_t)a.b.max_new * (a.q_heads / a.c.heads) <= 32)
    return kv.d.dtype == MOE_KV_BF16 ? kv_decode_bf16(kv, a, s) : kv_decode_f16(kv, a, s);
  const int64_t warps = (int64_t)a.b.batch * a.b.max_new * a.q_heads;
  if (warps / 4 + 1 > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV_DISPATCH(kv.d, {
    kv_attention_kernel<T, D, G><<<(unsigned)((warps + 3) / 4), 128, 0, s>>>(a);
    e = cudaGetLastError();
  });
  return e;
}
