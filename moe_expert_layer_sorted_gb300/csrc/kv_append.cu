// Writing and reading the 4-bit key/value cache.
//
// A group of G channels of one token and head is stored as u in 0..15 with a
// step s and a centre c in the cache's 16-bit type:
//     s = rn((max - min) / 15),  c = rn(min + 8 s),
//     u = clamp(rint((x - c) / s) + 8, 0, 15)  (8 where s = 0),
//     stored value c + s (u - 8).
// s and c are rounded before u is chosen, so that their rounding costs no more
// than a clamped end code.  The centre sits at code 8 and not at the minimum:
// the codes the attention multiplies are then the small signed u - 8, and the
// rounding of a probability times s is not amplified by an offset.  A group
// that holds an infinity or a NaN gets c = NaN, s = 0: it reads as NaN and
// harms no other group.  All arithmetic is fp32, one rounding per operation.
#include "kv_internal.h"

using namespace moe;

namespace {

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// One CTA per (sequence, page it writes to, head), the first half of its warps
// on the keys and the second on the values; D / 8 lanes hold a row, eight
// channels each, so that a lane makes one code word.  The page is the CTA's
// own, so its bounds need no atomics.
template <typename T, int D, int G>
__global__ void kv_append_kernel(KvView c, KvBatch b, const uint16_t* __restrict__ k, KvRows ks,
                                 const uint16_t* __restrict__ v, KvRows vs, int pages_per_seq) {
  using Geo = KvGeom<D, G>;
  constexpr int kLanes = D / 8, kTok = 32 / kLanes;  // lanes per row, rows per warp
  extern __shared__ float red[];                     // [key warps][max, min][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = blockDim.x >> 6;
  const int h = blockIdx.x % c.heads;
  const int u = blockIdx.x / c.heads, s = u / pages_per_seq;
  const KvSeq q = kv_seq(b, s);
  const int64_t first = (int64_t)q.len - q.rows;  // position of row 0 (negative: rows before the sequence, dropped)
  const int64_t p0 = first > 0 ? first : 0;
  const int64_t j = (p0 >> c.page_shift) + u % pages_per_seq;
  const int64_t begin = max(p0, j << c.page_shift);
  const int64_t end = min(min((j + 1) << c.page_shift, (int64_t)q.len), (int64_t)kv_capacity(c, b));
  if (begin >= end) return;
  const int64_t pid = kv_page(c, b, s, (int)j);
  if (pid < 0) return;
  uint8_t* base = c.pages + pid * c.page_stride + h * c.head_stride;
  const bool keys = warp < half;
  const uint16_t* src = (keys ? k : v) + kv_row_offset(b, keys ? ks : vs, s, q.row0, 0) + h * (keys ? ks.head : vs.head);
  const int64_t stride = keys ? ks.row : vs.row;
  const int w = lane % kLanes, g = 8 * w / G;
  float top[8], bot[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top[e] = -__int_as_float(0x7f800000);
    bot[e] = __int_as_float(0x7f800000);
  }
  for (int64_t p = begin + (warp % half) * kTok; p < end; p += half * kTok) {
    const int64_t pos = p + lane / kLanes;
    const bool live = pos < end;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(src + (pos - first) * stride + 8 * w);
    const uint32_t r4[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = KvType<T>::lo(r4[i]);
      x[2 * i + 1] = KvType<T>::hi(r4[i]);
    }
    float lo = x[0], hi = x[0], zero = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      zero = fmaf(x[e], 0.0f, zero);  // NaN where an element is not finite
    }
    bool bad = !(zero == 0.0f);
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
    }
    uint16_t sb = KvType<T>::from_f(__fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f)));
    uint16_t cb = KvType<T>::from_f(fmaf(8.0f, KvType<T>::to_f(sb), lo));  // 8 s is exact
    if (bad) {
      sb = 0;
      cb = 0x7fff;  // NaN in both types
    }
    const float sf = KvType<T>::to_f(sb), cf = KvType<T>::to_f(cb);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float q8 = sf > 0.0f ? rintf(__fdiv_rn(__fsub_rn(x[e], cf), sf)) : 0.0f;
      q8 = fminf(fmaxf(q8, -8.0f), 7.0f);
      word |= (uint32_t)((int)q8 + 8) << (4 * ((e >> 1) + 4 * (e & 1)));
      if (live && keys) {
        const float y = fmaf(sf, q8, cf);  // s q8 is exact
        top[e] = max_nan(top[e], y);
        bot[e] = min_nan(bot[e], y);
      }
    }
    uint32_t other = 0;  // groups of 32: the values' words join half a word of two neighbouring groups
    if constexpr (G == 32)
      other = __shfl_xor_sync(0xffffffffu, (g & 1) ? (word & 0x00ff00ffu) << 8 : (word & 0xff00ff00u) >> 8, 4);
    if (!live) continue;
    const int off = (int)(pos & (c.page_size - 1)), t = off & 15;
    uint8_t* blk = base + (int64_t)(off >> 4) * Geo::kBytes;
    if (keys) {
      reinterpret_cast<uint32_t*>(blk + t * Geo::kRow)[Geo::k_word(w)] = word;
    } else {
      int at;
      if constexpr (G == 32) {
        word = (g & 1) ? (word & 0xff00ff00u) | other : (word & 0x00ff00ffu) | other;
        at = (2 * (w % 4) + (g & 1)) * (D / 64) + g / 2;
      } else {
        at = Geo::v_word(w);
      }
      reinterpret_cast<uint32_t*>(blk + Geo::kVOff + kv_v_row(t) * Geo::kRow)[at ^ kv_v_flip<D>(t)] = word;
    }
    if (8 * w % G == 0)
      reinterpret_cast<uint32_t*>(blk + (keys ? Geo::kKPar : Geo::kVPar) + t * Geo::kParRow)[g] =
          (uint32_t)sb | (uint32_t)cb << 16;
  }
  if (!c.bounds) return;
  if (keys) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) {
        top[e] = max_nan(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
        bot[e] = min_nan(bot[e], __shfl_xor_sync(0xffffffffu, bot[e], o));
      }
      if (lane < kLanes) {
        red[(warp * 2) * D + 8 * w + e] = top[e];
        red[(warp * 2 + 1) * D + 8 * w + e] = bot[e];
      }
    }
  }
  __syncthreads();
  uint16_t* ends = c.bounds + (pid * c.heads + h) * (2 * D);
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
    float y = red[i];
    for (int ww = 1; ww < half; ++ww) y = i < D ? max_nan(y, red[ww * 2 * D + i]) : min_nan(y, red[ww * 2 * D + i]);
    if (begin > (j << c.page_shift)) {  // the page held tokens before
      const float z = KvType<T>::to_f(ends[i]);
      y = i < D ? max_nan(y, z) : min_nan(y, z);
    }
    ends[i] = KvType<T>::from_f(y);
  }
}

// One warp per (sequence, block of 16 positions, head): a lane turns one code
// word into eight channels, 16 bytes.
template <typename T, int D, int G>
__global__ void __launch_bounds__(256) kv_read_kernel(KvView c, KvBatch b, uint16_t* __restrict__ k, KvRows ks,
                                                      uint16_t* __restrict__ v, KvRows vs, int blocks_per_seq) {
  using Geo = KvGeom<D, G>;
  constexpr int kWords = D / 8, kTok = 32 / kWords;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int h = (int)(unit % c.heads);
  const int64_t u = unit / c.heads;
  if (u >= (int64_t)b.batch * blocks_per_seq) return;
  const int s = (int)(u / blocks_per_seq);
  const KvSeq q = kv_seq(b, s);
  const int64_t first = (int64_t)q.len - q.rows;
  const int64_t blk16 = (first >> 4) + u % blocks_per_seq;  // the floor of a negative position too
  const int64_t begin = max(first, blk16 << 4), end = min((int64_t)q.len, (blk16 + 1) << 4);
  if (begin >= end) return;
  const uint8_t* blk = nullptr;  // rows that are in no page read as zero
  const int64_t p16 = blk16 << 4;
  if (p16 >= 0 && p16 < kv_capacity(c, b)) {
    const int64_t pid = kv_page(c, b, s, (int)(p16 >> c.page_shift));
    if (pid >= 0)
      blk = c.pages + pid * c.page_stride + h * c.head_stride +
            ((p16 & (c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
  }
  uint16_t* ko = k + kv_row_offset(b, ks, s, q.row0, 0) + h * ks.head;
  uint16_t* vo = v + kv_row_offset(b, vs, s, q.row0, 0) + h * vs.head;
  const int w = lane % kWords, g = 8 * w / G;
#pragma unroll
  for (int i = 0; i < 16 / kTok; ++i) {
    const int t = i * kTok + lane / kWords;
    const int64_t pos = p16 + t;
    if (pos < begin || pos >= end) continue;
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (blk) {
      const uint32_t kw = reinterpret_cast<const uint32_t*>(blk + t * Geo::kRow)[Geo::k_word(w)];
      const uint32_t vw = kv_v_codes<D, G>(
          reinterpret_cast<const uint32_t*>(blk + Geo::kVOff + kv_v_row(t) * Geo::kRow), w, kv_v_flip<D>(t));
      const uint32_t kp = reinterpret_cast<const uint32_t*>(blk + Geo::kKPar + t * Geo::kParRow)[g];
      const uint32_t vp = reinterpret_cast<const uint32_t*>(blk + Geo::kVPar + t * Geo::kParRow)[g];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t word = m ? vw : kw, par = m ? vp : kp;
        const float sf = KvType<T>::lo(par), cf = KvType<T>::hi(par);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = KvType<T>::pack(fmaf(sf, kv_code(word, 2 * e), cf), fmaf(sf, kv_code(word, 2 * e + 1), cf));
        out[m] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    *reinterpret_cast<uint4*>(ko + (pos - first) * ks.row + 8 * w) = out[0];
    *reinterpret_cast<uint4*>(vo + (pos - first) * vs.row + 8 * w) = out[1];
  }
}

}  // namespace

cudaError_t moe::kv_append(const Kv& kv, const KvView& c, const KvBatch& b, const uint16_t* k, const KvRows& ks,
                           const uint16_t* v, const KvRows& vs, cudaStream_t s) {
  const int per_seq = (int)(((int64_t)b.max_new + c.page_size - 2) / c.page_size) + 1;
  const int64_t ctas = (int64_t)b.batch * per_seq * c.heads;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int half = b.max_new == 1 ? 1 : 4;  // key warps
  cudaError_t e = cudaSuccess;
  KV_DISPATCH(kv.d, {
    kv_append_kernel<T, D, G><<<(unsigned)ctas, half * 64, half * 2 * D * sizeof(float), s>>>(c, b, k, ks, v, vs, per_seq);
    e = cudaGetLastError();
  });
  return e;
}

cudaError_t moe::kv_read(const Kv& kv, const KvView& c, const KvBatch& b, uint16_t* k, const KvRows& ks, uint16_t* v,
                         const KvRows& vs, cudaStream_t s) {
  const int per_seq = (int)(((int64_t)b.max_new + 14) / 16) + 1;
  const int64_t warps = (int64_t)b.batch * per_seq * c.heads;
  if (warps / 8 + 1 > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV_DISPATCH(kv.d, {
    kv_read_kernel<T, D, G><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(c, b, k, ks, v, vs, per_seq);
    e = cudaGetLastError();
  });
  return e;
}
