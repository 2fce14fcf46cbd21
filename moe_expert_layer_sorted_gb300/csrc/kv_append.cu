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

// Larger halves of two pairs of the cache's type, NaN where either is.
template <typename T>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
constexpr uint32_t kNegate = 0x80008000u;

// x / 15 rounded to nearest: the product with the reciprocal and Markstein's correction of it by
// its remainder.  Equal to the division for every finite 16-bit x (tests/test_kv_division.py).
__device__ __forceinline__ float over15(float x) {
  constexpr float kInv = 1.0f / 15.0f;
  const float q = __fmul_rn(x, kInv);
  return fmaf(fmaf(-15.0f, q, x), kInv, q);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float reciprocal(float x) {  // within an ulp; infinite for a subnormal
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// One CTA per (sequence, page it writes to, head), the first half of its warps
// on the keys and the second on the values; D / 8 lanes hold a row, eight
// channels each, so that a lane makes one code word.  The page is the CTA's
// own, so its bounds need no atomics.
//
// Bound by instructions: about 260 per warp and 256 elements.  8,192 rows of 8
// heads of 128 channels (fp16, 33.6 MB read, 9.4 MB of pages written) take 23 us,
// 1.9 TB/s, at 71 % of the issue slots; half the warps per CTA (36.1 us with the
// read back, against 35.3), registers for a fifth CTA per SM (37.7) or both (35.5)
// win nothing.  A single row per sequence takes one warp for the keys and one for
// the values: 256 sequences, written and read back, 11.4 us, two launches' latency.
template <typename T, int D, int G>
__global__ void kv_append_kernel(KvView c, KvBatch b, const uint16_t* __restrict__ k, KvRows ks,
                                 const uint16_t* __restrict__ v, KvRows vs, int pages_per_seq) {
  using Geo = KvGeom<D, G>;
  constexpr int kLanes = D / 8, kTok = 32 / kLanes;  // lanes per row, rows per warp
  extern __shared__ uint32_t red[];                  // [key warps][max, -min][D / 2] pairs
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
  // largest stored keys, and largest of the negated ones, as pairs of the cache's type: what is
  // rounded after the maximum is the maximum of the rounded
  const uint32_t least = (uint32_t)KvType<T>::from_f(-__int_as_float(0x7f800000)) * 0x10001u;
  uint32_t top[4], bot[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) top[e] = bot[e] = least;
  const int step = half * kTok;
  // offsets in the page
  const int p_end = (int)(end - (j << c.page_shift));
  int off = (int)(begin - (j << c.page_shift)) + (warp % half) * kTok + lane / kLanes;
  const uint16_t* row = src + ((j << c.page_shift) + off - first) * stride + 8 * w;
  uint4 next = make_uint4(0, 0, 0, 0);
  if (off < p_end) next = *reinterpret_cast<const uint4*>(row);
  for (; __any_sync(0xffffffffu, off < p_end); off += step) {  // the next row arrives while this one is turned
    const bool live = off < p_end;
    const uint4 raw = next;
    row += step * stride;
    if (off + step < p_end) next = *reinterpret_cast<const uint4*>(row);
    const uint32_t r4[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = KvType<T>::lo(r4[i]);
      x[2 * i + 1] = KvType<T>::hi(r4[i]);
    }
    // the group's largest element and the largest of its negated ones, exact in 16 bits
    uint32_t hl = max_pair<T>(max_pair<T>(r4[0], r4[1]), max_pair<T>(r4[2], r4[3]));
    const uint32_t neg = max_pair<T>(max_pair<T>(r4[0] ^ kNegate, r4[1] ^ kNegate), max_pair<T>(r4[2] ^ kNegate, r4[3] ^ kNegate));
    hl = max_pair<T>(__byte_perm(hl, neg, 0x5410), __byte_perm(hl, neg, 0x7632));
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) hl = max_pair<T>(hl, __shfl_xor_sync(0xffffffffu, hl, o));
    const float hi = KvType<T>::lo(hl), lo = -KvType<T>::hi(hl);
    const bool bad = !(fabsf(hi) < __int_as_float(0x7f800000) && fabsf(lo) < __int_as_float(0x7f800000));
    uint16_t sb = KvType<T>::from_f(__fsub_rn(over15(hi), over15(lo)));
    uint16_t cb = KvType<T>::from_f(fmaf(8.0f, KvType<T>::to_f(sb), lo));  // 8 s is exact
    if (bad) {
      sb = 0;
      cb = 0x7fff;  // NaN in both types
    }
    const float sf = KvType<T>::to_f(sb), cf = KvType<T>::to_f(cb);
    const float inv = sf > 0.0f ? reciprocal(sf) : 0.0f;
    // rint of the quotients: (x - c) / s as a product with the reciprocal, rounded to a whole
    // number by an addition of 1.5 2^23, is right for all but quotients that near a half (the
    // product is within 2^-18 of one that is not cut to -8 or 7); those rows are divided.
    constexpr float kWhole = 12582912.0f;
    float q[8], worst = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float num = __fsub_rn(x[e], cf);
      q[e] = __fsub_rn(fmaf(num, inv, kWhole), kWhole);
      worst = max_nan(worst, fabsf(fmaf(num, inv, -q[e])));
    }
    if (!(worst < 0.4999f) && sf > 0.0f) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const float num = __fsub_rn(e < 4 ? (e < 2 ? (e ? x[1] : x[0]) : (e == 2 ? x[2] : x[3]))
                                          : (e < 6 ? (e == 4 ? x[4] : x[5]) : (e == 6 ? x[6] : x[7])), cf);
        const float y = rintf(__fdiv_rn(num, sf));
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = i == e ? y : q[i];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = fminf(fmaxf(q[e], -8.0f), 7.0f);
    // the word's half-words, each a whole number below 2^16 in fp32's low bits
    auto half_word = [&](int e) {
      return __float_as_uint(fmaf(q[e + 6], 4096.0f, fmaf(q[e + 4], 256.0f, fmaf(q[e + 2], 16.0f, q[e]))) + (kWhole + 34952.0f));
    };
    uint32_t word = __byte_perm(half_word(0), half_word(1), 0x5410);
    if (bad) word = 0x88888888u;
    if (live && keys) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t y = KvType<T>::pack(fmaf(sf, q[2 * e], cf), fmaf(sf, q[2 * e + 1], cf));  // s q is exact
        top[e] = max_pair<T>(top[e], y);
        bot[e] = max_pair<T>(bot[e], y ^ kNegate);
      }
    }
    uint32_t other = 0;  // groups of 32: the values' words join half a word of two neighbouring groups
    if constexpr (G == 32)
      other = __shfl_xor_sync(0xffffffffu, (g & 1) ? (word & 0x00ff00ffu) << 8 : (word & 0xff00ff00u) >> 8, 4);
    if (!live) continue;
    const int t = off & 15;
    uint8_t* blk = base + (off >> 4) * Geo::kBytes;
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
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) {
        top[e] = max_pair<T>(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
        bot[e] = max_pair<T>(bot[e], __shfl_xor_sync(0xffffffffu, bot[e], o));
      }
      if (lane < kLanes) {
        red[warp * D + 4 * w + e] = top[e];
        red[warp * D + D / 2 + 4 * w + e] = bot[e];
      }
    }
  }
  __syncthreads();
  uint32_t* ends = reinterpret_cast<uint32_t*>(c.bounds + (pid * c.heads + h) * (2 * D));  // [max, min][D / 2] pairs
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    const uint32_t flip = i < D / 2 ? 0u : kNegate;  // minima as negated maxima
    uint32_t y = red[i];
    for (int ww = 1; ww < half; ++ww) y = max_pair<T>(y, red[ww * D + i]);
    if (begin > (j << c.page_shift)) y = max_pair<T>(y, ends[i] ^ flip);  // the page held tokens before
    ends[i] = y ^ flip;
  }
}

// One warp per (sequence, block of 16 positions, head): a lane turns one code
// word into eight channels, 16 bytes.  Bound by the memory from a few thousand
// rows on: 131,072 rows of 8 heads of 128 channels 127 us, 5.4 TB/s read and
// written; 8,192 rows 12 us, 3.5 TB/s.
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
  // key warps: as few as the rows of a page keep busy.  Measured with 1 / 2 / 4 (8 heads of 128
  // channels, us): 256 sequences of 1 row 5.2 / 7.0 / -, of 2 rows 7.6 / 8.7 / 14.5, of 4 rows
  // 9.9 / 9.9 / 15.7, of 8 rows 14.4 / 13.2 / 17.9, of 64 rows 69 / 60 / 64; 1 sequence of 4 rows
  // 4.5 / 3.2 / 3.5, of 8 rows 6.2 / 4.2 / 3.6, of 64 rows 14.7 / 11.9 / 8.8.
  const int half = b.max_new == 1 ? 1 : b.max_new <= 4 ? 2 : 4;
  cudaError_t e = cudaSuccess;
  KV_DISPATCH(kv.d, {
    kv_append_kernel<T, D, G><<<(unsigned)ctas, half * 64, half * D * sizeof(uint32_t), s>>>(c, b, k, ks, v, vs, per_seq);
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
