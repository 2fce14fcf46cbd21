// Writing and reading the 8-bit key/value cache.
//
// The 16 tokens of a block share a step: s = rn(max |x| / 127) in fp32 over the block's new rows
// (those without an infinity or a NaN), or the step that its older tokens have where that is larger;
//     u = x / s to the nearest whole number, ties to even, -127..127,
// and where the older tokens' step grew, u_old s_old / s likewise.  Both are the quotients themselves, rounded
// once (kv8_common.cuh).
#include "kv8_internal.h"

using namespace moe;

namespace {

template <typename T>
struct Limits;
template <>
struct Limits<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80u;
};
template <>
struct Limits<__half> {
  static constexpr uint32_t kInf = 0x7c00u;
};

// 1 / s for the quotients, and the power of two that both sides of them are multiplied with first.
struct Step {
  float s, up, inv;
  __device__ __forceinline__ explicit Step(float step) {
    up = kv8_lift(step);
    s = step * up;
    inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
  }
};

// x / s of eight elements as codes u + 128 in two words.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], const Step& st) {
  uint64_t y[4];
  uint32_t near = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = kv8_round2(kv8_two(x[2 * e], x[2 * e + 1]), kv8_two(st.inv, st.inv), near);
  uint32_t lo = kv8_word(y[0], y[1]), hi = kv8_word(y[2], y[3]);
  while (near) {
    const int bit = 31 - __clz(near), e = 7 - bit;
    near ^= 1u << bit;
    float v = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) v = e == i ? x[i] : v;
    const uint32_t code = (uint32_t)((int)kv8_settle(v, 1.0f, st.s, v * st.inv) + 128), at = 8 * (e & 3);
    if (e < 4) lo = (lo & ~(0xffu << at)) | code << at;
    else hi = (hi & ~(0xffu << at)) | code << at;
  }
  return make_uint2(lo, hi);
}

// Codes of two words of the step s, turned to `to` >= s.
__device__ __forceinline__ uint2 turn8(uint2 w, float s, float to) {
  const float up = kv8_lift(to);
  s *= up;
  to *= up;
  const float ratio = __fdiv_rn(s, to);
  uint32_t near = 0;
  uint32_t lo = kv8_turn(w.x, ratio, near), hi = kv8_turn(w.y, ratio, near);
  while (near) {
    const int bit = 31 - __clz(near), e = 7 - bit;
    near ^= 1u << bit;
    const uint32_t code = kv8_settle_byte(e < 4 ? w.x : w.y, e & 3, s, to, ratio), at = 8 * (e & 3);
    if (e < 4) lo = (lo & ~(0xffu << at)) | code << at;
    else hi = (hi & ~(0xffu << at)) | code << at;
  }
  return make_uint2(lo, hi);
}

// One warp per (sequence, block that its rows touch, head, keys or values), since the block's step
// needs all of its rows: they stay in registers between the maximum and the codes.  D / 8 lanes hold a
// row, eight channels each.
//
// 8,192 rows of 8 heads of 128 channels (fp16, 33.6 MB read, 16.8 MB of pages written): 16.6 us, 3.0 TB/s; bound
// by instructions and by 2.3 waves of CTAs (64 registers for a fourth CTA per SM 18.5 us, CTAs of 128 or 64 threads
// 17.1; without what settles halves 14.3).  256 sequences of a row each: 8.3 us, the chain length -> page -> step and
// row -> step -> codes.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_append_kernel(KvView c, KvBatch b, const uint16_t* __restrict__ k, KvRows ks,
                                                         const uint16_t* __restrict__ v, KvRows vs,
                                                         float* __restrict__ mass, int blocks_per_seq) {
  using Geo = Kv8Geom<D>;
  constexpr int L = D / 8, kTok = 32 / L, kPasses = 16 / kTok;  // lanes per row, rows per pass
  const int lane = threadIdx.x & 31, w = lane % L, sub = lane / L;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int side = (int)(unit & 1);
  const int h = (int)((unit >> 1) % c.heads);
  const int64_t n = (unit >> 1) / c.heads;
  if (n >= (int64_t)b.batch * blocks_per_seq) return;
  const int s = (int)(n / blocks_per_seq);
  const KvSeq q = kv_seq(b, s);
  const int64_t first = (int64_t)q.len - q.rows;  // position of row 0 (negative: rows before the sequence, dropped)
  const int64_t p0 = first > 0 ? first : 0;
  const int64_t p16 = ((p0 >> 4) + n % blocks_per_seq) << 4;
  const int64_t end64 = min(min((int64_t)q.len, (int64_t)kv_capacity(c, b)), p16 + 16);
  if (q.rows == 0 || max(p0, p16) >= end64) return;
  const int64_t pid = kv_page(c, b, s, (int)(p16 >> c.page_shift));
  if (pid < 0) return;
  const int off = (int)(p16 & (c.page_size - 1));
  uint8_t* blk = c.pages + pid * c.page_stride + h * c.head_stride + (off >> 4) * (int64_t)Geo::kBytes;
  const int begin = (int)(max(p0, p16) - p16), end = (int)(end64 - p16);  // the block's new tokens; those below `begin` are older
  Kv8Params* par = reinterpret_cast<Kv8Params*>(blk + Geo::kParams);
  float s_old = 0.0f;
  uint32_t marks = 0;
  if (begin > 0) {
    s_old = par->step[side];
    marks = par->mark[side] & ((1u << begin) - 1u);
  }
  const KvRows st = side ? vs : ks;
  const uint16_t* src = (side ? v : k) + kv_row_offset(b, st, s, q.row0, 0) + h * st.head + (p16 - first) * st.row + 8 * w;
  // the rows, older and missing ones as zeros, and the largest magnitude in them
  uint4 raw[kPasses];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kTok + sub;
    raw[i] = t >= begin && t < end ? __ldg(reinterpret_cast<const uint4*>(src + t * st.row)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                 __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)));
  top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
  if (top >= Limits<T>::kInf) {  // some rows are not finite: they are marked and enter as zeros
    top = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint32_t m = __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                            __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
      m = max(m >> 16, m & 0xffffu);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool bad = m >= Limits<T>::kInf;
      const uint32_t votes = __ballot_sync(0xffffffffu, bad && w == 0);
#pragma unroll
      for (int y = 0; y < kTok; ++y) marks |= ((votes >> (y * L)) & 1u) << (i * kTok + y);
      if (bad) raw[i] = make_uint4(0, 0, 0, 0);
      else top = max(top, m);
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const float fresh = __fdiv_rn(KvType<T>::to_f((uint16_t)top), 127.0f);
  const float step = fmaxf(fresh, s_old);
  const bool turn = begin > 0 && step > s_old;  // older codes change
  const Step q8(step);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kTok + sub;
    if (!turn && ((i + 1) * kTok <= begin || i * kTok >= end)) continue;  // nothing of this pass changes
    if (i * kTok >= end) continue;
    const uint32_t r4[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = KvType<T>::lo(r4[e]);
      x[2 * e + 1] = KvType<T>::hi(r4[e]);
    }
    if (q8.up != 1.0f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= q8.up;
    }
    uint2 code = quantise8(x, q8);
    if (side == 0) {
      uint2* dst = reinterpret_cast<uint2*>(blk + t * D + Geo::k_piece(t, w >> 1) * 16 + (w & 1) * 8);
      if (t < begin) {
        if (!turn) continue;
        code = turn8(*dst, s_old, step);
      }
      if (t < end) *dst = code;
    } else {
      // the pair's two tokens sit L lanes apart: the lane of the even one takes the lower four channels of both
      const bool odd = t & 1;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? code.x : code.y, L);
      const uint32_t even = odd ? got : code.x, uneven = odd ? code.y : got;
      uint2 both = make_uint2(__byte_perm(even, uneven, 0x5140), __byte_perm(even, uneven, 0x7362));
      const int pair = t >> 1;
      uint2* dst = reinterpret_cast<uint2*>(blk + Geo::kVOff + pair * 2 * D + Geo::v_piece(pair, w) * 16 + (odd ? 8 : 0));
      const int t0 = t & ~1;
      if (t0 < begin) {  // the first token of the pair, or both, are older
        if (t0 + 1 < begin && !turn) continue;
        uint2 old = *dst;
        if (turn) old = turn8(old, s_old, step);
        const uint32_t keep = t0 + 1 < begin ? 0xffffffffu : 0x00ff00ffu;
        both = make_uint2((old.x & keep) | (both.x & ~keep), (old.y & keep) | (both.y & ~keep));
      }
      *dst = both;  // a token past the end: 0
    }
  }
  __syncwarp();
  if (lane == 0) {
    par->step[side] = step;
    par->mark[side] = (uint16_t)marks;
    if (side == 0) par->zero = 0;
  }
  if (mass && side == 0 && lane >= begin && lane < end) mass[(pid * c.heads + h) * c.page_size + off + lane] = 0.0f;
}

// One warp per (sequence, block of 16 positions, head): a lane takes 16 bytes of codes at a time, 16
// channels of a token's keys, or 8 of the values of a pair of tokens.  Bound by the memory: 32 x 4,096 rows of 8
// heads of 128 channels 116 us, 6.9 TB/s read and written; 8,192 rows 12.3 us, 4.1 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(KvView c, KvBatch b, uint16_t* __restrict__ k, KvRows ks,
                                                       uint16_t* __restrict__ v, KvRows vs, int blocks_per_seq) {
  using Geo = Kv8Geom<D>;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int h = (int)(unit % c.heads);
  const int64_t u = unit / c.heads;
  if (u >= (int64_t)b.batch * blocks_per_seq) return;
  const int s = (int)(u / blocks_per_seq);
  const KvSeq q = kv_seq(b, s);
  const int64_t first = (int64_t)q.len - q.rows;
  const int64_t p16 = ((first >> 4) + u % blocks_per_seq) << 4;  // the floor of a negative position too
  const int begin = (int)(max(first, p16) - p16), end = (int)(min((int64_t)q.len, p16 + 16) - p16);
  if (begin >= end) return;
  const uint8_t* blk = nullptr;  // rows that are in no page read as zero
  if (p16 >= 0 && p16 < kv_capacity(c, b)) {
    const int64_t pid = kv_page(c, b, s, (int)(p16 >> c.page_shift));
    if (pid >= 0)
      blk = c.pages + pid * c.page_stride + h * c.head_stride + ((p16 & (c.page_size - 1)) >> 4) * (int64_t)Geo::kBytes;
  }
  uint16_t* ko = k + kv_row_offset(b, ks, s, q.row0, 0) + h * ks.head + (p16 - first) * ks.row;
  uint16_t* vo = v + kv_row_offset(b, vs, s, q.row0, 0) + h * vs.head + (p16 - first) * vs.row;
  Kv8Params par{};
  if (blk) {
    const uint4 x = *reinterpret_cast<const uint4*>(blk + Geo::kParams);
    par.step[0] = __uint_as_float(x.x);
    par.step[1] = __uint_as_float(x.y);
    par.mark[0] = (uint16_t)x.z;
    par.mark[1] = (uint16_t)(x.z >> 16);
  }
  constexpr int kLoads = 16 * D / 16 / 32;  // of 16 bytes a lane, keys and values each
  uint4 kw[kLoads], vw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int x = i * 32 + lane, t = x / (D / 16), pair = x / (D / 8);
    kw[i] = vw[i] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
    if (blk) {
      kw[i] = *reinterpret_cast<const uint4*>(blk + t * D + Geo::k_piece(t, x % (D / 16)) * 16);
      vw[i] = *reinterpret_cast<const uint4*>(blk + Geo::kVOff + pair * 2 * D + Geo::v_piece(pair, x % (D / 8)) * 16);
    }
  }
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int x = i * 32 + lane, t = x / (D / 16), t0 = x / (D / 8) * 2;
    {
      const float step = (par.mark[0] >> t) & 1 ? nan : par.step[0];
      const uint32_t in[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = KvType<T>::pack(kv8_code(in[e / 2], 2 * (e % 2)) * step, kv8_code(in[e / 2], 2 * (e % 2) + 1) * step);
      uint4* dst = reinterpret_cast<uint4*>(ko + t * ks.row + x % (D / 16) * 16);
      if (t >= begin && t < end) {
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int tv = t0 + y;
      const float step = (par.mark[1] >> tv) & 1 ? nan : par.step[1];
      const uint32_t in[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = KvType<T>::pack(kv8_code(in[e], y) * step, kv8_code(in[e], 2 + y) * step);
      if (tv >= begin && tv < end)
        *reinterpret_cast<uint4*>(vo + tv * vs.row + x % (D / 8) * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Blocks that `rows` consecutive positions can touch.
int blocks_of(int rows) { return (int)(((int64_t)rows + 14) / 16) + 1; }

}  // namespace

cudaError_t moe::kv8_append(const Kv8& kv, const KvView& c, const KvBatch& b, const uint16_t* k, const KvRows& ks,
                            const uint16_t* v, const KvRows& vs, float* mass, cudaStream_t s) {
  const int per_seq = blocks_of(b.max_new);
  const int64_t warps = (int64_t)b.batch * per_seq * c.heads * 2;
  if (warps / 8 + 1 > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV8_DISPATCH(kv.d, {
    kv8_append_kernel<T, D><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(c, b, k, ks, v, vs, mass, per_seq);
    e = cudaGetLastError();
  });
  return e;
}

cudaError_t moe::kv8_read(const Kv8& kv, const KvView& c, const KvBatch& b, uint16_t* k, const KvRows& ks, uint16_t* v,
                          const KvRows& vs, cudaStream_t s) {
  const int per_seq = blocks_of(b.max_new);
  const int64_t warps = (int64_t)b.batch * per_seq * c.heads;
  if (warps / 8 + 1 > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  KV8_DISPATCH(kv.d, {
    kv8_read_kernel<T, D><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(c, b, k, ks, v, vs, per_seq);
    e = cudaGetLastError();
  });
  return e;
}
