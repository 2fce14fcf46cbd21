// Device view of the 4-bit key/value cache and of a batch of sequences, and
// the placement of channels in its code words (included by the kv_*.cu files).
//
// A page holds, per kv head, P / 16 blocks of 16 tokens.  A block is one
// contiguous run of bytes,
//     K codes [16][D/2] | V codes [16][D/2] | K params [16][D/G][2] | V params [16][D/G][2]
// (params: step s and centre c in the cache's type, a stored value being
// c + s (u - 8)), so that any run of blocks of a page and head is one bulk
// copy.  The order of the codes inside a row is the order in which the
// attention over single tokens wants its matrix operands (kv_decode.cuh):
//   - K: a row is four quarters, one per lane of a quad, and a quarter holds
//     the matching quarter of every group, so that 16 bytes of a lane feed
//     whole k-steps of one group after the other;
//   - V: a row is eight pieces, one per lane octet, and a piece holds the
//     matching eighth of every group; rows are stored in the order
//     (t & 8) | (t & 1) << 2 | (t >> 1) & 3 with the two halves of the pieces
//     exchanged where t & 4, so that the 16 lanes of a half warp (four tokens
//     by four pieces) hit all 32 banks once.
// Eight channels 0..7 of a word take its nibbles 0 4 1 5 2 6 3 7: one mask
// gives the channel pair (2i, 2i + 1) in the low and high half-words.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"

namespace moe {

constexpr int kKvBlock = 16;  // tokens per block

struct KvView {  // one layer of the cache
  uint8_t* pages;
  uint16_t* bounds;  // [page][head][max, min][D] or nullptr
  int64_t page_stride, head_stride;  // bytes
  int64_t num_pages;
  int page_size, page_shift, heads;
};

struct KvBatch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;  // nullptr: max_new rows per sequence
  int64_t table_stride, rows;
  int batch, table_pages, max_new;
};

struct KvRows {  // a 16-bit tensor of rows by heads: element strides
  int64_t batch, row, head;
};

struct KvSeq {  // one sequence of a batch
  int64_t row0;  // its first row (ragged: in the whole tensor; uniform: 0, see kv_row_offset)
  int rows;      // its rows, the last of its tokens
  int len;       // its tokens
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int s) {
  KvSeq q;
  q.len = max(b.lens[s], 0);
  if (b.starts) {  // out-of-range starts are cut to the tensor's rows
    const int64_t a = min(max((int64_t)b.starts[s], (int64_t)0), b.rows);
    const int64_t e = min(max((int64_t)b.starts[s + 1], a), b.rows);
    q.row0 = a;
    q.rows = (int)min(e - a, (int64_t)b.max_new);
  } else {
    q.row0 = 0;
    q.rows = b.max_new;
  }
  return q;
}
__device__ __forceinline__ int64_t kv_row_offset(const KvBatch& b, const KvRows& r, int s, int64_t row0, int i) {
  return (b.starts ? row0 * r.row : (int64_t)s * r.batch) + (int64_t)i * r.row;
}
// Index of a row in per-row outputs laid out densely (lse, page lists).
__device__ __forceinline__ int64_t kv_row_index(const KvBatch& b, int s, int64_t row0, int i) {
  return (b.starts ? row0 : (int64_t)s * b.max_new) + i;
}
// Tokens the table can hold: positions beyond are neither written nor read.
__device__ __forceinline__ int kv_capacity(const KvView& c, const KvBatch& b) {
  return (int)min((int64_t)b.table_pages << c.page_shift, (int64_t)0x7ffff000);  // a block past it still has a position
}
// Page id of a sequence's page j, or -1 where the entry names no page of the pool.
__device__ __forceinline__ int64_t kv_page(const KvView& c, const KvBatch& b, int s, int j) {
  const int32_t id = b.table[(int64_t)s * b.table_stride + j];
  return (uint64_t)(int64_t)id < (uint64_t)c.num_pages ? (int64_t)id : -1;
}

template <int D, int G>
struct KvGeom {
  static_assert(D % G == 0 && G % 32 == 0, "groups of 32, 64 or 128 channels");
  static constexpr int NG = D / G;                   // groups per row
  static constexpr int kRow = D / 2;                 // bytes of a row's codes
  static constexpr int kVOff = kKvBlock * kRow;      // V codes
  static constexpr int kKPar = 2 * kVOff;            // K params
  static constexpr int kParRow = 4 * NG;             // bytes of a row's params
  static constexpr int kVPar = kKPar + kKvBlock * kParRow;
  static constexpr int kBytes = kVPar + kKvBlock * kParRow;
  static_assert(kBytes % 16 == 0, "blocks are bulk-copied");

  // K: word (of D / 8) of the channels 8w .. 8w + 7
  static __device__ __host__ constexpr int k_word(int w) {
    const int g = 8 * w / G, r = 8 * w % G;
    return r / (G / 4) * (D / 32) + g * (G / 32) + r % (G / 4) / 8;
  }
  // V, groups of 64 and 128: word of the channels 8w .. 8w + 7, in piece order
  static __device__ __host__ constexpr int v_word(int w) {
    const int g = 8 * w / G, r = 8 * w % G;
    return r / (G / 8) * (D / 64) + (g * (G / 8) + r % (G / 8)) / 8;
  }
};

__device__ __forceinline__ int kv_v_row(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }
// xor of a V word's index in its row (D / 8 words, half of them D / 16)
template <int D>
__device__ __forceinline__ int kv_v_flip(int t) {
  return ((t >> 2) & 1) * (D / 16);
}

template <typename T>
struct KvType;
template <>
struct KvType<__nv_bfloat16> {
  static __device__ __forceinline__ float to_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t from_f(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
template <>
struct KvType<__half> {
  static __device__ __forceinline__ float to_f(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ uint16_t from_f(float f) { return __half_as_ushort(__float2half_rn(f)); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return to_f((uint16_t)(w & 0xffffu)); }
  static __device__ __forceinline__ float hi(uint32_t w) { return to_f((uint16_t)(w >> 16)); }
};

// The eight codes of a word as (u - 8), in channel order.
__device__ __forceinline__ float kv_code(uint32_t w, int ch) {
  return (float)((int)((w >> (4 * ((ch >> 1) + 4 * (ch & 1)))) & 15u) - 8);
}

// V codes of the channels 8w .. 8w + 7 of a token as one word in the nibble
// order above.  words: the token's V row (D / 8 words), flip: kv_v_flip(token).
template <int D, int G>
__device__ __forceinline__ uint32_t kv_v_codes(const uint32_t* words, int w, int flip) {
  if constexpr (G >= 64) {
    return words[KvGeom<D, G>::v_word(w) ^ flip];
  } else {  // four channels in each of two neighbouring pieces, at nibble pairs 0-1 or 2-3 of the half-words
    const int g = w / 4, q = w % 4;
    const uint32_t a = words[(2 * q * (D / 64) + g / 2) ^ flip], b = words[((2 * q + 1) * (D / 64) + g / 2) ^ flip];
    return (g & 1) ? ((a >> 8) & 0x00ff00ffu) | (b & 0xff00ff00u) : (a & 0x00ff00ffu) | ((b & 0x00ff00ffu) << 8);
  }
}

}  // namespace moe
