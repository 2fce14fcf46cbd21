// The 4-bit key/value cache's handle and the launchers of its kernels.
#pragma once

#include <algorithm>
#include <atomic>
#include <string>

#include "internal.h"
#include "kv_common.cuh"

namespace moe {

struct Kv {
  moe_kv_desc d{};
  int sms = 0;
  int64_t block_bytes = 0, head_bytes = 0, page_bytes = 0, layer_bytes = 0, bounds_layer = 0;  // bounds_layer: elements
  // workspace: the selection's scores; partial results of attention items that are cut
  // between CTAs; their counters, zero between calls
  uint8_t* ws = nullptr;
  static constexpr size_t kScoreBytes = size_t(16) << 20;
  static constexpr size_t kPartsBytes = size_t(24) << 20;
  static constexpr int kCounters = 1024;
  static constexpr size_t kCounterBytes = kCounters * sizeof(unsigned);
  static constexpr size_t kWorkspace = kScoreBytes + kPartsBytes + kCounterBytes;
  float* parts() const { return reinterpret_cast<float*>(ws + kScoreBytes); }
  unsigned* counters() const { return reinterpret_cast<unsigned*>(ws + kScoreBytes + kPartsBytes); }
  volatile uint32_t* err_host = nullptr;  // mapped pinned word: set by a kernel whose bounded wait gave up
  uint32_t* err_dev = nullptr;
  bool fail_next = false;         // test hook: a wait of the next attention runs out
  cudaEvent_t ev_done = nullptr;  // end of the last call that used the workspace
  unsigned long long last_stream = 0;  // its identity
  bool have_last = false;
  std::atomic<int> busy{0};
  std::string last_error;
};

struct KvAttnArgs {
  KvView c;
  KvBatch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // [rows][q_heads] or nullptr
  KvRows qs, os;
  int q_heads;
  float scale;
  int causal;
  const int32_t* sel;  // [rows][heads][budget] page indices, or nullptr: every page
  int budget;
};

struct KvSelectArgs {
  KvView c;
  KvBatch b;
  const uint16_t* q;
  KvRows qs;
  int q_heads, budget, first, last;
  int32_t* out;  // [rows][heads][budget]
};

cudaError_t kv_append(const Kv& kv, const KvView& c, const KvBatch& b, const uint16_t* k, const KvRows& ks,
                      const uint16_t* v, const KvRows& vs, cudaStream_t s);
cudaError_t kv_read(const Kv& kv, const KvView& c, const KvBatch& b, uint16_t* k, const KvRows& ks, uint16_t* v,
                    const KvRows& vs, cudaStream_t s);
// Attention of few rows, or over chosen pages.
cudaError_t kv_decode_bf16(Kv& kv, const KvAttnArgs& a, cudaStream_t s);
cudaError_t kv_decode_f16(Kv& kv, const KvAttnArgs& a, cudaStream_t s);
// Attention of prompts.
cudaError_t kv_prompt_bf16(Kv& kv, const KvAttnArgs& a, cudaStream_t s);
cudaError_t kv_prompt_f16(Kv& kv, const KvAttnArgs& a, cudaStream_t s);
cudaError_t kv_attention(Kv& kv, const KvAttnArgs& a, cudaStream_t s);
cudaError_t kv_select(Kv& kv, const KvSelectArgs& a, cudaStream_t s);

// Rows of at most this many pages are scored and picked by one CTA, without the workspace.
// Measured, one CTA / two kernels (8 heads of 128 channels, us), 1, 16 and 64 rows: of 256 pages
// 8.9 / 10.4, 9.6 / 11.2, 13.3 / 19.0; of 512 pages 13.5 / 10.6, 14.1 / 13.0, 20.2 / 27.8; of 1,024
// pages 22.5 / 10.7, 23.7 / 16.5, 37.3 / 41.7.
constexpr int kKvSelOwn = 512;

// Rounds in shared memory of the decode kernel: 3 to 8, so that two CTAs of eight warps share an SM.
template <int D, int G>
constexpr int kDecStages = 9216 / KvGeom<D, G>::kBytes;

// Calls f with (T, D, G) of the cache as compile-time constants.
#define KV_DISPATCH(desc, ...)                                                            \
  do {                                                                                    \
    auto run_ = [&](auto tag_) {                                                          \
      using T = decltype(tag_);                                                           \
      const int dg_ = (desc).head_dim * 1000 + (desc).group_size;                         \
      if (dg_ == 64032) { constexpr int D = 64, G = 32; __VA_ARGS__ }                     \
      else if (dg_ == 64064) { constexpr int D = 64, G = 64; __VA_ARGS__ }                \
      else if (dg_ == 128032) { constexpr int D = 128, G = 32; __VA_ARGS__ }              \
      else if (dg_ == 128064) { constexpr int D = 128, G = 64; __VA_ARGS__ }              \
      else { constexpr int D = 128, G = 128; __VA_ARGS__ }                                \
    };                                                                                    \
    if ((desc).dtype == MOE_KV_BF16) run_(__nv_bfloat16());                               \
    else run_(__half());                                                                  \
  } while (0)

}  // namespace moe
