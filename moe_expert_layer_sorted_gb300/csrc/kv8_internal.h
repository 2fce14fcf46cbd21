// The 8-bit key/value cache's handle and the launchers of its kernels.
#pragma once

#include "kv8_common.cuh"
#include "kv_internal.h"

namespace moe {

struct Kv8 {
  moe_kv8_desc d{};
  int sms = 0;
  int64_t block_bytes = 0, head_bytes = 0, page_bytes = 0, layer_bytes = 0, mass_layer = 0;  // mass_layer: elements
  // workspace: partial results of attention items that are cut between CTAs, or of tokens' weights; counters of
  // the former, zero between calls; with mass, references, sums and scores of rows whose weights are counted
  uint8_t* ws = nullptr;
  static constexpr size_t kPartsBytes = size_t(24) << 20;
  static constexpr size_t kFewPartsBytes = size_t(8) << 20;  // of single tokens, and of weights
  static constexpr int64_t kFewRefs = (kPartsBytes - kFewPartsBytes) / sizeof(float2);
  float2* few_refs() const { return reinterpret_cast<float2*>(ws + kFewPartsBytes); }
  static constexpr int kCounters = 1024;
  static constexpr size_t kCounterBytes = kCounters * sizeof(unsigned);
  static constexpr size_t kScoreBytes = size_t(128) << 20;
  static constexpr int kScoreSeqs = 1 << 18;  // sequences whose scores are kept
  size_t workspace() const { return kPartsBytes + kCounterBytes + (d.mass ? kScoreBytes + kScoreSeqs * sizeof(int) : 0); }
  float* scores() const { return reinterpret_cast<float*>(ws + kPartsBytes + kCounterBytes); }
  int* score_bases() const { return reinterpret_cast<int*>(ws + kPartsBytes + kCounterBytes + kScoreBytes); }
  float* parts() const { return reinterpret_cast<float*>(ws); }
  unsigned* counters() const { return reinterpret_cast<unsigned*>(ws + kPartsBytes); }
  volatile uint32_t* err_host = nullptr;  // mapped pinned word: set by a kernel whose bounded wait gave up
  uint32_t* err_dev = nullptr;
  bool fail_next = false;         // test hook: a wait of the next attention runs out
  cudaEvent_t ev_done = nullptr;  // end of the last call that used the workspace
  unsigned long long last_stream = 0;  // its identity
  bool have_last = false;
  // of 2, 3, .. CTAs, as many as run at once (kv8_evict.cu), -1: not asked yet
  mutable int move_clusters[17] = {-1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1};
  std::atomic<int> busy{0};
  std::string last_error;
};

struct Kv8EvictArgs {
  KvView c;
  KvBatch b;      // max_new, rows and starts are not used
  float* mass;    // the layer's
  int budget, first, last;
  int32_t* kept;  // [batch][heads][budget]
};

// mass: the layer's, or nullptr
cudaError_t kv8_append(const Kv8& kv, const KvView& c, const KvBatch& b, const uint16_t* k, const KvRows& ks,
                       const uint16_t* v, const KvRows& vs, float* mass, cudaStream_t s);
cudaError_t kv8_read(const Kv8& kv, const KvView& c, const KvBatch& b, uint16_t* k, const KvRows& ks, uint16_t* v,
                     const KvRows& vs, cudaStream_t s);
// Columns (row, query head) of a kv head that are few.
constexpr int kKv8Columns = 32;
// Prompts: rows whose scores (log2 units) are as large as this round them before the reference is taken off, in the attention
// and in the weights made from its keys again, since there a weight is not the same with and without; below, what is added to
// a score (log2 of a step or a sum, less the reference) may be one number, off by 2^-16.
constexpr float kKv8Coarse = 256.0f;
// What an attention whose weights are counted leaves for that.
// Of each row and query head (numbered as lse is) the reference of its weights, log2 units, and 1 over their sum, of the
// first refs_limit that there is room for.  (In lse, one fp32 in natural units, a sum is lost beside a large reference.)
// Of the single-token kernel its scores too, log2 units, -infinity where not seen.  They lie in the line of rounds
// that its work is cut into (kv_rounds.cuh), so that only tokens that are there take room: [round][128 tokens][width], a
// round being one of a sequence's kv head and column tile.  base[sequence]: its first round, or -1 where there was no
// room for it (not written for a sequence without rounds).
struct Kv8Scores {
  float2* refs;  // nullptr: nothing of this is wanted
  int64_t refs_limit;
  float* to;
  int* base;   // nullptr: scores are not wanted
  int width;   // columns of a tile that are kept, a multiple of four
  int ctiles;  // column tiles of a kv head
  int limit;   // rounds that there is room for
};
// Attention of few rows.
cudaError_t kv8_decode_bf16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s);
cudaError_t kv8_decode_f16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s);
// Attention of prompts.
cudaError_t kv8_prompt_bf16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s);
cudaError_t kv8_prompt_f16(Kv8& kv, const KvAttnArgs& a, const Kv8Scores& scores, cudaStream_t s);
// mass: nullptr, or the layer's, to which the weights of the tokens are added (lse is then given).
cudaError_t kv8_attention(Kv8& kv, const KvAttnArgs& a, float* mass, cudaStream_t s);
// The weights of an attention whose lse is written; scores: what it left.
cudaError_t kv8_weigh(Kv8& kv, const KvAttnArgs& a, float* mass, const Kv8Scores& scores, cudaStream_t s);
cudaError_t kv8_evict(const Kv8& kv, const Kv8EvictArgs& a, cudaStream_t s);

// Calls f with (T, D) of the cache as compile-time constants.
#define KV8_DISPATCH(desc, ...)                                     \
  do {                                                              \
    auto run_ = [&](auto tag_) {                                    \
      using T = decltype(tag_);                                     \
      if ((desc).head_dim == 64) { constexpr int D = 64; __VA_ARGS__ } \
      else { constexpr int D = 128; __VA_ARGS__ }                   \
    };                                                              \
    if ((desc).dtype == MOE_KV_BF16) run_(__nv_bfloat16());         \
    else run_(__half());                                            \
  } while (0)

}  // namespace moe
