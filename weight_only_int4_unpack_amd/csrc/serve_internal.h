// Internal interface between the host side (serve_host.cpp) and the gfx950
// kernels of the operators around the weight products: rotary positions, the
// paged key/value cache, attention of drafted tokens, token scores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a16.h"
#include "w4a16_internal.h"

namespace w4a16 {

// Shared with w4a16_host.cpp: records the calling thread's message and
// returns `st`; and the current device's CU count (DEVICE unless gfx950).
w4a16_status report(w4a16_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
w4a16_status current_device(int* num_cus);

// A paged cache as the kernels see it: page_size = 1 << page_shift.
struct KvView {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int32_t page_shift, heads, dim;
};

// Lanes that hold one head, 8 dims each: the power of two that covers dim.
inline int lanes_per_head(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

struct RopeTableParams {
  double inv_freq[128];
  double amplitude;
  float* table;
  int64_t positions;
  int32_t half;             // rotated dims / 2
};

// One kernel rotates (hkv = 0), writes the cache (hq = 0, table null) or
// does both. Heads of a token are counted q, then k, then v.
struct RopeKvParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  const int64_t* positions;
  const int64_t* slots;
  const float* table;       // null: nothing is rotated
  KvView cache;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  int64_t table_rows;
  int32_t tokens, hq, hkv, dim, rot;
  int32_t interleaved, inverse;
  int32_t per_unit;         // heads that one lane group takes in turn
  int32_t units_per_token;
};

constexpr int kRopeUnit = 2;  // most heads of a unit: rotation and writing,
constexpr int kReadUnit = 4;  // and reading

struct KvReadParams {
  KvView cache;
  const int64_t* slots;
  uint16_t* k_out;
  uint16_t* v_out;
  int32_t tokens;
  int32_t per_unit, units_per_token;
};

// ---- token scores
constexpr int kScoreThreads = 256;
constexpr int kScoreTile = 8192;                          // least logits of a part: a round of the waves
constexpr int kScoreAlign = 64;                           // parts are multiples
constexpr int kScoreMaxTop = 64;
// Ints from a row's counter to the next one's: a cache line, on which parts of one row
// only arrive (64 rows x 16 parts on two lines waited 3 us for each other).
constexpr int kScoreCounterStride = 16;
constexpr int kScoreMaxSplits = 64;                       // parts of a row: lanes of the last wave
// What one part of a row hands over: max, sum, weighted sum, and top_k keys.
__host__ __device__ constexpr int64_t score_part_bytes(int top_k) { return 16 + (int64_t)top_k * 8; }

struct ScoreParams {
  const void* logits;
  const int64_t* ids;
  float* logprobs;
  float* entropy;
  float* top_logprobs;
  int64_t* top_ids;
  int64_t row_stride;
  char* parts;              // [tokens][splits] parts (splits > 1)
  int32_t* counters;        // [tokens], zero between launches
  int32_t tokens, vocab, top_k;
  int32_t splits;           // parts of a row
  int32_t part;             // logits of a part: a multiple of kScoreAlign
};

// ---- attention over the paged cache
constexpr int kAttnWaves = 4;
constexpr int kAttnTile = 32;            // tokens that a wave multiplies at a time
constexpr int kAttnStep = kAttnWaves * kAttnTile;  // tokens of a workgroup's step
// An item is at least this many steps long before there are more of them than
// CUs: parts cost their writing, a wait and their joining (one token over 32768
// e4m3 tokens, 8 heads: 24.6 us with 256 items of 8 steps, 26.7 with 512 of 4).
constexpr int kAttnFewSteps = 8;
constexpr int kAttnMaxSplits = 256;      // parts of a sequence
// Head dims a kernel is built for: the next of 64, 128, 256.
inline int attn_dim_block(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// Kernels by the rows (new token x query head) of a key/value head: up to 16 or
// 32, the waves of a workgroup share the rows and take turns at the tokens;
// above, each wave has 16 or 32 rows and they share the tokens through LDS.
// Measured at the borders (us, chosen / other): 32 rows, 64 trees over 4000 e4m3
// tokens 82 / 130 by the kernel of 64, 16 over int8 30 / 38, 16 over bf16 47 / 41;
// 56 rows, 16 trees over bf16 44 / 90 by the kernel of 32, 52 by that of 128; 96
// rows, 16 trees over int8 53 / 65 by that of 64, 2048 rows and more 213 / 301.
enum class AttnKind { kNarrow1, kNarrow2, kWide1, kWide2 };
inline AttnKind attn_kind(int64_t rows, int dim) {
  if (rows <= 16) return AttnKind::kNarrow1;
  if (attn_dim_block(dim) == 256) return AttnKind::kWide1;
  return rows <= 32 ? AttnKind::kNarrow2 : rows <= 64 ? AttnKind::kWide1 : AttnKind::kWide2;
}
inline int attn_rows(AttnKind k) {
  return k == AttnKind::kNarrow1 ? 16 : k == AttnKind::kNarrow2 ? 32 : k == AttnKind::kWide1 ? 64 : 128;
}
constexpr int kAttnStage = 64;           // tokens that the wide kernels stage at a time
// Floats of one part: rows of sums, then each row's maximum and denominator.
__host__ __device__ constexpr int64_t attn_part_floats(int rows, int dim_block) {
  return (int64_t)rows * (dim_block + 2);
}

struct AttnParams {
  KvView cache;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  const uint64_t* mask;     // null: causal
  float* parts;             // [items][attn_part_floats]
  int32_t* counters;        // one per (sequence, row block, head), zero between launches
  int64_t q_token, q_head, table_stride;
  int32_t tokens, sequences, table_pages, max_q, hq, group, mask_words;
  int32_t target;           // most work items aimed at; 0: never split a sequence
  int32_t few;              // ... while an item is shorter than kAttnFewSteps steps
  int32_t grid;
  float scale_log2;         // scale * log2(e)
};

// One per dtype and format, each a source file of its own (build time).
hipError_t attn_f16_same(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t attn_f16_e4m3(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t attn_f16_int8(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t attn_bf16_same(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t attn_bf16_e4m3(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t attn_bf16_int8(const AttnParams& p, AttnKind kind, hipStream_t stream);
hipError_t launch_rope_table(const RopeTableParams& p, hipStream_t stream);
hipError_t launch_rope_kv(const RopeKvParams& p, int dtype, int format, hipStream_t stream);
hipError_t launch_kv_read(const KvReadParams& p, int dtype, int format, hipStream_t stream);
hipError_t launch_token_logprobs(const ScoreParams& p, int dtype, hipStream_t stream);

}  // namespace w4a16
