// Internal interface between the host side (batch_host.cpp) and the gfx950 kernels of the
// operators of a batch of requests: verification of drafts, pages of the cache, adapters.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_internal.h"

namespace w4a16 {

// ---- verification of drafts
constexpr int kVerifyThreads = 256;       // weighing: a chunk of logits a wave
constexpr int kWalkThreads = 512;         // walking and drawing
constexpr int kVerifyMaxNodes = 1024;
constexpr int64_t kVerifyMaxVocab = (int64_t)1 << 20;
// Logits of a chunk: 4 vectors of 16 bytes a lane.
__host__ __device__ constexpr int verify_chunk(int dtype) { return dtype == W4A16_F32 ? 1024 : 2048; }
// Chunks of a row: they start at 16-byte boundaries of memory, so that the first may hold fewer.
__host__ __device__ constexpr int verify_chunks(int64_t vocab, int dtype) {
  return (int)((vocab + 7 + verify_chunk(dtype) - 1) / verify_chunk(dtype));
}

// Spans of a row, which the second kernel sums in fp64; they start as the chunks do. Its us
// with 512, 1024 and 2048 logits: 5 rows of 32000 13.1, 13.0, 14.9; 64 chains over 151667
// with drafts 30.0, 29.1, 32.0; 16 trees 17.5, 15.9, 16.8.
constexpr int kVerifySpan = 1024;
constexpr int verify_spans(int64_t vocab) { return (int)((vocab + 7 + kVerifySpan - 1) / kVerifySpan); }
constexpr int kVerifyMaxSpans = verify_spans(kVerifyMaxVocab);

// What a wave knows of its chunk: the weights' sum, formed in fp32, against the chunk's own
// largest logit m (NaN: the chunk holds NaN), and, greedy, where m stands first.
struct VerifyChunk {
  double s;
  float m;
  int32_t first;
};

struct VerifyParams {
  const void* logits;
  const int64_t* ids;
  const int32_t* q_starts;
  const int32_t* parents;
  const float* probs;
  const float* temperatures;
  const float* uniforms;
  const float* finals;
  int64_t* out_tokens;
  int32_t* path;
  int32_t* counts;
  int64_t row_stride, probs_stride;
  VerifyChunk* parts;       // [tokens][chunks]
  double* over;             // [sequences][3][spans], of the last node's row: the weights' sum in fp64, what
                            // of it is above a draft, and how that changes (two floats)
  int32_t* counters;        // [sequences], zero between launches (groups > 1)
  int32_t tokens, vocab, sequences, max_q;
  int32_t chunks, spans;
  int32_t groups;           // workgroups of a sequence in the second kernel
};

// ---- pages
constexpr int kPagesThreads = 1024;
constexpr int kPagesMaxList = 4096;
struct PagesParams {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  const int32_t* from;
  const int32_t* to;
  int32_t* served;
  int32_t* src;
  int32_t* dst;
  int64_t table_stride;
  int32_t pages, rows, table_pages, page_shift, count;
};

// Caches of one launch, whose addresses are kernel arguments: a launch with 2 KiB of them takes
// the host 0.6 us more than one with few.
constexpr int kFewCaches = 16, kGroupCaches = 64;
struct CacheAddresses {
  char* k;
  char* v;
  char* k_scale;
  char* v_scale;
};
template <int N>
struct CacheList {
  CacheAddresses at[N];
};
struct CopyPagesParams {
  const int32_t* src;
  const int32_t* dst;
  int64_t pages;
  uint32_t page_units, scale_units;       // 16-byte units of a page of k, and of its scales
  uint32_t chunks;                        // workgroups of a pair and cache
  int32_t count;
  int64_t pairs;
};
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;              // units of a thread

struct CompactParams {
  const int32_t* block_table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  const int32_t* path;
  const int32_t* counts;
  int32_t* new_lens;                      // null: not of this launch
  int64_t table_stride, pages;
  int32_t sequences, table_pages, width, count;
  int32_t page_shift, heads;
  int32_t row_units;                      // 16-byte units of a token's row of one head
  int32_t scaled;
  int32_t blocks;                         // workgroups of a sequence and cache
};
constexpr int kCompactThreads = 256;

// ---- adapters
constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraMaxTokens = 1 << 24;
constexpr int kLoraPlanThreads = 512;
constexpr int kLoraDownThreads = 512;
constexpr int kLoraThreads = 256;
constexpr int kUpColumns = 256;           // of n that a workgroup of the second kernel takes at a time
// Threads of a workgroup that does both products, and columns that it takes at a time: for
// 16 ranks more waves with one step's loads each, for more of them fewer with two.
__host__ __device__ constexpr int lora_once_threads(int rank_block) { return rank_block <= 16 ? 1024 : 512; }
constexpr int kLoraMaxSplits = 16;
constexpr int kLoraStep = 128;            // of k: splits are multiples
// Rows of a tile: tokens of one adapter that are multiplied at a time. us of a call with tiles of 16
// and of 64 rows, k 5120, n 17408, 24, 64 and 128 tokens an adapter: 32 adapters of 64 ranks
// 49.1 51.0, 86.0 61.1, 160.8 104.5; 32 of 16 26.5 29.2, 54.2 41.6, 89.3 80.4; 4 of 64 15.4 18.7,
// 23.6 26.4, 32.5 30.3; 4 of 16 10.3 13.2, 13.4 17.8, 17.4 19.7; 1 of 64 12.2 16.5, 13.2 16.9, 15.4 17.9.
inline int lora_tile_rows(int64_t tokens, int64_t adapters) { return tokens >= 64 * adapters ? 64 : 16; }
// Most tiles that a plan can hold; tokens without an adapter are a group of their own.
inline int64_t lora_max_tiles(int64_t tokens, int64_t adapters) {
  const int64_t rows = lora_tile_rows(tokens, adapters);
  const int64_t most = (tokens + rows - 1) / rows + adapters;
  return most < tokens ? most : tokens;
}
// Rank that the kernels are built for.
__host__ __device__ constexpr int lora_rank_block(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Parts of 16 tokens that a workgroup of the first kernel takes of a tile of 64: fewer read a
// again, more leave CUs idle or split k (8192 tokens, k 5120, rank 64: 1 part 43.5 us, 2 32.2,
// 4 42.1).
constexpr int kLoraDownParts = 2;
// k that a wave of the first kernel takes at a time, with `tiles` of 16 tokens.
__host__ __device__ constexpr int lora_step(int tiles, int rank_block) {
  return tiles * (rank_block / 16) <= 2 ? 128 : tiles * (rank_block / 16) <= 8 && rank_block <= 64 ? 64 : 32;
}

// A plan: each tile's adapter, and each tile's tokens in ascending order, -1 behind them.
// Rows lie where their tile is, so that a workgroup knows its rows without having seen the
// tile, and reads both at once.
constexpr int kLoraNone = -1;             // a tile of tokens without an adapter
constexpr int kLoraUnused = -2;           // no tile
struct LoraPlanParams {
  const int32_t* index;
  int32_t* tile;            // [max_tiles]
  int32_t* token;           // [max_tiles][tile_rows]
  int32_t tokens, adapters, tile_rows, max_tiles;
};
struct LoraParams {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const uint16_t* base;
  uint16_t* out;
  const float* scales;
  const int32_t* ranks;
  const int32_t* tile;
  const int32_t* token;
  float* parts;             // [splits][rows of all tiles][rank block] (splits > 1)
  uint16_t* high;           // [rows of all tiles][rank block]: v's parts
  uint16_t* low;
  float* factor;            // [rows of all tiles]: the adapter's scale, and a power of two
  int32_t* counters;        // [tiles], zero between launches (splits > 1)
  int64_t x_stride, base_stride, out_stride;
  int32_t tokens, k, n, adapters, rank, tiles_most;
  int32_t splits;           // of k over workgroups; 0: one kernel for both
  int32_t steps;            // of kLoraStep that a split takes
  int32_t columns;          // of n that a workgroup of the second kernel (or of the only one) takes
};

hipError_t launch_verify(const VerifyParams& p, int dtype, hipStream_t stream);
hipError_t launch_pages(const PagesParams& p, bool fork, hipStream_t stream);
hipError_t launch_copy_pages(const CopyPagesParams& p, const CacheList<kGroupCaches>& caches, hipStream_t stream);
hipError_t launch_compact(const CompactParams& p, const CacheList<kGroupCaches>& caches, hipStream_t stream);
hipError_t launch_lora_plan(const LoraPlanParams& p, hipStream_t stream);
hipError_t launch_lora(const LoraParams& p, int tile_rows, int dtype, hipStream_t stream);

}  // namespace w4a16
