// Host side of the operators of a batch of requests (include/w4a16.h): verification of
// drafts, pages of the cache, adapters. Argument checks, launch shapes, scratch accounting.
// Nothing here synchronises, allocates device memory, or reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <utility>

#include "batch_internal.h"
#include "serve_checks.h"

namespace w4a16 {
namespace {

using namespace checks;

// ---- verification of drafts
int32_t verify_groups(int64_t sequences, int spans, int num_cus) {
  // Workgroups of a sequence that share the last row: a span a wave, while all of them are
  // resident; counters bound how many sequences may have several.
  if (sequences > kCounterBytes / 4) return 1;
  const int64_t most = div_up(spans, kWalkThreads / 64);
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(most, 2 * (int64_t)num_cus / std::max<int64_t>(sequences, 1)));
}

w4a16_status check_logits_dtype(int32_t dtype) {
  if (dtype == W4A16_F16 || dtype == W4A16_BF16 || dtype == W4A16_F32) return W4A16_OK;
  return report(W4A16_ERR_DTYPE, "dtype %d: fp16 (0), bf16 (1) and fp32 (2) are supported", (int)dtype);
}

w4a16_status verify_workspace(int64_t tokens, int64_t vocab, int32_t sequences, int32_t max_q, int32_t dtype,
                              int64_t* bytes) {
  w4a16_status st = check_logits_dtype(dtype);
  if (st != W4A16_OK) return st;
  if (vocab < 1 || vocab > kVerifyMaxVocab || tokens < 0 || sequences < 0 || sequences > (1 << 20) || max_q < 0 ||
      max_q > kVerifyMaxNodes)
    return report(W4A16_ERR_SHAPE,
                  "need 1 <= vocab <= 2^20, tokens >= 0, 0..2^20 sequences and 0 <= max_q <= %d", kVerifyMaxNodes);
  const int64_t chunks = verify_chunks(vocab, dtype);
  if (tokens > kMaxGrid * (kVerifyThreads / 64) / chunks)
    return report(W4A16_ERR_SHAPE, "%lld tokens of %lld logits are too many for one launch", (long long)tokens,
                  (long long)vocab);
  const int64_t sums = tokens * chunks * (int64_t)sizeof(VerifyChunk) + (int64_t)sequences * verify_spans(vocab) * 24;
  *bytes = tokens == 0 ? 0 : kCounterBytes + sums;
  return W4A16_OK;
}

// ---- pages
w4a16_status check_page_size(int32_t page_size, int32_t* shift) {
  int s = 0;
  while ((1 << s) < page_size && s < 12) ++s;
  if (page_size < 16 || page_size != (1 << s))
    return report(W4A16_ERR_SHAPE, "page_size=%d must be a power of two in 16..4096", (int)page_size);
  *shift = s;
  return W4A16_OK;
}

w4a16_status pages_call(const w4a16_pages_t* a, bool fork, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  const w4a16_page_pool_t& pool = a->pool;
  PagesParams p{};
  w4a16_status st = check_page_size(pool.page_size, &p.page_shift);
  if (st != W4A16_OK) return st;
  if (pool.pages < 0 || pool.pages > kMaxInt / 2 || pool.rows < 0 || pool.table_pages < 0)
    return report(W4A16_ERR_SHAPE, "need 0 <= pages <= 2^30, rows >= 0 and table_pages >= 0");
  if (pool.table_stride < pool.table_pages || pool.table_stride >= kMaxStride)
    return report(W4A16_ERR_SHAPE, "need table_pages <= table_stride < 2^40 (got %d, %lld)", (int)pool.table_pages,
                  (long long)pool.table_stride);
  if ((int64_t)pool.table_pages << p.page_shift >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "a row's table_pages * page_size must be below 2^31");
  if (a->count < 0 || a->count > kPagesMaxList)
    return report(W4A16_ERR_SHAPE, "count=%d must lie in 0..%d", (int)a->count, kPagesMaxList);
  if (a->count == 0) return W4A16_OK;
  if (!a->from || !a->to || !a->served || !a->src || !a->dst || (pool.pages > 0 && !pool.refs) ||
      (pool.rows > 0 && (!pool.lens || (pool.table_pages > 0 && !pool.block_table))))
    return report(W4A16_ERR_NULL, "the pool's arrays, the lists and the outputs must be non-NULL");
  for (const void* x : {(const void*)pool.refs, (const void*)pool.block_table, (const void*)pool.lens,
                        (const void*)a->from, (const void*)a->to, (const void*)a->served, (const void*)a->src,
                        (const void*)a->dst})
    if (!aligned(x, 4)) return report(W4A16_ERR_ALIGN, "arrays must be aligned to their elements");
  int cus;
  st = current_device(&cus);
  if (st != W4A16_OK) return st;
  p.refs = pool.refs;
  p.table = pool.block_table;
  p.lens = pool.lens;
  p.from = a->from;
  p.to = a->to;
  p.served = a->served;
  p.src = a->src;
  p.dst = a->dst;
  p.table_stride = pool.table_stride;
  p.pages = (int32_t)pool.pages;
  p.rows = pool.rows;
  p.table_pages = pool.table_pages;
  p.count = a->count;
  return launched(launch_pages(p, fork, (hipStream_t)stream));
}

// Caches that one call covers: alike but for their addresses.
w4a16_status check_caches(const w4a16_kv_cache_t* caches, int32_t count, KvView* view) {
  if (count < 0 || count > 4096) return report(W4A16_ERR_SHAPE, "count=%d must lie in 0..4096", (int)count);
  if (count == 0) return W4A16_OK;
  if (!caches) return report(W4A16_ERR_NULL, "caches must be non-NULL");
  for (int i = 0; i < count; ++i) {
    const w4a16_status st = check_cache(caches[i], i == 0 ? view : nullptr);
    if (st != W4A16_OK) return st;
    const w4a16_kv_cache_t &c = caches[i], &f = caches[0];
    if (c.pages != f.pages || c.page_size != f.page_size || c.heads != f.heads || c.head_dim != f.head_dim ||
        c.format != f.format)
      return report(W4A16_ERR_SHAPE, "cache %d differs from the first in its sizes or format", i);
  }
  return W4A16_OK;
}

int fill_addresses(const w4a16_kv_cache_t* caches, int32_t first, int32_t count, CacheList<kGroupCaches>* to) {
  const int n = std::min<int32_t>(kGroupCaches, count - first);
  for (int i = 0; i < n; ++i) {
    const w4a16_kv_cache_t& c = caches[first + i];
    to->at[i] = CacheAddresses{(char*)c.k, (char*)c.v, (char*)c.k_scale, (char*)c.v_scale};
  }
  return n;
}

bool overlap(const int32_t* x, int64_t nx, const int32_t* y, int64_t ny) {
  const uintptr_t a = (uintptr_t)x, b = (uintptr_t)y;
  return nx > 0 && ny > 0 && a < b + (uintptr_t)ny * 4 && b < a + (uintptr_t)nx * 4;
}

int element_bytes(int32_t format) { return format == W4A16_KV_SAME ? 2 : 1; }

// ---- adapters
w4a16_status check_lora_counts(int64_t tokens, int32_t adapters) {
  if (tokens < 0 || tokens > kLoraMaxTokens || adapters < 1 || adapters > kLoraMaxAdapters)
    return report(W4A16_ERR_SHAPE, "need 0..2^24 tokens (got %lld) and 1..%d adapters (got %d)", (long long)tokens,
                  kLoraMaxAdapters, (int)adapters);
  return W4A16_OK;
}

// Where the tokens of a plan start.
int64_t plan_tokens_at(int64_t tokens, int32_t adapters) {
  return div_up(lora_max_tiles(tokens, adapters) * 4, 16) * 16;
}

// Splits of k over workgroups: as many as make one a CU, each with a step for every wave.
// us of the first kernel with 1, 3, this rule's and 8 splits: 64 tokens, k 5120, rank 16 6.9,
// 6.8, (5) 6.1, 7.0; 384, 2112, 64 8.6, 7.9, (5) 7.6, 7.9; 8192, 5120, 64 (1) 32.2, 3 42.0.
int32_t lora_splits(int64_t tokens, int32_t adapters, int32_t k, int32_t rank, int num_cus, int32_t* steps) {
  const int64_t all = div_up(k, kLoraStep);
  const int parts = lora_tile_rows(tokens, adapters) == 64 ? kLoraDownParts : 1;
  const int64_t groups = std::max<int64_t>(div_up(tokens, 16 * parts), 1);
  const int64_t step = lora_step(parts, lora_rank_block(rank));
  const int64_t want = std::max<int64_t>(
      1, std::min<int64_t>({num_cus / groups, div_up(k, step * (kLoraDownThreads / 64)), kLoraMaxSplits}));
  *steps = (int32_t)div_up(all, want);
  return (int32_t)div_up(all, *steps);
}

// Columns that a workgroup takes where one kernel does both products, or 0: two are launched.
// It wins while all its workgroups are resident, none takes many columns, and each wave has at
// most 4 steps of k, all of a being read by every workgroup. us of a call replayed from a
// graph, with two kernels (of which clearing their scratch is 1.8) and with one, n 4096:
//   1 token, 16 ranks: k 1024 7.1, 4.9; 4096 8.8, 6.9; 8192 9.2, 9.3; 12288 9.8, 11.8
//   64 tokens, 32 adapters of 16: k 1024 8.2, 5.4; 4096 10.7, 8.1; 8192 12.3, 10.7; 16384 15.4, 16.5
//   1 token, 32 ranks: k 1024 7.9, 5.2; 4096 9.8, 8.5; 8192 10.2, 12.3
//   1 token, 64 ranks: k 1024 10.5, 7.8; 2048 11.0, 9.2; 4096 11.9, 12.5
// 200 tokens, 64 adapters, k 1024, 6144 columns a workgroup: 16 ranks 15.9, 14.2, 64 ranks 37.2, 42.8.
// More tiles move the crossing up, which the rule leaves aside: 64 tokens, 32 adapters of 64, k 5120 20.6,
// 19.0; 200 tokens, 64 adapters of 16, k 12288 18.3, 16.0.
constexpr int kOnceSteps = 4;
constexpr int64_t kOnceMaxColumns = 4096;
int32_t lora_once_columns(int64_t tokens, int32_t k, int32_t n, int32_t adapters, int32_t rank, int num_cus) {
  const int block = lora_rank_block(rank), threads = lora_once_threads(block);
  const int64_t tiles = lora_max_tiles(tokens, adapters);
  if (lora_tile_rows(tokens, adapters) != 16 || block > 64 || tiles > num_cus ||
      k > kOnceSteps * (threads / 64) * lora_step(1, block))
    return 0;
  const int64_t columns = threads * div_up(div_up(n, threads), num_cus / tiles);
  return columns <= kOnceMaxColumns ? (int32_t)columns : 0;
}

w4a16_status lora_workspace(int64_t tokens, int32_t k, int32_t n, int32_t adapters, int32_t rank, int num_cus,
                            int64_t* bytes) {
  w4a16_status st = check_lora_counts(tokens, adapters);
  if (st != W4A16_OK) return st;
  if (rank < 8 || rank > 128 || rank % 8 != 0)
    return report(W4A16_ERR_SHAPE, "rank=%d must be a multiple of 8 in 8..128", (int)rank);
  if (k < 8 || k > (1 << 24) || k % 8 != 0)
    return report(W4A16_ERR_SHAPE, "k=%d must be a multiple of 8 in 8..2^24", (int)k);
  if (n < 8 || n > (1 << 22) || n % 8 != 0)
    return report(W4A16_ERR_SHAPE, "n=%d must be a multiple of 8 in 8..2^22", (int)n);
  *bytes = 0;
  if (tokens == 0 || lora_once_columns(tokens, k, n, adapters, rank, num_cus) > 0) return W4A16_OK;
  int32_t steps;
  const int64_t splits = lora_splits(tokens, adapters, k, rank, num_cus, &steps);
  // counters, the splits' sums, v's two parts and a factor for each row
  const int64_t rows = lora_max_tiles(tokens, adapters) * lora_tile_rows(tokens, adapters);
  *bytes = kCounterBytes + rows * (((splits > 1 ? splits : 0) + 1) * lora_rank_block(rank) + 1) * 4;
  return W4A16_OK;
}

w4a16_status check_rows(const char* what, int64_t stride, int64_t tokens, int64_t width, bool apart) {
  if (stride % 8 != 0) return report(W4A16_ERR_ALIGN, "%s: a stride of %lld is no multiple of 8", what, (long long)stride);
  if (stride < 0 || stride >= kMaxStride || (apart && tokens > 1 && stride < width))
    return report(W4A16_ERR_SHAPE, "%s: rows of %lld lie at a stride of %lld", what, (long long)width,
                  (long long)stride);
  return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_verify_drafts_workspace_bytes(int64_t tokens, int64_t vocab, int32_t sequences, int32_t max_q,
                                                 int32_t dtype, int32_t num_cus, int64_t* bytes) {
  (void)num_cus;  // scratch is one sum a chunk, however the chunks are spread
  if (!bytes) return report(W4A16_ERR_NULL, "bytes must be non-NULL");
  return verify_workspace(tokens, vocab, sequences, max_q, dtype, bytes);
}

w4a16_status w4a16_verify_drafts(const w4a16_verify_drafts_t* a, void* workspace, int64_t ws_bytes, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  int64_t need;
  CHECK(verify_workspace(a->tokens, a->vocab, a->sequences, a->max_q, a->dtype, &need));
  if (a->draft_probs && a->parents)
    return report(W4A16_ERR_SHAPE, "draft_probs go with chains: parents must be NULL");
  if (a->row_stride < 0 || a->row_stride >= kMaxStride || a->probs_stride < 0 || a->probs_stride >= kMaxStride)
    return report(W4A16_ERR_SHAPE, "row strides must lie in 0..2^40");
  if (a->sequences == 0) return W4A16_OK;
  if (!a->q_starts || !a->final_uniforms || !a->counts || (a->max_q > 0 && (!a->out_tokens || !a->path)) ||
      (a->tokens > 0 && (!a->logits || !a->ids || !a->uniforms)))
    return report(W4A16_ERR_NULL, "logits, ids, q_starts, the random numbers and every output must be non-NULL");
  if (!aligned(a->logits, a->dtype == W4A16_F32 ? 4 : 2) || !aligned(a->ids, 8) || !aligned(a->out_tokens, 8) ||
      !aligned(a->q_starts, 4) || !aligned(a->parents, 4) || !aligned(a->draft_probs, 4) ||
      !aligned(a->temperatures, 4) || !aligned(a->uniforms, 4) || !aligned(a->final_uniforms, 4) ||
      !aligned(a->path, 4) || !aligned(a->counts, 4))
    return report(W4A16_ERR_ALIGN, "arrays must be aligned to their elements");
  int cus = kWholeDevice;
  const w4a16_status device = current_device(&cus);
  CHECK(check_workspace(workspace, ws_bytes, need));
  if (device != W4A16_OK) return device;
  VerifyParams p{};
  p.logits = a->logits;
  p.ids = a->ids;
  p.q_starts = a->q_starts;
  p.parents = a->parents;
  p.probs = a->draft_probs;
  p.temperatures = a->temperatures;
  p.uniforms = a->uniforms;
  p.finals = a->final_uniforms;
  p.out_tokens = a->out_tokens;
  p.path = a->path;
  p.counts = a->counts;
  p.row_stride = a->row_stride;
  p.probs_stride = a->probs_stride;
  p.tokens = (int32_t)a->tokens;
  p.vocab = (int32_t)a->vocab;
  p.sequences = a->sequences;
  p.max_q = a->max_q;
  p.chunks = verify_chunks(a->vocab, a->dtype);
  p.spans = verify_spans(a->vocab);
  p.groups = a->tokens > 0 ? verify_groups(a->sequences, p.spans, cus) : 1;
  if (need > 0) {
    p.counters = (int32_t*)workspace;
    p.parts = (VerifyChunk*)((char*)workspace + kCounterBytes);
    p.over = (double*)(p.parts + a->tokens * p.chunks);
  }
  return launched(launch_verify(p, a->dtype, (hipStream_t)stream));
}

w4a16_status w4a16_pages_resize(const w4a16_pages_t* a, void* stream) { return pages_call(a, false, stream); }

w4a16_status w4a16_pages_fork(const w4a16_pages_t* a, void* stream) { return pages_call(a, true, stream); }

w4a16_status w4a16_kv_copy_pages(const w4a16_kv_copy_pages_t* a, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  KvView view{};
  CHECK(check_caches(a->caches, a->count, &view));
  if (a->pairs < 0 || a->pairs >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "need 0 <= pairs < 2^31 (got %lld)", (long long)a->pairs);
  if (a->pairs == 0 || a->count == 0 || view.pages == 0) return W4A16_OK;
  if (!a->src || !a->dst) return report(W4A16_ERR_NULL, "src and dst must be non-NULL");
  if (!aligned(a->src, 4) || !aligned(a->dst, 4))
    return report(W4A16_ERR_ALIGN, "src and dst must be aligned to their elements");
  const int32_t format = a->caches[0].format;
  const int64_t tokens = (int64_t)view.heads << view.page_shift;
  CopyPagesParams p{};
  CacheList<kGroupCaches> caches{};
  p.page_units = (uint32_t)(tokens * view.dim * element_bytes(format) / 16);
  p.scale_units = format == W4A16_KV_SAME ? 0 : (uint32_t)(tokens * 4 / 16);
  p.chunks = (uint32_t)div_up(2 * ((int64_t)p.page_units + p.scale_units), kCopyThreads * kCopyEach);
  if (a->pairs > kMaxGrid / ((int64_t)p.chunks * kGroupCaches))
    return report(W4A16_ERR_SHAPE, "%lld pairs of these pages are too many for one launch", (long long)a->pairs);
  int cus;
  CHECK(current_device(&cus));
  p.src = a->src;
  p.dst = a->dst;
  p.pages = view.pages;
  p.pairs = a->pairs;
  for (int32_t first = 0; first < a->count; first += p.count) {
    p.count = fill_addresses(a->caches, first, a->count, &caches);
    CHECK(launched(launch_copy_pages(p, caches, (hipStream_t)stream)));
  }
  return W4A16_OK;
}

w4a16_status w4a16_kv_compact(const w4a16_kv_compact_t* a, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  KvView view{};
  CHECK(check_caches(a->caches, a->count, &view));
  if (a->sequences < 0 || a->sequences > (1 << 20) || a->width < 0 || a->table_pages < 0)
    return report(W4A16_ERR_SHAPE, "need 0..2^20 sequences, width >= 0 and table_pages >= 0");
  if (a->table_stride < 0 || a->table_stride >= kMaxStride || (a->sequences > 1 && a->table_stride < a->table_pages))
    return report(W4A16_ERR_SHAPE, "block_table: rows of %d pages lie at a stride of %lld", (int)a->table_pages,
                  (long long)a->table_stride);
  if (a->sequences == 0) return W4A16_OK;
  if (!a->kv_lens || !a->q_starts || !a->counts || !a->new_lens || (a->width > 0 && !a->path) ||
      (a->table_pages > 0 && !a->block_table))
    return report(W4A16_ERR_NULL, "block_table, kv_lens, q_starts, path, counts and new_lens must be non-NULL");
  if (!aligned(a->block_table, 4) || !aligned(a->kv_lens, 4) || !aligned(a->q_starts, 4) || !aligned(a->path, 4) ||
      !aligned(a->counts, 4) || !aligned(a->new_lens, 4))
    return report(W4A16_ERR_ALIGN, "arrays must be aligned to their elements");
  // other workgroups, and the launches of later caches, read these after the lengths are written
  const int64_t B = a->sequences, width = a->width;
  const int64_t entries = a->table_pages ? (B - 1) * a->table_stride + a->table_pages : 0;
  using Read = std::pair<const int32_t*, int64_t>;
  for (const auto& [x, count] : {Read{a->kv_lens, B}, Read{a->q_starts, B + 1}, Read{a->counts, B},
                                 Read{a->path, B * width}, Read{a->block_table, entries}})
    if (overlap(a->new_lens, B, x, count))
      return report(W4A16_ERR_SHAPE, "new_lens must be apart from block_table, kv_lens, q_starts, path and counts");
  const bool none = a->count == 0 || view.pages == 0;
  CompactParams p{};
  CacheList<kGroupCaches> caches{};
  p.row_units = none ? 0 : view.dim * element_bytes(a->caches[0].format) / 16;
  p.scaled = !none && a->caches[0].format != W4A16_KV_SAME;
  const int64_t work = (int64_t)view.heads * 2 * (p.row_units + p.scaled);
  p.blocks = (int32_t)std::max<int64_t>(1, div_up(work, kCompactThreads));
  if (a->sequences > kMaxGrid / ((int64_t)p.blocks * kGroupCaches))
    return report(W4A16_ERR_SHAPE, "%d sequences of %d heads are too many for one launch", (int)a->sequences,
                  (int)view.heads);
  int cus;
  CHECK(current_device(&cus));
  p.block_table = a->block_table;
  p.kv_lens = a->kv_lens;
  p.q_starts = a->q_starts;
  p.path = a->path;
  p.counts = a->counts;
  p.new_lens = a->new_lens;
  p.table_stride = a->table_stride;
  p.pages = none ? 0 : view.pages;
  p.sequences = a->sequences;
  p.table_pages = a->table_pages;
  p.width = a->width;
  p.page_shift = view.page_shift;
  p.heads = view.heads;
  if (none) {  // lengths alone
    p.count = 1;
    return launched(launch_compact(p, caches, (hipStream_t)stream));
  }
  for (int32_t first = 0; first < a->count; first += p.count) {
    p.count = fill_addresses(a->caches, first, a->count, &caches);
    CHECK(launched(launch_compact(p, caches, (hipStream_t)stream)));
    p.new_lens = nullptr;
  }
  return W4A16_OK;
}

w4a16_status w4a16_lora_plan_bytes(int64_t tokens, int32_t adapters, int64_t* bytes) {
  if (!bytes) return report(W4A16_ERR_NULL, "bytes must be non-NULL");
  CHECK(check_lora_counts(tokens, adapters));
  *bytes = plan_tokens_at(tokens, adapters) + lora_max_tiles(tokens, adapters) * lora_tile_rows(tokens, adapters) * 4;
  return W4A16_OK;
}

w4a16_status w4a16_lora_plan(const int32_t* index, int64_t tokens, int32_t adapters, void* plan, void* stream) {
  CHECK(check_lora_counts(tokens, adapters));
  if (tokens == 0) return W4A16_OK;
  if (!index || !plan) return report(W4A16_ERR_NULL, "index and plan must be non-NULL");
  if (!aligned(index, 4) || !aligned(plan, 16))
    return report(W4A16_ERR_ALIGN, "index must be 4-byte aligned, the plan 16-byte");
  int cus;
  CHECK(current_device(&cus));
  LoraPlanParams p{};
  p.index = index;
  p.tile = (int32_t*)plan;
  p.token = (int32_t*)((char*)plan + plan_tokens_at(tokens, adapters));
  p.tokens = (int32_t)tokens;
  p.adapters = adapters;
  p.tile_rows = lora_tile_rows(tokens, adapters);
  p.max_tiles = (int32_t)lora_max_tiles(tokens, adapters);
  return launched(launch_lora_plan(p, (hipStream_t)stream));
}

w4a16_status w4a16_lora_workspace_bytes(int64_t tokens, int32_t k, int32_t n, int32_t adapters, int32_t rank,
                                        int32_t num_cus, int64_t* bytes) {
  if (!bytes) return report(W4A16_ERR_NULL, "bytes must be non-NULL");
  return lora_workspace(tokens, k, n, adapters, rank, num_cus > 0 ? num_cus : kWholeDevice, bytes);
}

w4a16_status w4a16_lora(const w4a16_lora_t* a, void* workspace, int64_t ws_bytes, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  CHECK(check_dtype(a->dtype));
  int64_t need;
  CHECK(lora_workspace(a->tokens, a->k, a->n, a->adapters, a->rank, kWholeDevice, &need));
  CHECK(check_rows("x", a->x_stride, a->tokens, a->k, false));
  CHECK(check_rows("base", a->base ? a->base_stride : 0, a->tokens, a->n, false));
  CHECK(check_rows("out", a->out_stride, a->tokens, a->n, true));
  if (a->tokens == 0) return W4A16_OK;
  if (!a->x || !a->a || !a->b || !a->out || !a->plan)
    return report(W4A16_ERR_NULL, "x, a, b, out and the plan must be non-NULL");
  if (!aligned(a->x, 16) || !aligned(a->a, 16) || !aligned(a->b, 16) || !aligned(a->base, 16) ||
      !aligned(a->out, 16) || !aligned(a->plan, 16) || !aligned(a->scales, 4) || !aligned(a->ranks, 4))
    return report(W4A16_ERR_ALIGN, "x, a, b, base, out and the plan must be 16-byte aligned, the rest to its elements");
  if (a->base == a->out && a->base_stride != a->out_stride)
    return report(W4A16_ERR_SHAPE, "in place, out needs base's stride");
  if (a->x == a->out) return report(W4A16_ERR_SHAPE, "x must not be out: it is read while out is written");
  int cus = kWholeDevice;
  const w4a16_status device = current_device(&cus);
  CHECK(lora_workspace(a->tokens, a->k, a->n, a->adapters, a->rank, cus, &need));
  CHECK(check_workspace(workspace, ws_bytes, need));
  if (device != W4A16_OK) return device;
  LoraParams p{};
  p.x = (const uint16_t*)a->x;
  p.a = (const uint16_t*)a->a;
  p.b = (const uint16_t*)a->b;
  p.base = (const uint16_t*)a->base;
  p.out = (uint16_t*)a->out;
  p.scales = a->scales;
  p.ranks = a->ranks;
  p.tile = (const int32_t*)a->plan;
  p.token = (const int32_t*)((const char*)a->plan + plan_tokens_at(a->tokens, a->adapters));
  p.x_stride = a->x_stride;
  p.base_stride = a->base_stride;
  p.out_stride = a->out_stride;
  p.tokens = (int32_t)a->tokens;
  p.k = a->k;
  p.n = a->n;
  p.adapters = a->adapters;
  p.rank = a->rank;
  p.tiles_most = (int32_t)lora_max_tiles(a->tokens, a->adapters);
  p.splits = lora_splits(a->tokens, a->adapters, a->k, a->rank, cus, &p.steps);
  const int rows = lora_tile_rows(a->tokens, a->adapters);
  const int64_t values = (int64_t)p.tiles_most * rows * lora_rank_block(a->rank);
  p.counters = (int32_t*)workspace;
  p.high = (uint16_t*)((char*)workspace + kCounterBytes);
  p.low = p.high + values;
  p.parts = (float*)(p.low + values);
  p.factor = p.parts + (p.splits > 1 ? p.splits : 0) * values;
  // columns of a workgroup of the second kernel: those of a step until there are 2048 of them
  const int64_t steps = div_up(a->n, kUpColumns);
  p.columns = (int32_t)(kUpColumns * std::min(div_up(p.tiles_most * steps, 2048), steps));
  const int32_t once = lora_once_columns(a->tokens, a->k, a->n, a->adapters, a->rank, cus);
  if (once > 0) {
    p.splits = 0;
    p.columns = once;
  }
  if ((int64_t)p.tiles_most * div_up(a->n, p.columns) > kMaxGrid)
    return report(W4A16_ERR_SHAPE, "%lld tokens of %d columns are too many for one launch", (long long)a->tokens,
                  (int)a->n);
  return launched(launch_lora(p, rows, a->dtype, (hipStream_t)stream));
}

}  // extern "C"
