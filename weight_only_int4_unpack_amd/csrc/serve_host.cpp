// Host side of the operators around the weight products (include/w4a16.h):
// argument checks, launch shapes, scratch accounting. Nothing here
// synchronises, allocates device memory, or reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "serve_internal.h"

namespace w4a16 {
namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// All kernels here run workgroups of 256 threads, and a grid holds fewer than 2^32 threads.
constexpr int kServeThreads = 256;
constexpr int64_t kMaxGrid = ((int64_t)1 << 32) / kServeThreads - 1;
static_assert(kScoreThreads == kServeThreads && 64 * kAttnWaves == kServeThreads, "one limit for all");
// CUs of a device that is not partitioned. Sizes are checked for it before there is a
// device to ask; scratch, once there is one, for that device's own.
constexpr int kWholeDevice = 256;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

w4a16_status launched(hipError_t e) {
  if (e == hipSuccess) return W4A16_OK;
  return report(W4A16_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

w4a16_status check_dtype(int32_t dtype) {
  if (dtype == W4A16_F16 || dtype == W4A16_BF16) return W4A16_OK;
  return report(W4A16_ERR_DTYPE, "dtype %d: only fp16 (0) and bf16 (1) are supported", (int)dtype);
}

w4a16_status check_dim(int32_t dim) {
  if (dim >= 8 && dim <= 256 && dim % 8 == 0) return W4A16_OK;
  return report(W4A16_ERR_SHAPE, "head_dim=%d must be a multiple of 8 in 8..256", (int)dim);
}

// Token and head strides of an array of 16-bit heads.
w4a16_status check_strides(const char* what, int64_t token, int64_t head) {
  if (token % 8 != 0 || head % 8 != 0)
    return report(W4A16_ERR_ALIGN, "%s: strides (%lld, %lld) must be multiples of 8 elements", what,
                  (long long)token, (long long)head);
  if (token < 0 || head < 0 || token >= kMaxStride || head >= kMaxStride)
    return report(W4A16_ERR_SHAPE, "%s: strides (%lld, %lld) must lie in 0..2^40", what,
                  (long long)token, (long long)head);
  return W4A16_OK;
}

// An output's heads may lie in any order, but not one in another.
w4a16_status check_apart(const char* what, int64_t tokens, int64_t token, int64_t heads, int64_t head,
                         int64_t dim) {
  if (heads < 1) return W4A16_OK;
  int64_t inner = head, n = heads, outer = token, m = tokens;
  if (heads == 1 || (tokens > 1 && token < head)) {
    std::swap(inner, outer);
    std::swap(n, m);
  }
  if ((n > 1 && inner < dim) || (m > 1 && (outer < dim || (outer - dim) / inner < n - 1)))
    return report(W4A16_ERR_SHAPE, "%s: heads of %lld dims overlap at strides (%lld, %lld)", what,
                  (long long)dim, (long long)token, (long long)head);
  return W4A16_OK;
}

w4a16_status check_cache(const w4a16_kv_cache_t& c, KvView* view) {
  if (c.format != W4A16_KV_SAME && c.format != W4A16_KV_E4M3 && c.format != W4A16_KV_INT8)
    return report(W4A16_ERR_DTYPE, "cache format %d: 0 (same), 1 (e4m3) and 2 (int8) are supported",
                  (int)c.format);
  w4a16_status st = check_dim(c.head_dim);
  if (st != W4A16_OK) return st;
  // a lane of the attention kernels holds 16 dims of an 8-bit head, or of one above 128
  if (c.head_dim % 16 != 0 && (c.format != W4A16_KV_SAME || c.head_dim > 128))
    return report(W4A16_ERR_SHAPE,
                  "head_dim=%d must be a multiple of 16 above 128 and in a quantised cache",
                  (int)c.head_dim);
  int shift = 0;
  while ((1 << shift) < c.page_size && shift < 12) ++shift;
  if (c.page_size < 16 || c.page_size != (1 << shift))
    return report(W4A16_ERR_SHAPE, "page_size=%d must be a power of two in 16..4096",
                  (int)c.page_size);
  if (c.heads < 1 || c.heads > 4096 || c.pages < 0 || c.pages >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "need 1..4096 cache heads and 0..2^31 pages (got %d, %lld)",
                  (int)c.heads, (long long)c.pages);
  if (c.pages > 0) {
    if (!c.k || !c.v) return report(W4A16_ERR_NULL, "the cache's k and v must be non-NULL");
    if (!aligned(c.k, 16) || !aligned(c.v, 16))
      return report(W4A16_ERR_ALIGN, "the cache's k and v must be 16-byte aligned");
    if (c.format != W4A16_KV_SAME) {
      if (!c.k_scale || !c.v_scale)
        return report(W4A16_ERR_NULL, "a quantised cache needs k_scale and v_scale");
      if (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))
        return report(W4A16_ERR_ALIGN, "the cache's scales must be 16-byte aligned");
    }
  }
  if (view)
    *view = KvView{c.k, c.v, c.k_scale, c.v_scale, c.pages, shift, c.heads, c.head_dim};
  return W4A16_OK;
}

w4a16_status check_rotation(const int64_t* positions, const float* table, int64_t rows,
                            int32_t rot, int32_t dim) {
  if (!positions || !table)
    return report(W4A16_ERR_NULL, "a rotation needs positions and a table");
  if (rot < 2 || rot % 2 != 0 || rot > dim)
    return report(W4A16_ERR_SHAPE, "rot_dim=%d must be even and in 2..head_dim (%d)", (int)rot,
                  (int)dim);
  if (rows < 1 || rows >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "a table needs 1..2^31 rows (got %lld)", (long long)rows);
  if (!aligned(table, 16) || !aligned(positions, 8))
    return report(W4A16_ERR_ALIGN, "the table must be 16-byte aligned, positions 8-byte");
  return W4A16_OK;
}

// Heads that one lane group takes in turn: `most`, or fewer where that would
// leave less than 4096 waves (16 a CU).
w4a16_status shape_units(int64_t tokens, int64_t heads, int dim, int most, int32_t* per_unit, int32_t* units) {
  const int64_t waves = tokens * heads * lanes_per_head(dim) / 64;
  *per_unit = (int32_t)std::min<int64_t>({std::max<int64_t>(waves / 4096, 1), most, heads});
  *units = (int32_t)div_up(heads, *per_unit);
  if (div_up(tokens * *units, kServeThreads / lanes_per_head(dim)) > kMaxGrid)
    return report(W4A16_ERR_SHAPE, "%lld tokens of %lld heads are too many for one launch", (long long)tokens,
                  (long long)heads);
  return W4A16_OK;
}

w4a16_status check_count(int64_t tokens, int64_t heads) {
  if (tokens < 0 || tokens * heads >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "%lld tokens of %lld heads: need 0 <= tokens * heads < 2^31",
                  (long long)tokens, (long long)heads);
  return W4A16_OK;
}

// Parts of a row of logits: one round of the workgroups that the CUs hold, four
// each (300 rows x 50257 fp32: 1200 workgroups 36 us, 900 30 us; 256 rows x 151667
// bf16: twice as many 45 us, 1024 33 us, half as many 36 us), never more than a
// tile each asks for, and one per row when the rows alone are many.
int32_t score_splits(int64_t tokens, int64_t vocab, int num_cus, int32_t* part) {
  const int64_t tiles = div_up(vocab, kScoreTile);
  int64_t want = 4 * (int64_t)num_cus / std::max<int64_t>(tokens, 1);
  want = std::min<int64_t>({want, tiles, kScoreMaxSplits});
  if (tokens > kCounterBytes / (4 * kScoreCounterStride)) want = 1;
  // equal parts, whole cache lines: a part of a few logits more than its waves' tiles
  // takes as long as one of many
  *part = (int32_t)(div_up(div_up(vocab, std::max<int64_t>(want, 1)), kScoreAlign) * kScoreAlign);
  return (int32_t)div_up(vocab, *part);
}

w4a16_status score_workspace(int64_t tokens, int64_t vocab, int32_t top_k, int num_cus,
                             int64_t* bytes) {
  if (tokens < 0 || tokens > kMaxGrid || vocab < 1 || vocab > kMaxInt / 2)
    return report(W4A16_ERR_SHAPE, "need 0 <= tokens < 2^24 and 1 <= vocab <= 2^30");
  if (top_k < 0 || top_k > kScoreMaxTop || top_k > vocab)
    return report(W4A16_ERR_SHAPE, "top_k=%d must lie in 0..%d and not exceed the vocabulary",
                  (int)top_k, kScoreMaxTop);
  int32_t part;
  const int32_t splits = score_splits(tokens, vocab, num_cus, &part);
  *bytes = splits > 1 ? kCounterBytes + tokens * splits * score_part_bytes(top_k) : 0;
  return W4A16_OK;
}

// Most groups (sequence, row block, head) for which sequences are split, and
// the most scratch that the parts may take: beyond, the groups alone fill the
// device many times over.
constexpr int64_t kAttnMaxSplitGroups = 4096;
constexpr int64_t kAttnMaxParts = 256ll << 20;
static_assert(kAttnMaxSplitGroups <= kCounterBytes / 4, "one counter per group");

struct AttnShape {
  AttnKind kind;
  int rows, target, few;
  int64_t grid, workspace;
};

// Work items aimed at for `groups` on a device that holds `slots` workgroups.
// Few groups: as many as there are slots. More: whole rounds of slots cost
// whole rounds of time, so each group is split in the 1 to 4 that leaves the
// last round fullest, a split counted as 2 % (parts are written and joined).
// Measured in 4, 2 and 1: 640 groups on 512 slots, 2 x 1024 tokens over 16384
// bf16 715, 705 and 833 us, over int8 889, 908 and 1096; 1 x 2048 over 32768 1316,
// 1357 and 1623. Where the groups are of different lengths the rounds are not what
// this takes them for: 2 x 2048 tokens over themselves, e4m3, 227, 226 and 161.
int64_t attn_target(int64_t groups, int64_t slots) {
  if (groups <= slots) return slots;
  int64_t best = 1;
  double least = 1e30;
  for (int64_t s = 1; s <= 4; ++s) {
    const double time = (double)div_up(groups * s, slots) / (double)s * (1.0 + 0.02 * (double)(s - 1));
    if (time < least) {
      least = time;
      best = s;
    }
  }
  return groups * best;
}

w4a16_status attn_shape(int64_t sequences, int64_t max_q, int64_t q_heads, int64_t kv_heads,
                        int64_t dim, int num_cus, AttnShape* s) {
  if (sequences < 0 || max_q < 0 || sequences > (1 << 20) || max_q >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "need 0..2^20 sequences and 0 <= max_q < 2^31");
  if (kv_heads < 1 || kv_heads > 4096 || q_heads < 1 || q_heads > (1 << 16) ||
      q_heads % kv_heads != 0)
    return report(W4A16_ERR_SHAPE, "q_heads=%lld must be a multiple of the cache's %lld heads",
                  (long long)q_heads, (long long)kv_heads);
  const int64_t rows = max_q * (q_heads / kv_heads);
  if (rows >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "max_q times the heads of a group must be below 2^31");
  s->kind = attn_kind(rows, (int)dim);
  s->rows = attn_rows(s->kind);
  const int64_t groups = sequences * div_up(rows, s->rows) * kv_heads;
  const int64_t part = attn_part_floats(s->rows, attn_dim_block((int)dim)) * 4;
  // narrow items: 4 a CU (3 are resident; batches of mixed lengths end evener:
  // 32 x up to 8192 tokens 119.8 us, with 2 or 3 a CU 125); wide ones: 2, all resident
  const bool narrow = s->rows <= 32;
  s->target = (int)attn_target(groups, (narrow ? 4 : 2) * (int64_t)num_cus);
  s->few = narrow ? num_cus : s->target;
  if (groups > kAttnMaxSplitGroups || (groups + s->target) * part > kAttnMaxParts) s->target = 0;
  s->grid = groups + s->target;
  if (s->grid > kMaxGrid)
    return report(W4A16_ERR_SHAPE, "too many sequences, tokens and heads for one launch");
  s->workspace =
      s->target > 0 ? kCounterBytes + s->grid * part
                    : 0;
  return W4A16_OK;
}

w4a16_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return W4A16_OK;
  if (have < need)
    return report(W4A16_ERR_WORKSPACE, "the launch needs %lld bytes of workspace, %lld given",
                  (long long)need, (long long)have);
  if (!ws) return report(W4A16_ERR_NULL, "the launch needs a workspace and none was given");
  if (!aligned(ws, 16)) return report(W4A16_ERR_ALIGN, "workspace must be 16-byte aligned");
  return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

#define CHECK(call)                       \
  do {                                    \
    const w4a16_status st_ = (call);      \
    if (st_ != W4A16_OK) return st_;      \
  } while (0)

extern "C" {

w4a16_status w4a16_rope_frequencies(const w4a16_rope_scale_t* a, double* inv_freq) {
  if (!a || !inv_freq) return report(W4A16_ERR_NULL, "scale and inv_freq must be non-NULL");
  const int32_t r = a->rot_dim;
  if (r < 2 || r > 256 || r % 2 != 0)
    return report(W4A16_ERR_SHAPE, "rot_dim=%d must be even and in 2..256", (int)r);
  if (a->scaling < W4A16_ROPE_NONE || a->scaling > W4A16_ROPE_RAMP)
    return report(W4A16_ERR_VALUE, "scaling %d is not a w4a16_rope_scaling", (int)a->scaling);
  if (!(a->base > 1.0) || !std::isfinite(a->base))
    return report(W4A16_ERR_VALUE, "base must be finite and above 1");
  if (a->scaling != W4A16_ROPE_NONE && (!(a->factor >= 1.0) || !std::isfinite(a->factor)))
    return report(W4A16_ERR_VALUE, "factor must be finite and at least 1");
  if (a->scaling == W4A16_ROPE_NTK && r == 2)
    return report(W4A16_ERR_SHAPE, "NTK scaling needs rot_dim above 2");
  const bool turns = a->scaling == W4A16_ROPE_BANDS || a->scaling == W4A16_ROPE_RAMP;
  if (turns && (!(a->original > 0.0) || !std::isfinite(a->original) || !(a->low > 0.0) ||
                !(a->high > a->low) || !std::isfinite(a->high)))
    return report(W4A16_ERR_VALUE, "need original > 0 and 0 < low < high, all finite");
  const double kTwoPi = 6.283185307179586476925286766559;
  double base = a->base;
  if (a->scaling == W4A16_ROPE_NTK) base *= std::pow(a->factor, (double)r / (r - 2));
  // RAMP: the index at which the trained context makes `n` turns
  auto index_of = [&](double n) {
    return 0.5 * r * std::log(a->original / (n * kTwoPi)) / std::log(base);
  };
  double i0 = 0.0, i1 = 1.0;
  if (a->scaling == W4A16_ROPE_RAMP) {
    i0 = std::max(std::floor(index_of(a->high)), 0.0);
    i1 = std::min(std::ceil(index_of(a->low)), (double)(r - 1));
    if (!(i1 > i0)) i1 = i0 + 1e-3;  // no room between them: a step
  }
  for (int i = 0; i < r / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // share of the unscaled frequency
    if (a->scaling == W4A16_ROPE_LINEAR) keep = 0.0;
    if (a->scaling == W4A16_ROPE_BANDS)
      keep = (a->original * f / kTwoPi - a->low) / (a->high - a->low);
    if (a->scaling == W4A16_ROPE_RAMP) keep = 1.0 - (i - i0) / (i1 - i0);
    keep = std::min(std::max(keep, 0.0), 1.0);
    const bool scaled = a->scaling != W4A16_ROPE_NONE && a->scaling != W4A16_ROPE_NTK;
    inv_freq[i] = scaled ? keep * f + (1.0 - keep) * f / a->factor : f;
  }
  return W4A16_OK;
}

w4a16_status w4a16_rope_table(const double* inv_freq, int32_t rot_dim, double amplitude,
                              int64_t positions, float* table, void* stream) {
  if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2 != 0)
    return report(W4A16_ERR_SHAPE, "rot_dim=%d must be even and in 2..256", (int)rot_dim);
  if (positions < 0 || positions >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "need 0 <= positions < 2^31 (got %lld)", (long long)positions);
  if (!inv_freq) return report(W4A16_ERR_NULL, "inv_freq must be non-NULL");
  if (positions == 0) return W4A16_OK;
  if (!table) return report(W4A16_ERR_NULL, "table must be non-NULL");
  if (!aligned(table, 16)) return report(W4A16_ERR_ALIGN, "the table must be 16-byte aligned");
  int cus;
  CHECK(current_device(&cus));
  RopeTableParams p{};
  std::copy(inv_freq, inv_freq + rot_dim / 2, p.inv_freq);
  p.amplitude = amplitude;
  p.table = table;
  p.positions = positions;
  p.half = rot_dim / 2;
  return launched(launch_rope_table(p, (hipStream_t)stream));
}

w4a16_status w4a16_rope(const w4a16_rope_t* a, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  CHECK(check_dtype(a->dtype));
  CHECK(check_dim(a->head_dim));
  if (a->heads < 0) return report(W4A16_ERR_SHAPE, "heads must be >= 0");
  CHECK(check_count(a->tokens, std::max(a->heads, 1)));
  if (a->tokens == 0 || a->heads == 0) return W4A16_OK;
  if (!a->x || !a->out) return report(W4A16_ERR_NULL, "x and out must be non-NULL");
  CHECK(check_rotation(a->positions, a->table, a->table_rows, a->rot_dim, a->head_dim));
  if (!aligned(a->x, 16) || !aligned(a->out, 16))
    return report(W4A16_ERR_ALIGN, "x and out must be 16-byte aligned");
  CHECK(check_strides("x", a->x_token, a->x_head));
  CHECK(check_strides("out", a->out_token, a->out_head));
  CHECK(check_apart("out", a->tokens, a->out_token, a->heads, a->out_head, a->head_dim));
  if (a->x == a->out && (a->x_token != a->out_token || a->x_head != a->out_head))
    return report(W4A16_ERR_SHAPE, "in place, out needs x's strides");
  RopeKvParams p{};
  CHECK(shape_units(a->tokens, a->heads, a->head_dim, kRopeUnit, &p.per_unit, &p.units_per_token));
  int cus;
  CHECK(current_device(&cus));
  p.q = (const uint16_t*)a->x;
  p.q_out = (uint16_t*)a->out;
  p.positions = a->positions;
  p.table = a->table;
  p.q_token = a->x_token;
  p.q_head = a->x_head;
  p.out_token = a->out_token;
  p.out_head = a->out_head;
  p.table_rows = a->table_rows;
  p.tokens = (int32_t)a->tokens;
  p.hq = a->heads;
  p.dim = a->head_dim;
  p.rot = a->rot_dim;
  p.interleaved = a->interleaved != 0;
  p.inverse = a->inverse != 0;
  return launched(launch_rope_kv(p, a->dtype, W4A16_KV_SAME, (hipStream_t)stream));
}

w4a16_status w4a16_kv_write(const w4a16_kv_write_t* a, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  CHECK(check_dtype(a->dtype));
  KvView view;
  CHECK(check_cache(a->cache, &view));
  const int32_t hq = a->q ? a->q_heads : 0;
  if (hq < 0) return report(W4A16_ERR_SHAPE, "q_heads must be >= 0");
  CHECK(check_count(a->tokens, (int64_t)hq + 2 * a->cache.heads));
  if (a->tokens == 0) return W4A16_OK;
  if (!a->k || !a->v || !a->slots || (a->q && !a->q_out))
    return report(W4A16_ERR_NULL, "k, v, slots (and q_out with q) must be non-NULL");
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->slots, 8) ||
      (a->q && (!aligned(a->q, 16) || !aligned(a->q_out, 16))))
    return report(W4A16_ERR_ALIGN, "k, v, q and q_out must be 16-byte aligned, slots 8-byte");
  CHECK(check_strides("k", a->k_token, a->k_head));
  CHECK(check_strides("v", a->v_token, a->v_head));
  if (a->q) {
    CHECK(check_strides("q", a->q_token, a->q_head));
    CHECK(check_strides("q_out", a->out_token, a->out_head));
    CHECK(check_apart("q_out", a->tokens, a->out_token, hq, a->out_head, a->cache.head_dim));
    if (a->q == a->q_out && (a->q_token != a->out_token || a->q_head != a->out_head))
      return report(W4A16_ERR_SHAPE, "in place, q_out needs q's strides");
  }
  if (a->positions || a->table)
    CHECK(check_rotation(a->positions, a->table, a->table_rows, a->rot_dim, a->cache.head_dim));
  else if (a->q)
    return report(W4A16_ERR_NULL, "q is given to be rotated: positions and a table are needed");
  RopeKvParams p{};
  CHECK(shape_units(a->tokens, (int64_t)hq + 2 * view.heads, view.dim, kRopeUnit, &p.per_unit,
                    &p.units_per_token));
  int cus;
  CHECK(current_device(&cus));
  p.q = (const uint16_t*)a->q;
  p.k = (const uint16_t*)a->k;
  p.v = (const uint16_t*)a->v;
  p.q_out = (uint16_t*)a->q_out;
  p.positions = a->positions;
  p.slots = a->slots;
  p.table = a->table;
  p.cache = view;
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.k_token = a->k_token;
  p.k_head = a->k_head;
  p.v_token = a->v_token;
  p.v_head = a->v_head;
  p.out_token = a->out_token;
  p.out_head = a->out_head;
  p.table_rows = a->table_rows;
  p.tokens = (int32_t)a->tokens;
  p.hq = hq;
  p.hkv = a->cache.heads;
  p.dim = a->cache.head_dim;
  p.rot = a->rot_dim;
  p.interleaved = a->interleaved != 0;
  return launched(launch_rope_kv(p, a->dtype, a->cache.format, (hipStream_t)stream));
}

w4a16_status w4a16_kv_read(const w4a16_kv_read_t* a, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  CHECK(check_dtype(a->dtype));
  KvView view;
  CHECK(check_cache(a->cache, &view));
  CHECK(check_count(a->tokens, 2 * (int64_t)a->cache.heads));
  if (a->tokens == 0) return W4A16_OK;
  if (!a->slots || !a->k_out || !a->v_out)
    return report(W4A16_ERR_NULL, "slots, k_out and v_out must be non-NULL");
  if (!aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !aligned(a->slots, 8))
    return report(W4A16_ERR_ALIGN, "k_out and v_out must be 16-byte aligned, slots 8-byte");
  KvReadParams p{};
  CHECK(shape_units(a->tokens, 2 * (int64_t)view.heads, view.dim, kReadUnit, &p.per_unit, &p.units_per_token));
  int cus;
  CHECK(current_device(&cus));
  p.cache = view;
  p.slots = a->slots;
  p.k_out = (uint16_t*)a->k_out;
  p.v_out = (uint16_t*)a->v_out;
  p.tokens = (int32_t)a->tokens;
  return launched(launch_kv_read(p, a->dtype, a->cache.format, (hipStream_t)stream));
}

w4a16_status w4a16_tree_attention_workspace_bytes(int32_t sequences, int32_t max_q,
                                                  int32_t q_heads, int32_t kv_heads,
                                                  int32_t head_dim, int32_t num_cus,
                                                  int64_t* bytes) {
  if (!bytes) return report(W4A16_ERR_NULL, "bytes must be non-NULL");
  CHECK(check_dim(head_dim));
  AttnShape s;
  CHECK(attn_shape(sequences, max_q, q_heads, kv_heads, head_dim, num_cus > 0 ? num_cus : kWholeDevice, &s));
  *bytes = s.workspace;
  return W4A16_OK;
}

w4a16_status w4a16_tree_attention(const w4a16_tree_attention_t* a, void* workspace,
                                  int64_t ws_bytes, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  CHECK(check_dtype(a->dtype));
  KvView view;
  CHECK(check_cache(a->cache, &view));
  AttnShape s;
  CHECK(attn_shape(a->sequences, a->max_q, a->q_heads, view.heads, view.dim, kWholeDevice, &s));
  CHECK(check_count(a->tokens, a->q_heads));
  if (a->table_pages < 0 || a->table_stride < 0 || a->table_stride >= kMaxStride ||
      (a->table_stride < a->table_pages && a->table_stride != 0))
    return report(W4A16_ERR_SHAPE, "need 0 <= table_pages <= table_stride, or a stride of 0 (got %d, %lld)",
                  (int)a->table_pages, (long long)a->table_stride);
  // 32-bit counts of work: row blocks times steps of 128 tokens, over all heads
  const int64_t capacity = std::min<int64_t>((int64_t)a->table_pages * a->cache.page_size, kMaxInt - 1);
  const int64_t rows = (int64_t)a->max_q * (a->q_heads / view.heads);
  const double work = (double)a->sequences * (double)div_up(rows, s.rows) *
                      (double)view.heads * (double)(div_up(capacity, kAttnStep) + 1);
  if (work >= 2147483648.0)
    return report(W4A16_ERR_SHAPE, "sequences x new tokens x cached tokens too large for one launch");
  if (!std::isfinite(a->scale)) return report(W4A16_ERR_VALUE, "scale must be finite");
  if (a->tokens == 0 || a->sequences == 0 || a->max_q == 0) return W4A16_OK;
  if (a->mask && (a->mask_words < 1 || a->mask_words > (1 << 20)))
    return report(W4A16_ERR_SHAPE, "a mask needs 1..2^20 words a row (got %d)", (int)a->mask_words);
  if (!a->q || !a->out || !a->lse || !a->kv_lens || !a->q_starts ||
      (a->table_pages > 0 && !a->block_table))
    return report(W4A16_ERR_NULL, "q, out, lse, block_table, kv_lens and q_starts must be non-NULL");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->lse, 4) ||
      !aligned(a->block_table, 4) || !aligned(a->kv_lens, 4) || !aligned(a->q_starts, 4) ||
      !aligned(a->mask, 8))
    return report(W4A16_ERR_ALIGN, "q and out must be 16-byte aligned, the rest to its elements");
  CHECK(check_strides("q", a->q_token, a->q_head));
  int cus = kWholeDevice;
  const w4a16_status device = current_device(&cus);
  CHECK(attn_shape(a->sequences, a->max_q, a->q_heads, view.heads, view.dim, cus, &s));
  CHECK(check_workspace(workspace, ws_bytes, s.workspace));
  if (device != W4A16_OK) return device;
  AttnParams p{};
  p.cache = view;
  p.q = (const uint16_t*)a->q;
  p.out = (uint16_t*)a->out;
  p.lse = a->lse;
  p.block_table = a->block_table;
  p.kv_lens = a->kv_lens;
  p.q_starts = a->q_starts;
  p.mask = a->mask;
  if (s.target > 0) {
    p.counters = (int32_t*)workspace;
    p.parts = (float*)((char*)workspace + kCounterBytes);
  }
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.table_stride = a->table_stride;
  p.tokens = (int32_t)a->tokens;
  p.sequences = a->sequences;
  p.table_pages = a->table_pages;
  p.max_q = a->max_q;
  p.hq = a->q_heads;
  p.group = a->q_heads / view.heads;
  p.mask_words = a->mask_words;
  p.target = s.target;
  p.few = s.few;
  p.grid = (int32_t)s.grid;
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  using Launch = hipError_t (*)(const AttnParams&, AttnKind, hipStream_t);
  static constexpr Launch kLaunch[2][3] = {{attn_f16_same, attn_f16_e4m3, attn_f16_int8},
                                           {attn_bf16_same, attn_bf16_e4m3, attn_bf16_int8}};
  return launched(kLaunch[a->dtype][a->cache.format](p, s.kind, (hipStream_t)stream));
}

w4a16_status w4a16_token_logprobs_workspace_bytes(int64_t tokens, int64_t vocab, int32_t top_k,
                                                  int32_t num_cus, int64_t* bytes) {
  if (!bytes) return report(W4A16_ERR_NULL, "bytes must be non-NULL");
  return score_workspace(tokens, vocab, top_k, num_cus > 0 ? num_cus : kWholeDevice, bytes);
}

w4a16_status w4a16_token_logprobs(const w4a16_token_logprobs_t* a, void* workspace,
                                  int64_t ws_bytes, void* stream) {
  if (!a) return report(W4A16_ERR_NULL, "args must be non-NULL");
  if (a->dtype != W4A16_F32) {
    if (a->dtype != W4A16_F16 && a->dtype != W4A16_BF16)
      return report(W4A16_ERR_DTYPE, "dtype %d: fp16 (0), bf16 (1) and fp32 (2) are supported",
                    (int)a->dtype);
  }
  int64_t need;
  CHECK(score_workspace(a->tokens, a->vocab, a->top_k, kWholeDevice, &need));
  if (a->tokens == 0) return W4A16_OK;
  if (a->row_stride < 0 || a->row_stride >= kMaxStride)
    return report(W4A16_ERR_SHAPE, "row_stride must lie in 0..2^40");
  if (!a->logits || !a->ids || !a->logprobs || !a->entropy ||
      (a->top_k > 0 && (!a->top_logprobs || !a->top_ids)))
    return report(W4A16_ERR_NULL, "logits, ids and every output must be non-NULL");
  if (!aligned(a->logits, a->dtype == W4A16_F32 ? 4 : 2) || !aligned(a->ids, 8) ||
      !aligned(a->logprobs, 4) || !aligned(a->entropy, 4) || !aligned(a->top_logprobs, 4) ||
      !aligned(a->top_ids, 8))
    return report(W4A16_ERR_ALIGN, "arrays must be aligned to their elements");
  int cus = kWholeDevice;
  const w4a16_status device = current_device(&cus);
  CHECK(score_workspace(a->tokens, a->vocab, a->top_k, cus, &need));
  CHECK(check_workspace(workspace, ws_bytes, need));
  if (device != W4A16_OK) return device;
  ScoreParams p{};
  p.logits = a->logits;
  p.ids = a->ids;
  p.logprobs = a->logprobs;
  p.entropy = a->entropy;
  p.top_logprobs = a->top_logprobs;
  p.top_ids = a->top_ids;
  p.row_stride = a->row_stride;
  p.tokens = (int32_t)a->tokens;
  p.vocab = (int32_t)a->vocab;
  p.top_k = a->top_k;
  p.splits = score_splits(a->tokens, a->vocab, cus, &p.part);
  if (p.splits > 1) {
    p.counters = (int32_t*)workspace;
    p.parts = (char*)workspace + kCounterBytes;
  }
  return launched(launch_token_logprobs(p, a->dtype, (hipStream_t)stream));
}

}  // extern "C"
