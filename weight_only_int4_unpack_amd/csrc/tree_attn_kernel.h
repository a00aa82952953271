// Attention of new tokens (plain, or drafted as a tree) over a paged cache.
//
// Transposed products keep everything in registers. For a tile of 32 tokens
// and a block of 16 rows (row = new token x query head of one key/value head)
// a wave forms
//   S^T[token, row] = K Q^T    two 16x16 tiles, contraction over the dims
//   O^T[dim, row]  += V^T P^T  DB/16 tiles, contraction over the 32 tokens
// with v_mfma_f32_16x16x32. In S^T's accumulators lane (g, c) = (lane / 16,
// lane % 16) holds row c and tokens 4g..4g+3 of each half tile: exactly the 8
// contraction slots that the B operand of the second product wants from this
// lane, once slot 8g + 4u + i stands for token 16u + 4g + i. So weights go from
// one product into the next without leaving their lane, a row's maximum, sum
// and rescaling are per lane, and only joining the four lane groups shuffles.
//
// The A operands follow: K rows are read along the dims as they lie in memory
// (lane (g, c): token c, 16 bytes at dim chunk g). V is read in rows too.
//
// 8-bit codes are widened exactly to 16 bits; a token's scales multiply its
// scores and its weights, which are one value per lane and token. Weights times
// scales are held between bounds of fp16 by a power of two of each row's own.
//
// Two kernels share this, by the rows of a group (new tokens x query heads of a
// key/value head). Up to 32 rows (narrow): the four waves of a workgroup hold the
// same rows and take turns at the tokens, operands go from memory into
// registers, and the waves' sums are joined at the end: nothing waits for LDS,
// and every byte of the cache is read once. More rows (wide): each wave holds
// rows of its own, and the workgroup stages 64 tokens at a time in LDS for all
// four, since a wave that reads the cache alone feeds too few products.
#pragma once

#include <type_traits>

#include "serve_device.h"

namespace w4a16 {
namespace serve {

constexpr float kNegInf = -__builtin_inff();

template <typename T>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (T::kCode == W4A16_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The largest of eight; NaN where one is. (IEEE maximum: one instruction for
// three values, where fmaxf first quiets each product by one of its own.)
__device__ __forceinline__ float largest(f32x4 a, f32x4 b) {
  auto max3 = [](float x, float y, float z) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(x, y), z);
  };
  const float x = max3(a[0], a[1], a[2]), y = max3(a[3], b[0], b[1]);
  return __builtin_elementwise_maximum(max3(x, b[2], b[3]), y);
}

// Two fp32 as a 16-bit pair, rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pair(float lo, float hi) {
  if constexpr (T::kCode == W4A16_F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
  }
}

// Codes in the low (HI = false) or high half of a word as a 16-bit pair, exactly.
// int8 (fp16 only): u = code + 128 in the mantissa of 1024, then 1152 off.
template <typename T, int FMT, bool HI>
__device__ __forceinline__ uint32_t widen_pair(uint32_t w) {
  if constexpr (FMT == W4A16_KV_E4M3) {
    if constexpr (T::kCode == W4A16_F16)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  } else {
    static_assert(T::kCode == W4A16_F16, "int8 codes are widened to fp16");
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w ^ 0x80808080u,
                                             HI ? 0x04030402u : 0x04010400u);
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, u) -
                                            f16x2{(_Float16)1152.0f, (_Float16)1152.0f});
  }
}

// What a workgroup works on.
struct Item {
  int seq, head, block, split;   // block: row block
  int splits;                    // of this sequence
  int blocks;                    // row blocks of this sequence
  int chunk;                     // tokens of a split
  int len, prefix;               // tokens on pages of the table, and those of them that are before
                                 // the new ones (negative: some new ones are before the first)
  int news, start;               // new tokens that are computed (max_q at most), first row in q
  int group;                     // counter: (sequence, block, head)
  int first;                     // index of this group's split 0 among the items
};

// Sums over the lanes up to each one, without LDS: four steps inside rows of 16
// lanes, then the last lane of the first and third row, and of the second, added
// to the rows after it. Lanes that a step does not reach add 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lane_step(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int sum_upto(int x) {
  x = lane_step<0x111, 0xF>(x);           // row_shr 1, 2, 4, 8
  x = lane_step<0x112, 0xF>(x);
  x = lane_step<0x114, 0xF>(x);
  x = lane_step<0x118, 0xF>(x);
  x = lane_step<0x142, 0xA>(x);           // row_bcast 15, 31
  return lane_step<0x143, 0xC>(x);
}

// Finds work item `index`: every wave scans the sequences, 64 at a time, each
// lane one, twice over (the total sets the chunk length, then the item counts
// are summed up to the item). Lengths live on the device, so that a captured
// launch follows them; splits follow the total work, so that one long
// sequence among short ones is still spread over the device.
template <int ROWS>
__device__ __forceinline__ bool find_item(const AttnParams& p, int index, Item* it) {
  const int lane = threadIdx.x & 63;
  const int most = p.cache.pages > 0 ? min((int64_t)p.table_pages << p.cache.page_shift,
                                           (int64_t)0x7FFFFF00) : 0;
  auto load = [&](int b, int* len, int* prefix, int* news, int* start, int* blocks) {
    *len = *prefix = *news = *start = *blocks = 0;
    if (b < p.sequences) {
      const int whole = max(p.kv_lens[b], 0);
      *len = min(whole, most);
      const int s0 = min(max(p.q_starts[b], 0), p.tokens);
      const int s1 = min(max(p.q_starts[b + 1], s0), p.tokens);
      *start = s0;
      *prefix = min(whole - (s1 - s0), *len);
      *news = min(s1 - s0, p.max_q);
      *blocks = (*news * p.group + ROWS - 1) / ROWS;
    }
  };
  int len, prefix, news, start, blocks;
  uint32_t steps = 0;
  const bool one_round = p.sequences <= 64;
  for (int b0 = 0; b0 < p.sequences; b0 += 64) {
    load(b0 + lane, &len, &prefix, &news, &start, &blocks);
    steps += (uint32_t)blocks * (uint32_t)((len + kAttnStep - 1) / kAttnStep);
  }
  steps = (uint32_t)__builtin_amdgcn_readlane(sum_upto((int)steps), 63);
  uint32_t per = 0x7FFFFFFF / kAttnStep;   // steps of a split
  if (p.target > 0) {
    const uint32_t work = steps * (uint32_t)p.cache.heads;
    per = (work + p.target - 1) / (uint32_t)p.target;
    per = max(max(per, min((work + p.few - 1) / (uint32_t)p.few, (uint32_t)kAttnFewSteps)), 1u);
  }
  int items_before = 0, groups_before = 0;
  for (int b0 = 0; b0 < p.sequences; b0 += 64) {
    if (!one_round) load(b0 + lane, &len, &prefix, &news, &start, &blocks);
    const uint32_t mine = (uint32_t)(len + kAttnStep - 1) / kAttnStep;
    uint32_t own = per;
    if (p.target > 0) own = max(own, (mine + kAttnMaxSplits - 1) / kAttnMaxSplits);
    const int splits = max((int)((mine + own - 1) / own), 1);
    const int groups = blocks * p.cache.heads, items = groups * splits;
    const int upto = sum_upto(items), gupto = sum_upto(groups);
    const uint64_t past = __ballot(items_before + upto > index);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      // into scalar registers: everything below is the same for all lanes
      auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
      it->seq = b0 + l;
      it->splits = of(splits);
      it->blocks = of(blocks);
      it->chunk = min(of((int)own), 0x7FFFFF00 / kAttnStep) * kAttnStep;
      it->len = of(len);
      it->prefix = of(prefix);
      it->news = of(news);
      it->start = of(start);
      const int local = index - (items_before + of(upto - items));
      // heads innermost: workgroups go round the 8 XCDs, so with 8 heads the
      // row blocks that share a head's keys and values share an L2
      it->head = local % p.cache.heads;
      const int rest = local / p.cache.heads;
      it->block = it->blocks - 1 - rest % it->blocks;  // causal: the longest first
      it->split = rest / it->blocks;
      it->group = groups_before + of(gupto - groups) + it->block * p.cache.heads + it->head;
      it->first = index - it->split * it->blocks * p.cache.heads;  // + split * blocks * heads
      return true;
    }
    items_before += __builtin_amdgcn_readlane(upto, 63);
    groups_before += __builtin_amdgcn_readlane(gupto, 63);
  }
  return false;
}

// Four dims from d0 of a finished row: o / z, and (with d0 = 0) the row's lse.
// The held maximum m is in log2, and z was summed `lift` above it.
template <typename T>
__device__ __forceinline__ void finish4(const AttnParams& p, const Item& it, int row, int d0, int dim,
                                        float m, float z, float lift, f32x4 o) {
  const int query = row / p.group, head = it.head * p.group + row - query * p.group;
  const int64_t at = (int64_t)(it.start + query) * p.hq + head;
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
  if (d0 < dim)
    *(u32x2*)(p.out + at * dim + d0) = u32x2{pair<T>(o[0] * inv, o[1] * inv),
                                             pair<T>(o[2] * inv, o[3] * inv)};
  if (d0 == 0)
    p.lse[at] = z == 0.0f ? kNegInf : 0.69314718055994530942f * (m - lift + __log2f(z));
}

// Types of the two products. 8-bit codes are multiplied by fp16 weights
// whatever the activations are (2^-11 instead of bf16's 2^-8 per weight), and
// int8 ones by fp16 queries (bf16 queries are scaled by a power of two per row
// into fp16's range first: what that drops is below 2^-39 of the row's largest).
constexpr float kSlack = 8.0f;  // how far (log2) a score may exceed the held maximum
template <typename T, int FMT>
struct Types {
  using K = typename std::conditional<FMT == W4A16_KV_INT8, F16, T>::type;
  using P = typename std::conditional<FMT == W4A16_KV_SAME, T, F16>::type;
  static constexpr bool kSame = FMT == W4A16_KV_SAME;
  static constexpr bool kRescaleQ = FMT == W4A16_KV_INT8 && T::kCode == W4A16_BF16;
  // fp16 weights are held 2^6 above 1, at most 2^14, so that the small ones
  // stay above fp16's subnormals (2^-14) down to 2^-20 of the largest. Those
  // that meet a scale first are at most 1 (no product overflows), and the
  // products are held between the same bounds by a reference of their own.
  static constexpr float kLift = !kSame ? -kSlack : P::kCode == W4A16_F16 ? 6.0f : 0.0f;
};
constexpr float kHeldMost = 0x1p15f;   // weight x scale in units of its reference,
constexpr float kHeldLeast = 0x1p6f;   // and the largest when that has just been set
constexpr float kMostUnit = 0x1p126f;
// A positive normal number's power of two, and a power of two's reciprocal.
__device__ __forceinline__ float power_of(float x) { return __uint_as_float(__float_as_uint(x) & 0x7F800000u); }
__device__ __forceinline__ float over_power(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

// 16-bit values: 1, the exponent's mask (all ones: infinity or NaN), and, for a
// word of two, the halves that are such (as masks), and 1 in each half of a kind.
template <typename T>
constexpr uint32_t kOne16 = T::kCode == W4A16_F16 ? 0x3C00u : 0x3F80u;
template <typename T>
constexpr uint32_t kExp16 = T::kCode == W4A16_F16 ? 0x7C00u : 0x7F80u;
template <typename T>
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
  return ((x & kExp16<T>) == kExp16<T> ? 0xFFFFu : 0u) |
         (((x >> 16) & kExp16<T>) == kExp16<T> ? 0xFFFF0000u : 0u);
}
template <typename T>
__device__ __forceinline__ uint32_t ones_where(uint32_t x, int kind) {
  auto is = [&](uint32_t h) {
    return kind == 0 ? h == kExp16<T> : kind == 1 ? h == (kExp16<T> | 0x8000u) : (h & 0x7FFFu) > kExp16<T>;
  };
  return (is(x & 0xFFFFu) ? kOne16<T> : 0u) | (is(x >> 16) ? kOne16<T> << 16 : 0u);
}
__device__ __forceinline__ bool nan_codes(uint32_t y) {  // of e4m3: seven ones
  return (((y & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// A wave's rows: R blocks of 16, lane (g, c) holding row c of each.
// ROWS16: tile j of O^T holds dims 16 j.. (else dims j, j + kVD, ...).
template <typename T, int FMT, int DB, int R, bool ROWS16>
struct Rows {
  using TY = Types<T, FMT>;
  static constexpr int kSteps = DB / 32;  // contraction steps of S^T
  static constexpr int kVD = DB / 16;     // tiles of O^T, and dims of V per lane
  u32x4 q[R][kSteps];
  f32x4 acc[R][kVD];
  float factor[R];                        // of the scores: scale, log2(e), the row's rescaling
  float top[R], total[R];                 // held maximum (log2) and this lane's sum of weights
  int query[R];                           // new token of the row
  // Power of two by which the row's weights x scales are held, set by what the row
  // sees and weighs: another row's tokens, however large, cost this one no bits. (A
  // reference for all rows of a wave, by the scales alone: 512 tokens over 8192 e4m3
  // 273 us instead of 279, and rows wiped out by a large value that they do not see.)
  float unit[R];
  float held_most[R];                     // log2 of the scores' factor x scale that reaches kHeldMost
  int start, prefix, len;

  // `row0`: the wave's first row. `stop`: no token from there on exists or (without a mask
  // of its own, as sees() is one) is seen by a row. `dim_of(s)`:
  // dims of contraction step s.
  template <typename DimOf>
  __device__ __forceinline__ void init(const AttnParams& p, const Item& it, int row0, int stop, int dim,
                                       DimOf dim_of) {
    const int c = threadIdx.x & 15;
    start = it.start;
    prefix = it.prefix;
    len = stop;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      unit[r] = kMostUnit;
      held_most[r] = kNegInf;
      const int row = min(row0 + 16 * r + c, it.news * p.group - 1);
      query[r] = row / p.group;
      const uint16_t* src = p.q + (int64_t)(it.start + query[r]) * p.q_token +
                            (int64_t)(it.head * p.group + row - query[r] * p.group) * p.q_head;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d = dim_of(s);
        q[r][s] = u32x4{0, 0, 0, 0};
        if (d < dim) q[r][s] = load16(src + d);
        // the largest score is the largest product times a factor >= 0
        if (p.scale_log2 < 0.0f) q[r][s] ^= 0x80008000u;
      }
      factor[r] = fabsf(p.scale_log2);
      top[r] = kNegInf;
      total[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < kVD; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
      if constexpr (TY::kRescaleQ) {
        uint32_t big = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const f32x8 x = widen8<T>(q[r][s]);
#pragma unroll
          for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        }
        big = max(big, (uint32_t)__shfl_xor((int)big, 16));
        big = max(big, (uint32_t)__shfl_xor((int)big, 32));
        // largest magnitude into [2^14, 2^15); zero, subnormal and non-finite rows as they are
        const int e = (int)(big >> 23) - 127;
        const bool some = big >= 0x00800000u && big < 0x7F800000u;
        const int by = some ? min(14 - e, 126) : 0;
        const float up = ldexpf(1.0f, by);
        factor[r] = ldexpf(factor[r], -by);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[r][s] = narrow8<F16>(widen8<T>(q[r][s]) * up);
      }
    }
  }

  // Waits for the loads of init(): left to the compiler, that wait would sit in
  // the token loop and hold up each pass for the loads of the next one.
  __device__ __forceinline__ void settle() {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }

  // Which of the tile's tokens that exist this lane's row r sees: bit 4u + i for token
  // 16u + 4g + i. The row's 32 bits of the mask lie in two words, loaded together
  // (one load a token cost a drafted tree 10 us).
  __device__ __forceinline__ uint32_t sees(const AttnParams& p, int r, int t0) const {
    const int g = (threadIdx.x & 63) >> 4;
    const int j0 = t0 - prefix;           // the first token among the new ones, if >= 0
    uint32_t bits;
    if (p.mask == nullptr) {
      const int upto = query[r] - j0 + 1; // tokens of the tile up to the row's own
      bits = upto >= 32 ? ~0u : upto <= 0 ? 0u : (1u << upto) - 1;
    } else {
      const uint64_t* row = p.mask + (int64_t)(start + query[r]) * p.mask_words;
      const int at = j0 >> 6, by = j0 & 63;
      const uint64_t a = row[min(max(at, 0), p.mask_words - 1)];
      const uint64_t b = row[min(max(at + 1, 0), p.mask_words - 1)];
      auto word = [&](int i, uint64_t x) { return i < 0 ? ~0ull : i < p.mask_words ? x : 0ull; };
      bits = (uint32_t)(word(at, a) >> by | (by > 0 ? word(at + 1, b) << (64 - by) : 0ull));
    }
    return ((bits >> (4 * g)) & 0xFu) | ((bits >> (16 + 4 * g)) & 0xFu) << 4;
  }

  // One tile of 32 tokens from t0. k_op(u, i): operand of half tile u and step
  // i; k_scale(u), v_scale(u): scales of this lane's 4 tokens; after(): called
  // once the K operands are consumed; v_op(j): operand of O^T's tile j. EDGE: some
  // token may be unseen by some row; without TREE none is unseen before `len`.
  // exists[u]: half tile u lies on a page. v_edge(in): lets the caller clear V of
  // tokens that do not exist (bit 4u + i of `in`: this lane's token does) and say
  // (uniform) whether V holds an infinity or NaN.
  template <bool EDGE, bool TREE, typename KOp, typename KScale, typename After, typename VEdge,
            typename VScale, typename VOp, typename Fresh>
  __device__ __forceinline__ void tile(const AttnParams& p, int t0, const bool* exists,
                                       KOp k_op, KScale k_scale, After after, VEdge v_edge,
                                       VScale v_scale, VOp v_op, Fresh fresh) {
    const int g = (threadIdx.x & 63) >> 4;
    // ---- S^T, times the tokens' scales; factor[r] makes it units of log2
    f32x4 s[R][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r) s[r][u] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const u32x4 a = k_op(u, i);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][u] = mfma16<typename TY::K>(a, q[r][i], s[r][u]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        if constexpr (!TY::kSame) s[r][u] *= k_scale(u);
    }
    after();

    // ---- what a row does not see: score -inf (and, below, weight 0)
    uint32_t seen[R], in_all = 0xFF;      // bit 4u + i: this lane's token (u, i)
    bool apart = false;
    if constexpr (EDGE) {
      in_all = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int left = exists[u] ? min(max(len - (t0 + 16 * u + 4 * g), 0), 4) : 0;
        in_all |= ((1u << left) - 1) << (4 * u);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        seen[r] = in_all;
        if constexpr (TREE) seen[r] &= sees(p, r, t0);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[r][u][i] = (seen[r] >> (4 * u + i)) & 1 ? s[r][u][i] : kNegInf;
      }
      apart = v_edge(in_all) && TREE;
    }

    // ---- the held maximum rises only when a score exceeds it by 2^8
    // Nor, in front of 8-bit codes, does a weight x scale reach fp16's end: a lane's
    // largest score and largest scale bound its products. Where they do not (or a scale
    // is negative, infinite or NaN, above all others as an integer) the products tell.
    bool rise = false;
    float high[R];
    f32x4 vs[2];
    float scale_log2 = 0.0f;
    if constexpr (!TY::kSame) {
      uint32_t big = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        vs[u] = v_scale(u);
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(vs[u][i]));
      }
      rise = big > 0x7F7FFFFFu;
      scale_log2 = __builtin_amdgcn_logf(__uint_as_float(big));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      high[r] = largest(s[r][0], s[r][1]) * factor[r];
      rise |= high[r] > top[r] + kSlack;
      if constexpr (!TY::kSame) rise |= high[r] + scale_log2 > held_most[r];
    }
    const auto seen_by = [&](int r, int u, int i) { return !EDGE || ((seen[r] >> (4 * u + i)) & 1); };
    // 0 where unseen, whatever -inf times a factor of 0 and NaN scales make of it
    const auto weight = [&](int r, int u, int i, float ref) {
      const float x = __builtin_amdgcn_exp2f(fmaf(s[r][u][i], factor[r], -ref));
      return seen_by(r, u, i) ? x : 0.0f;
    };
    const auto ref_of = [&](int r) { return (top[r] == kNegInf ? 0.0f : top[r]) - TY::kLift; };
    if (__any(rise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float m = fmaxf(high[r], __shfl_xor(high[r], 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        m = fmaxf(m, top[r]);
        const float f = top[r] == m ? 1.0f : __builtin_amdgcn_exp2f(top[r] - m);
        top[r] = m;
        total[r] *= f;
        float held = f;
        if constexpr (!TY::kSame) {       // the reference sinks with the old weights
          const float old = over_power(unit[r]) * f, ref = ref_of(r);
          float most = 0.0f;              // the largest finite product
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y = seen_by(r, u, i) ? fabsf(weight(r, u, i, ref) * vs[u][i]) : 0.0f;
              most = y < __builtin_inff() ? fmaxf(most, y) : most;
            }
          most = fmaxf(most, __shfl_xor(most, 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          const float sunk = fmaxf(power_of(old), 1.0f / kMostUnit);
          const float to = most > sunk * kHeldMost ? power_of(most) * (1.0f / kHeldLeast) : sunk;
          unit[r] = over_power(to);
          // (opaque: what the compiler knows of it made it copy all sums on the common path)
          asm("" : "+v"(unit[r]));
          held = old * unit[r];
          held_most[r] = ref + __builtin_amdgcn_logf(to * kHeldMost);
        }
#pragma unroll
        for (int j = 0; j < kVD; ++j) acc[r][j] *= held;
      }
    }

    // ---- weights
    u32x4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ref = ref_of(r);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = weight(r, u, i, ref);
          total[r] += x[i];
          if constexpr (!TY::kSame) x[i] = seen_by(r, u, i) ? x[i] * vs[u][i] * unit[r] : 0.0f;
        }
        w[r][2 * u] = pair<typename TY::P>(x[0], x[1]);
        w[r][2 * u + 1] = pair<typename TY::P>(x[2], x[3]);
      }
    }

    // ---- O^T
    // kRare: told that this is rare, the compiler spills there and not in the token loop
    // (512 tokens over 8192 e4m3 126 us, else 165; 64 trees of 6 over 4000 e4m3 82, else
    // 97), but for the narrow kernels of 16-bit caches (16 trees of 4 over 4000 40, with
    // it 51).
    constexpr bool kRare = ROWS16 || !TY::kSame;
    const bool usual = !TREE || !apart;
    if (kRare ? __builtin_expect(usual, 1) : usual) {
#pragma unroll
      for (int j = 0; j < kVD; ++j) {
        const u32x4 a = v_op(j);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][j] = mfma16<typename TY::P>(a, w[r], acc[r][j]);
      }
    } else {
      // Infinities or NaN among values that some rows may not see: the product
      // takes 0 in their place, and three products of ones tell which sums they
      // reach. fresh(): operands from here on are formed anew, not for both branches.
      fresh();
      u32x4 sees_it[R];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sees_it[r][e] = ((seen[r] >> (2 * e)) & 1 ? kOne16<typename TY::P> : 0u) |
                          ((seen[r] >> (2 * e + 1)) & 1 ? kOne16<typename TY::P> << 16 : 0u);
#pragma unroll
      for (int j = 0; j < kVD; ++j) {
        u32x4 a = v_op(j), finite;
#pragma unroll
        for (int e = 0; e < 4; ++e) finite[e] = a[e] & ~odd_halves<typename TY::P>(a[e]);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][j] = mfma16<typename TY::P>(finite, w[r], acc[r][j]);
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {  // +inf, -inf, NaN
          u32x4 at;
#pragma unroll
          for (int e = 0; e < 4; ++e) at[e] = ones_where<typename TY::P>(a[e], kind);
          const float value = kind == 0 ? __builtin_inff() : kind == 1 ? kNegInf : __builtin_nanf("");
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const f32x4 n = mfma16<typename TY::P>(at, sees_it[r], f32x4{0, 0, 0, 0});
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][j][i] += n[i] > 0.0f ? value : 0.0f;
          }
        }
      }
    }
  }

  // This row's sum of weights over all lane groups.
  __device__ __forceinline__ float denominator(int r) const {
    float z = total[r] + __shfl_xor(total[r], 16);
    return z + __shfl_xor(z, 32);
  }
  // Puts the sums of row c of block r into a row of DB floats, V's reference put back.
  __device__ __forceinline__ void put_row(float* row, int r) const {
    const int g = (threadIdx.x & 63) >> 4;
    const float back = TY::kSame ? 1.0f : over_power(unit[r]);
    if constexpr (ROWS16) {
#pragma unroll
      for (int j = 0; j < kVD; ++j) *(f32x4*)(row + 16 * j + 4 * g) = acc[r][j] * back;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kVD; j += 4)
          *(f32x4*)(row + (4 * g + i) * kVD + j) =
              f32x4{acc[r][j][i], acc[r][j + 1][i], acc[r][j + 2][i], acc[r][j + 3][i]} * back;
    }
  }
};

// Tokens [begin, end) of an item, the first that some row of it may not see, and the
// first from which on none sees any.
struct Range {
  int begin, end, see_all, stop;
};
__device__ __forceinline__ Range range_of(const AttnParams& p, const Item& it, int row0, int rows) {
  const int last = (min(row0 + rows, it.news * p.group) - 1) / p.group;
  Range r;
  r.see_all = p.mask ? it.prefix : it.prefix + row0 / p.group + 1;
  r.stop = max(p.mask ? it.len : min(it.len, it.prefix + last + 1), 0);
  r.begin = it.split * it.chunk;
  r.end = (int)min((int64_t)r.begin + it.chunk, (int64_t)r.stop);
  return r;
}

// The item's row of the block table, and the first row (of head_dim values, or of
// scales) of a token for the item's head. Scalar arithmetic in 32 bits where it
// can be: there is no scalar comparison of 64 bits, and the lookups are a part of
// each pass that nothing hides.
struct Pages {
  // the constant address space: nothing writes the table while the kernel runs,
  // so the loads may be scalar ones, apart from the vector loads' counter
  typedef const __attribute__((address_space(4))) int32_t* Table;
  Table table;
  uint32_t pages;
  int shift, last, heads, head, len;
  __device__ __forceinline__ Pages(const AttnParams& p, const Item& it)
      : table((Table)(p.block_table + it.seq * p.table_stride)),
        pages((uint32_t)min(p.cache.pages, (int64_t)0x7FFFFFFF)),
        shift(p.cache.page_shift),
        last(it.len - 1),
        heads(p.cache.heads),
        head(it.head),
        len(it.len) {}
  // The page of token t (uniform; past the end, of the last token).
  __device__ __forceinline__ int of(int t) const { return table[(uint32_t)min(t, last) >> shift]; }
  __device__ __forceinline__ bool there(int page, int t) const {
    return (uint32_t)page < pages && t < len;
  }
  // Row 0 of page 0 where the token is not there.
  __device__ __forceinline__ int64_t row(int page, int t, bool there) const {
    return (((int64_t)(there ? page : 0) * heads + head) << shift) + (t & ((1 << shift) - 1));
  }
};

// The parts, as a bounded buffer. A part's rows (DB floats each), then their
// statistics (maximum, denominator). Stores are written through to the device's
// point of coherence and loads read there (sc1), 16 bytes a lane and 256
// contiguous ones for the 16 lanes of a row; the wait and the counter in
// arrive() order them.
struct Parts {
  __amdgpu_buffer_rsrc_t buffer;
  static constexpr int kSc1 = 16;
  __device__ __forceinline__ Parts(const AttnParams& p, int part_floats)
      : buffer(__builtin_amdgcn_make_buffer_rsrc(p.parts, 0, p.grid * part_floats * 4, 0x00020000)) {}
  __device__ __forceinline__ void put4(uint32_t at, f32x4 x) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), buffer, (int)(4 * at), 0, kSc1);
  }
  __device__ __forceinline__ void put2(uint32_t at, float a, float b) const {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{a, b}), buffer, (int)(4 * at),
                                          0, kSc1);
  }
  __device__ __forceinline__ f32x4 get4(uint32_t at) const {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(buffer, (int)(4 * at), 0, kSc1));
  }
  __device__ __forceinline__ f32x2 get2(uint32_t at) const {
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(buffer, (int)(4 * at), 0, kSc1));
  }
};

// Whether this workgroup is the last of its group's splits to arrive.
__device__ __forceinline__ bool arrive(const AttnParams& p, const Item& it, int* flag) {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);     // vmcnt(0): this wave's stores are complete
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before = __hip_atomic_fetch_add(p.counters + it.group, 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
    *flag = before == it.splits - 1;
    if (before == it.splits - 1)
      __hip_atomic_store(p.counters + it.group, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool last = *flag != 0;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  return last;
}

// The last workgroup of a group joins its parts, in an order that does not
// depend on who arrived when. 16 lanes hold a row (dims 64 h + 4 lane..); with
// fewer than 9 rows several such lane rows share a row's splits, and are joined
// through `lds` (16 rows of DB + 4 floats).
template <typename T, int DB, int ROWS>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Item& it, int rows, int dim,
                                           float lift, float* lds) {
  constexpr int kH = DB / 64, kPad = DB + 4;
  constexpr int kPart = (int)attn_part_floats(ROWS, DB);
  constexpr int kDeep = 16 / kH;          // parts in flight
  const Parts parts(p, kPart);
  const int slot = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  const uint32_t stride = (uint32_t)(it.blocks * p.cache.heads) * kPart;
  const uint32_t first = (uint32_t)it.first * kPart;
  rows = min(rows, ROWS);
  const int held = min(rows, 16);         // rows at a time
  const int share = 16 / held, lead = slot / held;
  for (int at0 = 0; at0 < rows; at0 += held) {
    const int at = at0 + slot - lead * held;
    const uint32_t base = first + at * DB + 4 * l16, stats = first + ROWS * DB + 2 * at;
    float m = kNegInf, z = 0.0f;
    f32x4 o[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) o[h] = f32x4{0, 0, 0, 0};
    if (at < rows && lead < share) {
#pragma unroll 1
      for (int s0 = lead; s0 < it.splits; s0 += share * kDeep) {
        f32x2 st[kDeep];
        f32x4 x[kDeep][kH];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {  // past the last split: that one again, not counted
          const uint32_t off = (uint32_t)min(s0 + d * share, it.splits - 1) * stride;
          st[d] = parts.get2(stats + off);
#pragma unroll
          for (int h = 0; h < kH; ++h) x[d][h] = parts.get4(base + off + 64 * h);
        }
        float big = m;
#pragma unroll
        for (int d = 0; d < kDeep; ++d) big = fmaxf(big, st[d].x);
        const float f0 = m == big ? 1.0f : __builtin_amdgcn_exp2f(m - big);
        m = big;
        z *= f0;
#pragma unroll
        for (int h = 0; h < kH; ++h) o[h] *= f0;
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
          if (s0 + d * share < it.splits) {
            const float f = st[d].x == m ? 1.0f : __builtin_amdgcn_exp2f(st[d].x - m);
            z = fmaf(f, st[d].y, z);
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[h][e] = fmaf(f, x[d][h][e], o[h][e]);
          }
      }
    }
    if (share > 1) {                      // the same in the whole workgroup
      __syncthreads();
      float* mine = lds + slot * kPad;
#pragma unroll
      for (int h = 0; h < kH; ++h) *(f32x4*)(mine + 64 * h + 4 * l16) = o[h];
      if (l16 == 0) {
        mine[DB] = m;
        mine[DB + 1] = z;
      }
      __syncthreads();
      if (lead == 0) {
        float big = m;
        for (int s = 1; s < share; ++s) big = fmaxf(big, lds[(slot + s * held) * kPad + DB]);
        const float f0 = m == big ? 1.0f : __builtin_amdgcn_exp2f(m - big);
        m = big;
        z *= f0;
#pragma unroll
        for (int h = 0; h < kH; ++h) o[h] *= f0;
        for (int s = 1; s < share; ++s) {
          const float* other = lds + (slot + s * held) * kPad;
          const float f = other[DB] == big ? 1.0f : __builtin_amdgcn_exp2f(other[DB] - big);
          z = fmaf(f, other[DB + 1], z);
#pragma unroll
          for (int h = 0; h < kH; ++h) o[h] += f * *(const f32x4*)(other + 64 * h + 4 * l16);
        }
      }
    }
    if (lead == 0 && at < rows)
#pragma unroll
      for (int h = 0; h < kH; ++h)
        finish4<T>(p, it, it.block * ROWS + at, 64 * h + 4 * l16, dim, m, z, lift, o[h]);
  }
}

// ---------------------------------------------------------------- few rows
// Lane (g, c) reads V of its 8 tokens, dims c * DB/16 .. +DB/16, so that a row of
// the page is one contiguous run over 16 lanes; one byte permute joins two
// tokens' values of a dim into an operand word, and tile j of O^T holds dims
// c * DB/16 + j. A tile's loads are issued one tile ahead, its pages two.
//
// Bound by HBM where there is enough to read: 64 sequences of up to 8192 tokens,
// 8 heads of 128 in e4m3, 117 us (4.7 TB/s; a copy reaches 5.2); 32 such in bf16
// 108 us (5.1 TB/s). With little to read the chain of launch, item search, a
// few tiles, parts and their join: 4099 tokens of one sequence 11.7 us, of which
// the bytes are 3, and 57 % of the waves' time is waits. Partial head dims above 128
// over a 16-bit cache spill in the token loop: 32 sequences, 4 heads of 192, 142 us
// (2.9 TB/s), of 256 117 us (4.7).
//
// Without TREE (one row of new tokens per sequence and no mask) the kernel needs no
// masks but the length's, and its registers leave room for three waves per
// SIMD instead of two (16 rows, up to 128 dims).
//
// With TREE, 32 rows of 128 dims and a 16-bit cache, two waves a SIMD would spill in
// the token loop: one wave with twice the registers takes 30 instead of 38 us (8
// tokens of one sequence over 16384, bf16), 49 instead of 65 (16 trees over 4000).
// 16 rows of 256 dims as well: 36 instead of 48, and 51 instead of 67.
constexpr int narrow_waves(int fmt, int db, int r, bool tree) {
  return !tree && r * db <= 128 ? 3 : tree && r * db == 256 && fmt == W4A16_KV_SAME ? 1 : 2;
}
template <typename T, int FMT, int DB, int R, bool FULL, bool TREE>
__global__ __launch_bounds__(64 * kAttnWaves, narrow_waves(FMT, DB, R, TREE)) void attn_narrow_kernel(
    AttnParams p) {
  using TY = Types<T, FMT>;
  constexpr bool kSame = TY::kSame;
  constexpr int kRows = 16 * R;
  constexpr int kVD = DB / 16;
  constexpr int kBytes = kSame ? 2 : 1;
  constexpr int kVWords = kVD * kBytes / 4;    // words of a token's V per lane
  constexpr int kKLoads = DB * kBytes / 64;    // 16-byte loads of K per half tile
  constexpr int kPad = DB + 4;

  __shared__ float l_sum[kAttnWaves][16][kPad];
  __shared__ f32x2 l_stat[kAttnWaves][16];
  __shared__ int l_last;

  Item it;
  if (!find_item<kRows>(p, blockIdx.x, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int dim = FULL ? DB : p.cache.dim;
  const int row0 = it.block * kRows;
  const int rows = it.news * p.group - row0;   // of this block, may exceed kRows
  const Range range = range_of(p, it, row0, kRows);
  const int tiles = range.end > range.begin ? (range.end - range.begin + kAttnTile - 1) / kAttnTile : 0;

  const char* kbase = (const char*)p.cache.k;
  const char* vbase = (const char*)p.cache.v;
  const int row_bytes = dim * kBytes;

  u32x4 kreg[2][kKLoads];
  uint32_t vreg[2][4][kVWords];
  f32x4 kscale[2], vscale[2];
  int64_t at[2];                               // rows of the next tile's half tiles
  bool ok[2] = {false, false};

  const Pages table(p, it);
  int pages[2];
  auto look_up = [&](int n) {                  // two tiles ahead: scalar loads, never waited for
#pragma unroll
    for (int u = 0; u < 2; ++u) pages[u] = table.of(range.begin + n * kAttnTile + 16 * u);
  };
  auto take_rows = [&](int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = range.begin + n * kAttnTile + 16 * u;
      ok[u] = table.there(pages[u], t);
      at[u] = table.row(pages[u], t, ok[u]);
    }
  };
  auto load_k = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char* src = kbase + at[u] * row_bytes;  // uniform; lanes add 32-bit offsets
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) {
        const int d = i * (64 / kBytes) + g * (16 / kBytes);
        if constexpr (FULL) {
          kreg[u][i] = load16(src + (uint32_t)(c * row_bytes + d * kBytes));
        } else {                               // dims past the head's: zeros
          const bool in = d < dim;
          const u32x4 x = load16(src + (uint32_t)(c * row_bytes + (in ? d : 0) * kBytes));
          kreg[u][i] = in ? x : u32x4{0, 0, 0, 0};
        }
      }
      if constexpr (!kSame) kscale[u] = *(const f32x4*)(p.cache.k_scale + at[u] + 4 * g);
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d = FULL ? c * kVD : min(c * kVD, dim - kVD);  // dims past the head's: not stored
      const char* src = vbase + at[u] * row_bytes;
      const uint32_t off = 4 * g * row_bytes + d * kBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < kVWords; w += 4) {
          if constexpr (kVWords >= 4) {
            const u32x4 x = load16(src + (off + i * row_bytes + 4 * w));
#pragma unroll
            for (int e = 0; e < 4; ++e) vreg[u][i][w + e] = x[e];
          } else if constexpr (kVWords == 2) {
            const u32x2 x = load8(src + (off + i * row_bytes));
            vreg[u][i][0] = x.x;
            vreg[u][i][1] = x.y;
          } else {
            vreg[u][i][0] = *(const uint32_t*)(src + (off + i * row_bytes));
          }
        }
      if constexpr (!kSame) vscale[u] = *(const f32x4*)(p.cache.v_scale + at[u] + 4 * g);
    }
  };

  if (wave < tiles) {
    look_up(wave);
    take_rows(wave);
    look_up(wave + kAttnWaves);
    load_k();
    load_v();
  }
  Rows<T, FMT, DB, R, false> rw;
  rw.init(p, it, row0, TREE ? it.len : range.stop, dim, [&](int s) {
    return kSame ? 32 * s + 8 * g : 64 * (s / 2) + 16 * g + 8 * (s & 1);
  });

  rw.settle();
  int n = wave;
  auto tile = [&](auto edge) {
    const int t0 = range.begin + n * kAttnTile;
    const bool exists[2] = {ok[0], ok[1]};
    // the first loop's tiles all have a next one: no branches, hence no copies of
    // what the next loads replace
    const bool more = !decltype(edge)::value || n + kAttnWaves < tiles;
    if (more) {
      take_rows(n + kAttnWaves);
      look_up(n + 2 * kAttnWaves);
    }
    rw.template tile<decltype(edge)::value, TREE>(
        p, t0, exists,
        [&](int u, int i) -> u32x4 {
          if constexpr (kSame) {
            return kreg[u][i];
          } else {
            const uint32_t x = kreg[u][i / 2][2 * (i & 1)], y = kreg[u][i / 2][2 * (i & 1) + 1];
            using K = typename TY::K;
            return u32x4{widen_pair<K, FMT, false>(x), widen_pair<K, FMT, true>(x),
                         widen_pair<K, FMT, false>(y), widen_pair<K, FMT, true>(y)};
          }
        },
        [&](int u) { return kscale[u]; },
        [&]() {
          if (more) load_k();
        },
        [&](uint32_t in) -> bool {
          bool odd = false;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int x = 0; x < kVWords; ++x) {
                const uint32_t y = (in >> (4 * u + i)) & 1 ? vreg[u][i][x] : 0u;
                vreg[u][i][x] = y;
                if constexpr (kSame) odd |= odd_halves<T>(y) != 0;
                if constexpr (FMT == W4A16_KV_E4M3) odd |= nan_codes(y);
              }
          if constexpr (FMT == W4A16_KV_INT8 || !TREE) return false;
          return __any(odd);
        },
        [&](int u) { return vscale[u]; },
        // tokens (i, i + 1) of dim j side by side: one permute per word
        [&](int j) -> u32x4 {
          u32x4 a;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (kSame) {
                a[2 * u + h] = __builtin_amdgcn_perm(vreg[u][2 * h + 1][j / 2], vreg[u][2 * h][j / 2],
                                                     j & 1 ? 0x07060302u : 0x05040100u);
              } else {
                const uint32_t y = __builtin_amdgcn_perm(
                    vreg[u][2 * h + 1][j / 4], vreg[u][2 * h][j / 4],
                    j & 2 ? 0x07030602u : 0x05010400u);
                using P = typename TY::P;
                a[2 * u + h] = j & 1 ? widen_pair<P, FMT, true>(y) : widen_pair<P, FMT, false>(y);
              }
            }
          return a;
        },
        [&]() {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int x = 0; x < kVWords; ++x) asm volatile("" : "+v"(vreg[u][i][x]));
        });
    if (more) load_v();
    n += kAttnWaves;
  };
  // First the tiles that every row sees whole, then (in code of its own, which
  // costs the first loop no registers) those at the end, or after a lost page.
  const int whole = min(range.see_all, it.len);
  while (n + kAttnWaves < tiles && range.begin + (n + 1) * kAttnTile <= whole && ok[0] && ok[1])
    tile(std::false_type{});
  while (kSame ? n < tiles : __builtin_expect(n < tiles, 0)) tile(std::true_type{});

  // ---- join the four waves, a row block at a time
  constexpr int kH = DB / 64, kPart = (int)attn_part_floats(kRows, DB);
  const Parts parts(p, kPart);
  const int row = tid >> 4, l16 = tid & 15;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float sum = rw.denominator(r);
    if (r > 0) __syncthreads();
    if (g == 0) l_stat[wave][c] = f32x2{rw.top[r], sum};
    rw.put_row(l_sum[wave][c], r);
    __syncthreads();
    float m = kNegInf;
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) m = fmaxf(m, l_stat[v][row].x);
    float z = 0.0f;
    f32x4 o[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) o[h] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) {
      const f32x2 st = l_stat[v][row];
      const float f = st.x == m ? 1.0f : __builtin_amdgcn_exp2f(st.x - m);
      z = fmaf(f, st.y, z);
#pragma unroll
      for (int h = 0; h < kH; ++h) o[h] += f * *(const f32x4*)&l_sum[v][row][64 * h + 4 * l16];
    }
    const int at = 16 * r + row;
    if (at < rows) {
      if (it.splits == 1) {
#pragma unroll
        for (int h = 0; h < kH; ++h)
          finish4<T>(p, it, row0 + at, 64 * h + 4 * l16, dim, m, z, TY::kLift, o[h]);
      } else {
        const uint32_t part = (uint32_t)blockIdx.x * kPart;
#pragma unroll
        for (int h = 0; h < kH; ++h) parts.put4(part + at * DB + 64 * h + 4 * l16, o[h]);
        if (l16 == 0) parts.put2(part + kRows * DB + 2 * at, m, z);
      }
    }
  }
  if (it.splits > 1 && arrive(p, it, &l_last))
    join_parts<T, DB, kRows>(p, it, rows, dim, TY::kLift, &l_sum[0][0][0]);
}

// ---------------------------------------------------------------- many rows
// A stage: 64 tokens' K and V rows, 16 bits a value, DB values a row, in
// 16-byte pieces permuted inside each row so that what is read at once spreads
// over all 64 banks (256 bytes): an operand read takes one piece of 16 rows, a
// transposing read two neighbouring pieces of 8 rows.
template <int PIECES>
__device__ __forceinline__ int k_place(int piece, int row) {
  return piece ^ (PIECES >= 16 ? row & 15 : (row >> 1) & 7);
}
template <int PIECES>
__device__ __forceinline__ int v_place(int piece, int row) {
  return piece ^ (PIECES >= 16 ? (row & 7) << 1 : ((row >> 1) & 3) << 1);
}
template <int DB>
struct Stage {
  u32x4 k[kAttnStage * DB / 8];
  u32x4 v[kAttnStage * DB / 8];
  float k_scale[kAttnStage], v_scale[kAttnStage];
};

typedef __attribute__((address_space(3))) char* Lds;

// 16 bytes per lane from base + the lane's offset straight into LDS, lane after
// lane from `to` (uniform). The compiler does not count it: drain() before the
// barrier after which the data are read. (m0 is the compiler's own: it cannot be
// declared as overwritten, and no other instruction of the library names it.)
__device__ __forceinline__ void copy16(const void* base, uint32_t offset, Lds to) {
  const uint32_t lds = (uint32_t)(uintptr_t)to;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"(base), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory");
}
__device__ __forceinline__ void drain() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Four rows' values of a column: lane (g, c) of the wave gives the address of
// row 4g + c / 4, columns 4 (c % 4).. of a 16-column tile, and gets column c of
// rows 4g..4g + 3 (checked on the GPU).
__device__ __forceinline__ u32x2 read_transposed(Lds at) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* At;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)at));
}

// Two stages, so that the next one's copies run under the products; 16-bit rows go
// straight into LDS, 8-bit ones through registers, where they are widened. V lies
// in rows, as K does, and is read transposed.
//
// At 32 rows a wave, 64 tokens take 64 products (1024 cycles of the matrix core) and
// about as long again in exponentials (32 x 16 cycles), multiply-adds, sums,
// conversions and LDS reads, which two waves a SIMD overlap in part. 2 x 1024 new
// tokens over 16384, 40 query heads, bf16: 700 to 820 us, 0.81 to 0.95 PFLOP/s (a
// large product reaches 1.57); the matrix core is busy 42 % of the time, vector
// instructions issue 51 %. Short items wait more than they issue: 16 trees of 24 over
// 4000 in int8 take 50 us with the matrix core busy 12 %, vector issue 39 %, and half
// of the waves' time in waits (a first stage that nothing hides, few stages an item,
// parts and their join). Tried: wave priorities around the products (no change), V operands
// fetched before the exponentials (none), LDS addresses kept in registers (a
// quarter slower: the registers they take are spilled inside the loop).
template <typename T, int FMT, int DB, int R, bool FULL>
__global__ __launch_bounds__(64 * kAttnWaves, DB == 256 ? 1 : 2) void attn_wide_kernel(AttnParams p) {
  using TY = Types<T, FMT>;
  constexpr bool kSame = TY::kSame;
  constexpr int kWaveRows = 16 * R, kRows = kAttnWaves * kWaveRows;
  constexpr int kVD = DB / 16;
  constexpr int kBytes = kSame ? 2 : 1;
  constexpr int kPieces = DB / 8;              // 8-dim pieces of a row
  constexpr int kPass = 64 / kPieces;          // rows that a wave brings at once
  constexpr int kPasses = 16 / kPass;          // wave w brings tokens 16 w..16 w + 15
  extern __shared__ __align__(16) char l_raw[];
  Stage<DB>* stage = (Stage<DB>*)l_raw;        // two of them
  // byte addresses of a stage's K and V in LDS
  auto k_at = [&](int n) { return (Lds)l_raw + (n & 1) * (int)sizeof(Stage<DB>); };
  auto v_at = [&](int n) { return k_at(n) + kAttnStage * DB * 2; };

  Item it;
  if (!find_item<kRows>(p, blockIdx.x, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int dim = FULL ? DB : p.cache.dim;
  const int row0 = it.block * kRows;
  const int rows = it.news * p.group - row0;
  const Range range = range_of(p, it, row0, kRows);
  const int stages = range.end > range.begin ? (range.end - range.begin + kAttnStage - 1) / kAttnStage : 0;
  const bool busy = wave * kWaveRows < rows;   // this wave has rows

  const char* kbase = (const char*)p.cache.k;
  const char* vbase = (const char*)p.cache.v;
  const int row_bytes = dim * kBytes;
  const int piece = lane % kPieces, sub = lane / kPieces;  // this lane's place in a pass

  u32x2 kreg[kPasses], vreg[kPasses];          // 8-bit caches: on their way through registers
  float sreg = 0.0f;                           // a token's scale: lanes 0..15 K's, 16..31 V's
  bool exists[4];                              // of the stage on its way, by 16 tokens
  const Pages table(p, it);
  int pages[4];                                // of the stage after that
  auto look_up = [&](int n) {
#pragma unroll
    for (int u = 0; u < 4; ++u) pages[u] = table.of(range.begin + n * kAttnStage + 16 * u);
  };
  auto load = [&](int n) {
    const int t0 = range.begin + n * kAttnStage;
    int page = 0;
    bool there = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      exists[u] = table.there(pages[u], t0 + 16 * u);
      page = wave == u ? pages[u] : page;
      there = wave == u ? exists[u] : there;
    }
    const int64_t at = table.row(page, t0 + 16 * wave, there);
    look_up(n + 1);                            // scalar loads, back by the next stage
    const char* ksrc = kbase + at * row_bytes;
    const char* vsrc = vbase + at * row_bytes;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kPass + sub;           // row of the 16
      const int kp = k_place<kPieces>(piece, r), vp = v_place<kPieces>(piece, r);
      const uint32_t koff = r * row_bytes + kp * 8 * kBytes, voff = r * row_bytes + vp * 8 * kBytes;
      const bool kin = FULL || kp * 8 < dim, vin = FULL || vp * 8 < dim;
      if constexpr (kSame) {
        // lanes past the head's dims bring nothing: those pieces stay zeros
        if (kin) copy16(ksrc, koff, k_at(n) + (16 * wave + i * kPass) * DB * 2);
        if (vin) copy16(vsrc, voff, v_at(n) + (16 * wave + i * kPass) * DB * 2);
      } else {
        kreg[i] = load8(ksrc + (kin ? koff : 0));
        vreg[i] = load8(vsrc + (vin ? voff : 0));
        if (!kin) kreg[i] = u32x2{0, 0};
        if (!vin) vreg[i] = u32x2{0, 0};
      }
    }
    if constexpr (!kSame)
      if (lane < 32) sreg = (lane < 16 ? p.cache.k_scale : p.cache.v_scale)[at + c];
  };
  auto store = [&](int n) {                    // 8-bit caches: widened into the stage
    if constexpr (!kSame) {
      Stage<DB>& st = stage[n & 1];
      using KT = typename TY::K;
      using PT = typename TY::P;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int x = (16 * wave + i * kPass) * kPieces + lane;
        st.k[x] = u32x4{widen_pair<KT, FMT, false>(kreg[i].x), widen_pair<KT, FMT, true>(kreg[i].x),
                        widen_pair<KT, FMT, false>(kreg[i].y), widen_pair<KT, FMT, true>(kreg[i].y)};
        st.v[x] = u32x4{widen_pair<PT, FMT, false>(vreg[i].x), widen_pair<PT, FMT, true>(vreg[i].x),
                        widen_pair<PT, FMT, false>(vreg[i].y), widen_pair<PT, FMT, true>(vreg[i].y)};
      }
      if (lane < 32) (lane < 16 ? st.k_scale : st.v_scale)[16 * wave + c] = sreg;
    }
  };

  if constexpr (kSame && !FULL) {              // pieces that no load will reach
    for (int i = tid; i < 2 * kAttnStage * kPieces; i += 64 * kAttnWaves) {
      stage[i & 1].k[i >> 1] = u32x4{0, 0, 0, 0};
      stage[i & 1].v[i >> 1] = u32x4{0, 0, 0, 0};
    }
    __syncthreads();
  }
  if (stages > 0) {
    look_up(0);
    load(0);
  }
  Rows<T, FMT, DB, R, true> rw;
  rw.init(p, it, row0 + wave * kWaveRows, it.len, dim, [&](int s) { return 32 * s + 8 * g; });
  rw.settle();
  bool held[4] = {false, false, false, false};  // pages of the stage in LDS
  if (stages > 0) {
    store(0);
#pragma unroll
    for (int u = 0; u < 4; ++u) held[u] = exists[u];
  }
  drain();
  __syncthreads();
  int n = 0;
  auto pass = [&](auto edge) {
    const bool more = !decltype(edge)::value || n + 1 < stages;
    if (more) load(n + 1);                     // the other stage was last read before the barrier
    Stage<DB>& st = stage[n & 1];
    if (busy) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t0 = range.begin + n * kAttnStage + 32 * half;
        if (decltype(edge)::value && t0 >= range.end) break;
        u32x4 clear = {~0u, ~0u, ~0u, ~0u};    // V of tokens that do not exist
        auto v_raw = [&](int j) -> u32x4 {
          const Lds at = v_at(n) + (32 * half + 4 * g + (c >> 2)) * DB * 2 +
                         v_place<kPieces>(2 * j + ((c >> 1) & 1), 4 * g + (c >> 2)) * 16 + (c & 1) * 8;
          const u32x2 x = read_transposed(at), y = read_transposed(at + 16 * DB * 2);
          return u32x4{x.x, x.y, y.x, y.y};
        };
        rw.template tile<decltype(edge)::value, true>(
            p, t0, held + 2 * half,
            [&](int u, int i) -> u32x4 {
              return st.k[(32 * half + 16 * u + c) * kPieces + k_place<kPieces>(4 * i + g, c)];
            },
            [&](int u) { return *(const f32x4*)&st.k_scale[32 * half + 16 * u + 4 * g]; },
            []() {},
            [&](uint32_t in) -> bool {
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                clear[e] = ((in >> (2 * e)) & 1 ? 0xFFFFu : 0u) | ((in >> (2 * e + 1)) & 1 ? 0xFFFF0000u : 0u);
              if constexpr (FMT != W4A16_KV_INT8) {
#pragma unroll 1
                for (int j = 0; j < kVD; ++j) {
                  const u32x4 a = v_raw(j) & clear;
#pragma unroll
                  for (int e = 0; e < 4; ++e) odd |= odd_halves<typename TY::P>(a[e]) != 0;
                }
              }
              return FMT != W4A16_KV_INT8 && __any(odd);
            },
            [&](int u) { return *(const f32x4*)&st.v_scale[32 * half + 16 * u + 4 * g]; },
            [&](int j) -> u32x4 { return decltype(edge)::value ? v_raw(j) & clear : v_raw(j); },
            []() { asm volatile("" ::: "memory"); });
      }
    }
    if (more) {
      store(n + 1);
#pragma unroll
      for (int u = 0; u < 4; ++u) held[u] = exists[u];
    }
    drain();
    __syncthreads();
    ++n;
  };
  // as in the narrow kernel: whole stages first, the rest in code of its own
  const int whole = min(range.see_all, it.len);
  while (n + 1 < stages && range.begin + (n + 1) * kAttnStage <= whole && held[0] && held[1] && held[2] && held[3])
    pass(std::false_type{});
  while (__builtin_expect(n < stages, 0)) pass(std::true_type{});

  // ---- a wave's rows are its own: through its part of the LDS (for whole rows
  // at a time) to the output, or to the part
  constexpr int kH = DB / 64, kPad = DB + 4, kPart = (int)attn_part_floats(kRows, DB);
  static_assert(kAttnWaves * 16 * kPad * 4 <= 2 * (int)sizeof(Stage<DB>), "rows fit the stages' LDS");
  const Parts parts(p, kPart);
  float* mine = (float*)l_raw + wave * 16 * kPad;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float z = rw.denominator(r);
    __builtin_amdgcn_wave_barrier();
    rw.put_row(mine + c * kPad, r);
    if (g == 0) *(f32x2*)(mine + c * kPad + DB) = f32x2{rw.top[r], z};
    // LDS accesses of one wave take effect in order; this keeps the compiler to it
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 4 * k + g, at = wave * kWaveRows + 16 * r + row;
      if (at >= rows) continue;
      const f32x2 st = *(const f32x2*)(mine + row * kPad + DB);
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const f32x4 o = *(const f32x4*)(mine + row * kPad + 64 * h + 4 * c);
        if (it.splits == 1)
          finish4<T>(p, it, row0 + at, 64 * h + 4 * c, dim, st.x, st.y, TY::kLift, o);
        else
          parts.put4((uint32_t)blockIdx.x * kPart + at * DB + 64 * h + 4 * c, o);
      }
      if (it.splits > 1 && c == 0)
        parts.put2((uint32_t)blockIdx.x * kPart + kRows * DB + 2 * at, st.x, st.y);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (it.splits > 1 && arrive(p, it, (int*)stage[0].k_scale))
    join_parts<T, DB, kRows>(p, it, rows, dim, TY::kLift, (float*)l_raw);
}

template <typename T, int FMT, int DB, int R, bool WIDE>
hipError_t launch_attn(const AttnParams& p, hipStream_t stream) {
  const dim3 grid((uint32_t)p.grid), block(64 * kAttnWaves);
  constexpr int kLds = WIDE ? 2 * (int)sizeof(Stage<DB>) : 0;
  const bool full = p.cache.dim == DB;
  void (*kernel)(AttnParams);
  if constexpr (WIDE)
    kernel = full ? attn_wide_kernel<T, FMT, DB, R, true> : attn_wide_kernel<T, FMT, DB, R, false>;
  else if (p.max_q == 1 && p.mask == nullptr)
    kernel = full ? attn_narrow_kernel<T, FMT, DB, R, true, false> : attn_narrow_kernel<T, FMT, DB, R, false, false>;
  else
    kernel = full ? attn_narrow_kernel<T, FMT, DB, R, true, true> : attn_narrow_kernel<T, FMT, DB, R, false, true>;
  if (kLds > 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, grid, block, kLds, stream, p);
  return hipGetLastError();
}

// One (dtype, format): the shape and the head dim pick the kernel.
template <typename T, int FMT>
hipError_t launch_attn_shape(const AttnParams& p, AttnKind kind, hipStream_t stream) {
  const int db = attn_dim_block(p.cache.dim);
  if (db == 256)
    return kind == AttnKind::kNarrow1 ? launch_attn<T, FMT, 256, 1, false>(p, stream)
                                      : launch_attn<T, FMT, 256, 1, true>(p, stream);
  if (db == 128)
    return kind == AttnKind::kNarrow1   ? launch_attn<T, FMT, 128, 1, false>(p, stream)
           : kind == AttnKind::kNarrow2 ? launch_attn<T, FMT, 128, 2, false>(p, stream)
           : kind == AttnKind::kWide1   ? launch_attn<T, FMT, 128, 1, true>(p, stream)
                                        : launch_attn<T, FMT, 128, 2, true>(p, stream);
  return kind == AttnKind::kNarrow1   ? launch_attn<T, FMT, 64, 1, false>(p, stream)
         : kind == AttnKind::kNarrow2 ? launch_attn<T, FMT, 64, 2, false>(p, stream)
         : kind == AttnKind::kWide1   ? launch_attn<T, FMT, 64, 1, true>(p, stream)
                                      : launch_attn<T, FMT, 64, 2, true>(p, stream);
}

}  // namespace serve
}  // namespace w4a16
