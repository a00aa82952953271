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
// (lane (g, c): token c, 16 bytes at dim chunk g). V is read in rows too (lane
// (g, c): its 8 tokens, dims c * DB/16 .. +DB/16, so a row of the page is one
// contiguous run over 16 lanes); one byte permute joins two tokens' values of
// a dim into an operand word, and tile j of O^T holds dims c * DB/16 + j.
//
// 8-bit codes are widened (exactly) in registers; a token's scales multiply
// its scores and its weights, which are one value per lane and token.
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

// Codes in the low (HI = false) or high half of a word as a 16-bit pair.
template <typename T, int FMT, bool HI>
__device__ __forceinline__ uint32_t widen_pair(uint32_t w) {
  if constexpr (FMT == W4A16_KV_E4M3) {
    if constexpr (T::kCode == W4A16_F16)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  } else {
    return pair<T>((float)(int8_t)(w >> (HI ? 16 : 0)), (float)(int8_t)(w >> (HI ? 24 : 8)));
  }
}

// What a workgroup works on.
struct Item {
  int seq, head, block, split;   // block: row block
  int splits;                    // of this sequence
  int blocks;                    // row blocks of this sequence
  int chunk;                     // tokens of a split
  int len, news, start;          // cached tokens, new tokens, first row in q
  int group;                     // counter: (sequence, block, head)
  int first;                     // index of this group's split 0 among the items
};

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
  auto load = [&](int b, int* len, int* news, int* start, int* blocks) {
    *len = *news = *start = *blocks = 0;
    if (b < p.sequences) {
      *len = min(max(p.kv_lens[b], 0), most);
      const int s0 = min(max(p.q_starts[b], 0), p.tokens);
      const int s1 = min(max(p.q_starts[b + 1], s0), p.tokens);
      *start = s0;
      *news = min(s1 - s0, p.max_q);
      *blocks = (*news * p.group + ROWS - 1) / ROWS;
    }
  };
  int len, news, start, blocks;
  uint32_t steps = 0;
  const bool one_round = p.sequences <= 64;
  for (int b0 = 0; b0 < p.sequences; b0 += 64) {
    load(b0 + lane, &len, &news, &start, &blocks);
    steps += (uint32_t)blocks * (uint32_t)((len + kAttnStep - 1) / kAttnStep);
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) steps += (uint32_t)__shfl_xor((int)steps, s);
  uint32_t per = 0x7FFFFFFF / kAttnStep;   // steps of a split
  if (p.target > 0)
    per = max((steps * (uint32_t)p.cache.heads + p.target - 1) / (uint32_t)p.target, 1u);
  int items_before = 0, groups_before = 0;
  for (int b0 = 0; b0 < p.sequences; b0 += 64) {
    if (!one_round) load(b0 + lane, &len, &news, &start, &blocks);
    const uint32_t mine = (uint32_t)(len + kAttnStep - 1) / kAttnStep;
    uint32_t own = per;
    if (p.target > 0) own = max(own, (mine + kAttnMaxSplits - 1) / kAttnMaxSplits);
    const int splits = max((int)((mine + own - 1) / own), 1);
    const int groups = blocks * p.cache.heads, items = groups * splits;
    int upto = items, gupto = groups;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int a = __shfl_up(upto, s), g = __shfl_up(gupto, s);
      upto += lane >= s ? a : 0;
      gupto += lane >= s ? g : 0;
    }
    const uint64_t past = __ballot(items_before + upto > index);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      it->seq = b0 + l;
      it->splits = __shfl(splits, l);
      it->blocks = __shfl(blocks, l);
      it->chunk = (int)min(__shfl((int)own, l), 0x7FFFFF00 / kAttnStep) * kAttnStep;
      it->len = __shfl(len, l);
      it->news = __shfl(news, l);
      it->start = __shfl(start, l);
      const int local = index - (items_before + __shfl(upto - items, l));
      // heads innermost: workgroups go round the 8 XCDs, so with 8 heads the
      // row blocks that share a head's keys and values share an L2
      it->head = local % p.cache.heads;
      const int rest = local / p.cache.heads;
      it->block = rest % it->blocks;
      it->split = rest / it->blocks;
      it->group = groups_before + __shfl(gupto - groups, l) + it->block * p.cache.heads + it->head;
      it->first = index - it->split * it->blocks * p.cache.heads;
      return true;
    }
    items_before += __shfl(upto, 63);
    groups_before += __shfl(gupto, 63);
  }
  return false;
}

// Writes dims d0..d0+VD-1 of a finished row: o / z, and the row's lse. The
// held maximum m is in log2, and z was summed `lift` above it.
template <typename T, int VD>
__device__ __forceinline__ void finish(const AttnParams& p, const Item& it, int row, int d0, int dim,
                                       float m, float z, float lift, const float* o) {
  const int query = row / p.group, head = it.head * p.group + row - query * p.group;
  const int64_t at = (int64_t)(it.start + query) * p.hq + head;
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
  uint16_t* dst = p.out + at * dim + d0;
#pragma unroll
  for (int j = 0; j < VD; j += 4)
    if (d0 + j < dim)
      *(u32x2*)(dst + j) = u32x2{pair<T>(o[j] * inv, o[j + 1] * inv),
                                 pair<T>(o[j + 2] * inv, o[j + 3] * inv)};
  if (d0 == 0)
    p.lse[at] = z == 0.0f ? kNegInf : 0.69314718055994530942f * (m - lift + __log2f(z));
}

template <typename T, int FMT, int DB, int R, bool FULL>
__global__ __launch_bounds__(64 * kAttnWaves) void tree_attn_kernel(AttnParams p) {
  constexpr bool kSame = FMT == W4A16_KV_SAME;
  constexpr int kRows = 16 * R;
  constexpr int kSteps = DB / 32;              // contraction steps of S^T
  constexpr int kVD = DB / 16;                 // dims of V per lane, and tiles of O^T
  constexpr int kBytes = kSame ? 2 : 1;
  constexpr int kVWords = kVD * kBytes / 4;    // words of a token's V per lane
  constexpr int kKLoads = DB * kBytes / 64;    // 16-byte loads of K per half tile
  constexpr int kPad = DB + 4;
  // Weights against 8-bit codes carry the token's scale and are rounded to
  // bf16, whose range holds any scale (fp16 would lose them below 6e-5).
  using PT = typename std::conditional<kSame, T, BF16>::type;
  // fp16 weights are kept 2^6 above 1 for the same reason: at most 2^14.
  constexpr float kLift = PT::kCode == W4A16_F16 ? 6.0f : 0.0f;
  constexpr float kSlack = 8.0f;               // how far scores may exceed the held maximum

  __shared__ float l_sum[kAttnWaves][16][kPad];
  __shared__ f32x2 l_stat[kAttnWaves][16];
  __shared__ int l_last;

  Item it;
  if (!find_item<kRows>(p, blockIdx.x, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int dim = FULL ? DB : p.cache.dim;
  const int rows = it.news * p.group - it.block * kRows;  // of this block, may exceed kRows
  const int row0 = it.block * kRows;
  const int prefix = it.len - it.news;                    // may be negative

  // New token of this lane's row in row block r (clamped to the last one).
  int query[R];
  u32x4 qreg[R][kSteps];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + c, it.news * p.group - 1);
    query[r] = row / p.group;
    const uint16_t* src = p.q + (int64_t)(it.start + query[r]) * p.q_token +
                          (int64_t)(it.head * p.group + row - query[r] * p.group) * p.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = kSame ? 32 * s + 8 * g : 64 * (s / 2) + 16 * g + 8 * (s & 1);
      u32x4 x = {0, 0, 0, 0};
      if (FULL || d < dim) x = load16(src + d);
      qreg[r][s] = x;
    }
  }

  // Tokens [begin, end) of this split; the block's rows see none past `end`.
  const int last_query = min(row0 + kRows, it.news * p.group) - 1;
  const int see_all = p.mask ? prefix : prefix + row0 / p.group + 1;  // every row sees below
  const int block_end = p.mask ? it.len : min(it.len, prefix + last_query / p.group + 1);
  const int begin = it.split * it.chunk;
  const int end = (int)min((int64_t)begin + it.chunk, (int64_t)max(block_end, 0));
  const int tiles = end > begin ? (end - begin + kAttnTile - 1) / kAttnTile : 0;

  const int32_t* table = p.block_table + it.seq * p.table_stride;
  const int shift = p.cache.page_shift;
  const char* kbase = (const char*)p.cache.k;
  const char* vbase = (const char*)p.cache.v;
  const int64_t row_bytes = (int64_t)dim * kBytes;

  u32x4 kreg[2][kKLoads];
  uint32_t vreg[2][4][kVWords];
  f32x4 kscale[2], vscale[2];
  bool page_ok[2] = {true, true};

  // First token row of half tile u of tile n (uniform), and whether its page exists.
  auto place = [&](int n, int u, bool* ok) -> int64_t {
    const int t = begin + n * kAttnTile + 16 * u;
    const int page = t < it.len ? table[t >> shift] : -1;
    *ok = page >= 0 && page < p.cache.pages;
    return (((int64_t)(*ok ? page : 0) * p.cache.heads + it.head) << shift) + (t & ((1 << shift) - 1));
  };
  auto load_k = [&](int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t at = place(n, u, &page_ok[u]);
      const char* src = kbase + (at + c) * row_bytes;
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) {
        const int d = i * (64 / kBytes) + g * (16 / kBytes);
        if constexpr (FULL) {
          kreg[u][i] = load16(src + d * kBytes);
        } else {                               // dims past the head's: zeros
          const bool in = d < dim;
          const u32x4 x = load16(src + (in ? d : 0) * kBytes);
          kreg[u][i] = in ? x : u32x4{0, 0, 0, 0};
        }
      }
      if constexpr (!kSame) kscale[u] = *(const f32x4*)(p.cache.k_scale + at + 4 * g);
    }
  };
  auto load_v = [&](int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bool ok;
      const int64_t at = place(n, u, &ok);
      const int d = FULL ? c * kVD : min(c * kVD, dim - kVD);  // dims past the head's: not stored
      const char* src = vbase + (at + 4 * g) * row_bytes + d * kBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < kVWords; w += 4) {
          if constexpr (kVWords >= 4) {
            const u32x4 x = load16(src + i * row_bytes + 4 * w);
#pragma unroll
            for (int e = 0; e < 4; ++e) vreg[u][i][w + e] = x[e];
          } else if constexpr (kVWords == 2) {
            const u32x2 x = load8(src + i * row_bytes);
            vreg[u][i][0] = x.x;
            vreg[u][i][1] = x.y;
          } else {
            vreg[u][i][0] = *(const uint32_t*)(src + i * row_bytes);
          }
        }
      if constexpr (!kSame) vscale[u] = *(const f32x4*)(p.cache.v_scale + at + 4 * g);
    }
  };

  f32x4 acc[R][kVD];
  float top[R], total[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    top[r] = kNegInf;
    total[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < kVD; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
  }

  if (wave < tiles) {
    load_k(wave);
    load_v(wave);
  }
  for (int n = wave; n < tiles; n += kAttnWaves) {
    const int t0 = begin + n * kAttnTile;
    // ---- S^T, in units of log2
    f32x4 s[R][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 a[kSteps];
      if constexpr (kSame) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) a[i] = kreg[u][i];
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = kreg[u][i / 2][2 * (i & 1) + e];
            a[i][2 * e] = widen_pair<T, FMT, false>(w);
            a[i][2 * e + 1] = widen_pair<T, FMT, true>(w);
          }
      }
      f32x4 factor = f32x4{p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2};
      if constexpr (!kSame) factor *= kscale[u];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) x = mfma16<T>(a[i], qreg[r][i], x);
        s[r][u] = x * factor;
      }
    }
    const bool edge = t0 + kAttnTile > see_all || t0 + kAttnTile > it.len || !page_ok[0] ||
                      !page_ok[1];
    const bool ok0 = page_ok[0], ok1 = page_ok[1];
    if (n + kAttnWaves < tiles) load_k(n + kAttnWaves);

    // ---- what a row does not see: score -inf (and, below, weight 0)
    uint32_t seen[R];                          // bit 4u + i: this lane's token (u, i)
    if (edge) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        seen[r] = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 16 * u + 4 * g + i;
            const int j = t - prefix;
            bool in = t < it.len && (u == 0 ? ok0 : ok1);
            if (in && j >= 0) {
              if (p.mask == nullptr)
                in = j <= query[r];
              else
                in = j < 64 * p.mask_words &&
                     ((p.mask[(int64_t)(it.start + query[r]) * p.mask_words + (j >> 6)] >> (j & 63)) & 1);
            }
            seen[r] |= in ? 1u << (4 * u + i) : 0u;
            s[r][u][i] = in ? s[r][u][i] : kNegInf;
          }
      }
    }

    // ---- the held maximum rises only when a score exceeds it by 2^8
    bool rise = false;
    float high[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float m = fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3]));
      m = fmaxf(m, fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
      high[r] = m;
      rise |= m > top[r] + kSlack;
    }
    if (__any(rise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float m = fmaxf(high[r], __shfl_xor(high[r], 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        m = fmaxf(m, top[r]);
        const float f = top[r] == m ? 1.0f : __builtin_amdgcn_exp2f(top[r] - m);
        top[r] = m;
        total[r] *= f;
#pragma unroll
        for (int j = 0; j < kVD; ++j) acc[r][j] *= f;
      }
    }

    // ---- weights
    u32x4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ref = (top[r] == kNegInf ? 0.0f : top[r]) - kLift;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = __builtin_amdgcn_exp2f(s[r][u][i] - ref);
          total[r] += x[i];
          if constexpr (!kSame) x[i] *= vscale[u][i];
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = (seen[r] >> (4 * u + i)) & 1 ? x[i] : 0.0f;
        }
        w[r][2 * u] = pair<PT>(x[0], x[1]);
        w[r][2 * u + 1] = pair<PT>(x[2], x[3]);
      }
    }

    // ---- O^T
    bool apart = false;                        // a value that must not meet weight 0
    if (edge) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 16 * u + 4 * g + i;
          const bool in = t < it.len && (u == 0 ? ok0 : ok1);
#pragma unroll
          for (int x = 0; x < kVWords; ++x) {
            vreg[u][i][x] = in ? vreg[u][i][x] : 0u;
            const uint32_t y = vreg[u][i][x];
            if constexpr (kSame) {
              constexpr uint32_t kExp = T::kCode == W4A16_F16 ? 0x7C00u : 0x7F80u;
              apart |= (y & kExp) == kExp || ((y >> 16) & kExp) == kExp;
            } else if constexpr (FMT == W4A16_KV_E4M3) {
              const uint32_t z = (y & 0x7F7F7F7Fu) + 0x01010101u;  // NaN codes: 0x80
              apart |= (z & 0x80808080u) != 0;
            }
          }
        }
      apart = __any(apart);
    }
    // Operand words of tile j: tokens (i, i + 1) of dim j, joined by one permute.
    auto operand = [&](int j) -> u32x4 {
      u32x4 a;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (kSame) {
            a[2 * u + h] = __builtin_amdgcn_perm(vreg[u][2 * h + 1][j / 2], vreg[u][2 * h][j / 2],
                                                 j & 1 ? 0x07060302u : 0x05040100u);
          } else {
            // bytes j, j+1 of both tokens: {a_j, b_j, a_j+1, b_j+1}
            const uint32_t y = __builtin_amdgcn_perm(vreg[u][2 * h + 1][j / 4], vreg[u][2 * h][j / 4],
                                                     j & 2 ? 0x07030602u : 0x05010400u);
            a[2 * u + h] = j & 1 ? widen_pair<PT, FMT, true>(y) : widen_pair<PT, FMT, false>(y);
          }
        }
      return a;
    };
    if (!apart) {
#pragma unroll
      for (int j = 0; j < kVD; ++j) {
        const u32x4 a = operand(j);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][j] = mfma16<PT>(a, w[r], acc[r][j]);
      }
    } else {
      // An infinity or NaN among values that some rows may not see: token by
      // token, and a row that does not see the token keeps its sums.
      for (int t = 0; t < kAttnTile; ++t) {
        const int tu = t >> 4, tg = (t >> 2) & 3, ti = t & 3;
        u32x4 only = {0, 0, 0, 0};
        const uint32_t bits = tg == g ? (ti & 1 ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) only[e] = e == 2 * tu + (ti >> 1) ? bits : 0u;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool in = (__shfl((int)seen[r], tg * 16 + c) >> (4 * tu + ti)) & 1;
#pragma unroll
          for (int j = 0; j < kVD; ++j) {
            const f32x4 y = mfma16<PT>(operand(j) & only, w[r] & only, acc[r][j]);
            acc[r][j] = in ? y : acc[r][j];
          }
        }
      }
    }
    if (n + kAttnWaves < tiles) load_v(n + kAttnWaves);
  }

  // ---- join the lane groups' sums and the four waves, a row block at a time
  const int row = tid >> 4, chunk = tid & 15;
  const int64_t part_floats = attn_part_floats(kRows, DB);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float sum = total[r];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (r > 0) __syncthreads();
    if (g == 0) l_stat[wave][c] = f32x2{top[r], sum};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kVD; j += 4)
        *(f32x4*)&l_sum[wave][c][(4 * g + i) * kVD + j] =
            f32x4{acc[r][j][i], acc[r][j + 1][i], acc[r][j + 2][i], acc[r][j + 3][i]};
    __syncthreads();
    float m = kNegInf;
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) m = fmaxf(m, l_stat[v][row].x);
    float z = 0.0f, o[kVD];
#pragma unroll
    for (int j = 0; j < kVD; ++j) o[j] = 0.0f;
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) {
      const f32x2 st = l_stat[v][row];
      const float f = st.x == m ? 1.0f : __builtin_amdgcn_exp2f(st.x - m);
      z = fmaf(f, st.y, z);
#pragma unroll
      for (int j = 0; j < kVD; ++j) o[j] = fmaf(f, l_sum[v][row][chunk * kVD + j], o[j]);
    }
    const int at = 16 * r + row;
    if (at >= rows) continue;
    if (it.splits == 1) {
      finish<T, kVD>(p, it, row0 + at, chunk * kVD, dim, m, z, kLift, o);
    } else {
      // device-scope stores; the wait and the counter below order them
      float* part = p.parts + blockIdx.x * part_floats;
      uint64_t* dst = (uint64_t*)(part + at * DB + chunk * kVD);
#pragma unroll
      for (int j = 0; j < kVD; j += 2)
        __hip_atomic_store(dst + j / 2, __builtin_bit_cast(uint64_t, f32x2{o[j], o[j + 1]}),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (chunk == 0)
        __hip_atomic_store((uint64_t*)(part + kRows * DB) + at,
                           __builtin_bit_cast(uint64_t, f32x2{m, z}), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (it.splits == 1) return;

  // ---- hand-off: the last of a group's splits to arrive joins them all, in
  // split order (results do not depend on the order of arrival)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's stores are complete
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (tid == 0) {
    const int arrived = __hip_atomic_fetch_add(p.counters + it.group, 1, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
    l_last = arrived == it.splits - 1;
  }
  __syncthreads();
  if (!l_last) return;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  if (tid == 0)
    __hip_atomic_store(p.counters + it.group, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int64_t stride = (int64_t)it.blocks * p.cache.heads * part_floats;
  const float* parts = p.parts + (int64_t)it.first * part_floats;
  auto stat = [&](int split, int at) -> f32x2 {
    const uint64_t x = __hip_atomic_load((const uint64_t*)(parts + split * stride + kRows * DB) + at,
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(f32x2, x);
  };
  for (int at = row; at < min(rows, kRows); at += 16) {
    float m = kNegInf;
    for (int sp = chunk; sp < it.splits; sp += 16) m = fmaxf(m, stat(sp, at).x);
#pragma unroll
    for (int s = 1; s < 16; s *= 2) m = fmaxf(m, __shfl_xor(m, s));
    float z = 0.0f, o[kVD];
#pragma unroll
    for (int j = 0; j < kVD; ++j) o[j] = 0.0f;
#pragma unroll 4
    for (int sp = 0; sp < it.splits; ++sp) {
      const f32x2 st = stat(sp, at);
      const float f = st.x == m ? 1.0f : __builtin_amdgcn_exp2f(st.x - m);
      z = fmaf(f, st.y, z);
      const uint64_t* src = (const uint64_t*)(parts + sp * stride + at * DB + chunk * kVD);
#pragma unroll
      for (int j = 0; j < kVD; j += 2) {
        const f32x2 x = __builtin_bit_cast(
            f32x2, __hip_atomic_load(src + j / 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        o[j] = fmaf(f, x.x, o[j]);
        o[j + 1] = fmaf(f, x.y, o[j + 1]);
      }
    }
    finish<T, kVD>(p, it, row0 + at, chunk * kVD, dim, m, z, kLift, o);
  }
}

template <typename T, int FMT, int DB, int R>
hipError_t launch_attn(const AttnParams& p, hipStream_t stream) {
  const dim3 grid((uint32_t)p.grid), block(64 * kAttnWaves);
  if (p.cache.dim == DB)
    hipLaunchKernelGGL((tree_attn_kernel<T, FMT, DB, R, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((tree_attn_kernel<T, FMT, DB, R, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

// One (dtype, format): row_blocks and the head dim pick the kernel.
template <typename T, int FMT>
hipError_t launch_attn_rows(const AttnParams& p, int row_blocks, hipStream_t stream) {
  const int db = attn_dim_block(p.cache.dim);
  if (db == 256)
    return row_blocks == 1 ? launch_attn<T, FMT, 256, 1>(p, stream)
                           : launch_attn<T, FMT, 256, 2>(p, stream);
  if (db == 128)
    return row_blocks == 1   ? launch_attn<T, FMT, 128, 1>(p, stream)
           : row_blocks == 2 ? launch_attn<T, FMT, 128, 2>(p, stream)
                             : launch_attn<T, FMT, 128, 4>(p, stream);
  return row_blocks == 1   ? launch_attn<T, FMT, 64, 1>(p, stream)
         : row_blocks == 2 ? launch_attn<T, FMT, 64, 2>(p, stream)
                           : launch_attn<T, FMT, 64, 4>(p, stream);
}

}  // namespace serve
}  // namespace w4a16
