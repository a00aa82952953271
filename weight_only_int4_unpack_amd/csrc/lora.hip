// Low-rank adapters of many requests beside a shared product:
//   out[t] = base[t] + scale_i sum_r v_r b[i, :, r],  v_r = sum_k x[t, k] a[i, r, k].
//
// A plan orders the tokens by adapter and cuts each adapter's into tiles of 16 or 64
// tokens. Two kernels follow it. The first (down) forms v: a workgroup takes a tile and a
// range of k, its waves parts of that range, and their sums meet in LDS; the ranges' sums
// go to scratch in fp32. The second (up) takes a tile and a range of columns, adds the
// ranges of v in order, and multiplies it with b as two 16-bit parts, v = high + low:
// 16 bits of v in bf16 and 22 in fp16, each row scaled by a power of two in front of fp16
// so that it stays in range. The products are small beside the bytes: what bounds both is
// reading x, a and b once and base and out.
#include "batch_internal.h"
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

template <typename T>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (T::kCode == W4A16_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// ---- the plan: a counting sort of the tokens by adapter, by one workgroup. Each wave has
// a run of consecutive tokens and counts of its own, so that the order is the tokens' own
// within an adapter.
constexpr int kPlanWaves = kLoraPlanThreads / 64;
struct PlanLds {
  int32_t count[kPlanWaves][kLoraMaxAdapters + 1];
  int32_t tiles[kLoraMaxAdapters + 2];   // tiles of the groups before
  int32_t start[kLoraMaxAdapters + 2];   // tokens of the groups before
  int32_t wave[2][kPlanWaves];
};

__global__ __launch_bounds__(kLoraPlanThreads) void plan_kernel(LoraPlanParams p) {
  __shared__ PlanLds l;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = p.adapters + 1;     // the last: tokens without an adapter
  for (int i = tid; i < kPlanWaves * (kLoraMaxAdapters + 1); i += kLoraPlanThreads) (&l.count[0][0])[i] = 0;
  __syncthreads();
  const int run = (p.tokens + kLoraPlanThreads - 1) / kLoraPlanThreads * 64;
  const int lo = min(wave * run, p.tokens), hi = min(lo + run, p.tokens);
  // each token's place among its wave's of the same group, chunk by chunk of 64 tokens
  auto over = [&](auto place) {
    for (int base = lo; base < hi; base += 64) {
      const int t = base + lane;
      int key = -1;
      if (t < hi) {
        key = p.index[t];
        if (key < 0 || key >= p.adapters) key = p.adapters;
      }
      uint64_t rest = __ballot(t < hi);
      while (rest != 0) {
        const int k = __builtin_amdgcn_readlane(key, __builtin_ctzll(rest));
        const uint64_t same = __ballot(key == k);
        const int before = l.count[wave][k];
        if (key == k) place(t, before + __popcll(same & ((1ull << lane) - 1)));
        __builtin_amdgcn_wave_barrier();
        if (lane == 0) l.count[wave][k] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        rest &= ~same;
      }
    }
  };
  over([](int, int) {});
  __syncthreads();
  // groups: tokens and tiles before each, kEach groups a thread
  constexpr int kEach = (kLoraMaxAdapters + 1 + kLoraPlanThreads - 1) / kLoraPlanThreads;
  int tokens[kEach], tiles = 0, all = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int g = tid * kEach + e;
    tokens[e] = 0;
    if (g < groups)
      for (int w = 0; w < kPlanWaves; ++w) tokens[e] += l.count[w][g];
    all += tokens[e];
    tiles += (tokens[e] + p.tile_rows - 1) / p.tile_rows;
  }
  int upto = all, tiles_upto = tiles;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(upto, s), z = __shfl_up(tiles_upto, s);
    if (lane >= s) {
      upto += y;
      tiles_upto += z;
    }
  }
  if (lane == 63) {
    l.wave[0][wave] = upto;
    l.wave[1][wave] = tiles_upto;
  }
  __syncthreads();
  int before = upto - all, tiles_before = tiles_upto - tiles;
  for (int w = 0; w < wave; ++w) {
    before += l.wave[0][w];
    tiles_before += l.wave[1][w];
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int g = tid * kEach + e;
    if (g <= groups) {
      l.start[g] = before;
      l.tiles[g] = tiles_before;
    }
    if (g < groups) {
      int at = before;
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = l.count[w][g];
        l.count[w][g] = at;
        at += c;
      }
    }
    before += tokens[e];
    tiles_before += (tokens[e] + p.tile_rows - 1) / p.tile_rows;
  }
  __syncthreads();
  const int used = l.tiles[groups];
  for (int i = tid; i < p.max_tiles; i += kLoraPlanThreads) {
    LoraTile tile{-1, 0, 0, 0};
    if (i < used) {
      int g = 0, end = groups;           // the last group with tiles before <= i
      while (end - g > 1) {
        const int mid = (g + end) / 2;
        if (l.tiles[mid] <= i) g = mid; else end = mid;
      }
      tile.adapter = g < p.adapters ? g : -1;
      tile.start = l.start[g] + (i - l.tiles[g]) * p.tile_rows;
      tile.rows = min(p.tile_rows, l.start[g + 1] - tile.start);
    }
    p.tiles[i] = tile;
  }
  over([&](int t, int at) { p.order[at] = t; });
}

// A tile as the kernels may use it, whatever the plan holds.
__device__ __forceinline__ LoraTile tile_of(const LoraParams& p, int i, int most) {
  LoraTile t = p.tiles[i];
  t.start = min(max(t.start, 0), p.tokens);
  t.rows = min(min(max(t.rows, 0), most), p.tokens - t.start);
  if (t.adapter >= p.adapters) t.adapter = -1;
  return t;
}
__device__ __forceinline__ int token_of(const LoraParams& p, int at) {
  return min(max(p.order[at], 0), p.tokens - 1);
}
__device__ __forceinline__ int rank_of(const LoraParams& p, int adapter) {
  return p.ranks ? min(max(p.ranks[adapter], 0), p.rank) : p.rank;
}

// ---- down: MT tiles of 16 tokens, RB ranks (padded). A lane holds 8 PIECES consecutive k
// of its token (or rank) and step, four lanes 32 PIECES: any order of k will do, as long as x
// and a have the same.
template <typename T, int MT, int RB>
__global__ __launch_bounds__(kLoraThreads) void down_kernel(LoraParams p) {
  constexpr int RT = RB / 16;
  constexpr int PIECES = MT * RT <= 2 ? 4 : 2;
  constexpr int kStep = 32 * PIECES;
  constexpr int kMeet = MT * RT < 8 ? MT * RT : 8;          // results that meet at a time
  __shared__ f32x4 meet[4][kMeet][64];
  const LoraTile tile = tile_of(p, blockIdx.x, 16 * MT);
  if (tile.rows == 0 || tile.adapter < 0) return;
  const int split = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, group = lane >> 4;
  const int rank = rank_of(p, tile.adapter);
  const uint16_t* x[MT];
  const uint16_t* a[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    x[m] = p.x + token_of(p, tile.start + min(16 * m + col, tile.rows - 1)) * p.x_stride;
#pragma unroll
  for (int r = 0; r < RT; ++r)
    a[r] = p.a + ((int64_t)tile.adapter * p.rank + min(16 * r + col, p.rank - 1)) * p.k;
  f32x4 sum[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) sum[m][r] = f32x4{0, 0, 0, 0};

  // this wave's range: a quarter of the split's
  const int k_lo = split * p.steps * 128, k_hi = min(p.k, k_lo + p.steps * 128);
  const int each = ((k_hi - k_lo + 4 * kStep - 1) / (4 * kStep)) * kStep;
  const int from = k_lo + wave * each, to = min(k_hi, from + each);
  for (int k0 = from; k0 < to; k0 += kStep) {
    u32x4 xs[MT][PIECES], as[RT][PIECES];
    const int k = k0 + group * 8 * PIECES;
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const bool in = k + 8 * j < to;
      const int at = in ? k + 8 * j : 0;
#pragma unroll
      for (int m = 0; m < MT; ++m) xs[m][j] = load16(x[m] + at);
#pragma unroll
      for (int r = 0; r < RT; ++r) as[r][j] = load16(a[r] + at);
      // past the end and the rank: zeros on both sides, as 0 x NaN is NaN
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (!in) xs[m][j] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (!in) as[r][j] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) sum[m][r] = mfma<T>(as[r][j], xs[m][j], sum[m][r]);
  }
  // The waves' sums: a lane holds ranks 16 r + 4 group .. + 3 of token 16 m + col.
  float* out = p.parts + ((int64_t)split * p.tokens + tile.start) * RB;
#pragma unroll
  for (int first = 0; first < MT * RT; first += kMeet) {
    if (first > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < kMeet; ++i) meet[wave][i][lane] = sum[(first + i) / RT][(first + i) % RT];
    __syncthreads();
    for (int i = wave; i < kMeet; i += 4) {
      f32x4 v = meet[0][i][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += meet[w][i][lane];
      const int m = (first + i) / RT, r = (first + i) % RT;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * r + 4 * group + e >= rank) v[e] = 0.0f;
      if (16 * m + col < tile.rows) *(f32x4*)(out + (16 * m + col) * RB + 16 * r + 4 * group) = v;
    }
  }
}

// v as two 16-bit parts; what is not finite has no second one.
template <typename T>
__device__ __forceinline__ void halves(const f32x8& v, u32x4* high, u32x4* low) {
  const u32x4 h = narrow8<T>(v);
  const f32x8 wide = widen8<T>(h);
  f32x8 rest;
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = __builtin_isfinite(wide[e]) ? v[e] - wide[e] : 0.0f;
  *high = h;
  *low = narrow8<T>(rest);
}

// ---- up: a wave takes 64 columns of MT tiles of 16 tokens at a time. Rank blocks of 16
// are one matrix instruction of depth 32, v's high parts in the first half and its low ones
// in the second; larger ones two for each 32 ranks. b is the left operand, its rows in the
// order that gives a lane 8 consecutive columns of its token.
template <typename T, int MT, int RB>
__global__ __launch_bounds__(kLoraThreads) void up_kernel(LoraParams p) {
  constexpr int KS = RB <= 16 ? 1 : RB / 32;
  constexpr bool kPacked = RB <= 16;
  const LoraTile tile = tile_of(p, blockIdx.x, 16 * MT);
  if (tile.rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, group = lane >> 4;
  int64_t token[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) token[m] = token_of(p, tile.start + min(16 * m + col, tile.rows - 1));
  const int n_lo = blockIdx.y * p.columns, n_hi = min(p.n, n_lo + p.columns);
  if (tile.adapter < 0) {
    if (p.base == p.out) return;
    for (int n = n_lo + wave * 64 + group * 8; n < n_hi; n += 256) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (16 * m + col < tile.rows && n + 32 * j < n_hi) {
            u32x4 y{0, 0, 0, 0};
            if (p.base) y = load16(p.base + token[m] * p.base_stride + n + 32 * j);
            *(u32x4*)(p.out + token[m] * p.out_stride + n + 32 * j) = y;
          }
    }
    return;
  }
  const int rank = rank_of(p, tile.adapter);
  // v of this lane's tokens: the splits in order, then its parts
  u32x4 high[MT][KS], low[MT][KS];
  float factor[MT];
  const float scale = p.scales ? p.scales[tile.adapter] : 1.0f;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    f32x8 v[KS];
    const bool in = 16 * m + col < tile.rows;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      v[s] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (in) {
        const int r0 = kPacked ? (group & 1) * 8 : 32 * s + group * 8;
        const float* at = p.parts + ((int64_t)tile.start + 16 * m + col) * RB + r0;
        for (int i = 0; i < p.splits; ++i) v[s] += *(const f32x8*)(at + (int64_t)i * p.tokens * RB);
      }
    }
    factor[m] = scale;
    if constexpr (T::kCode == W4A16_F16) {
      // the row's largest magnitude to 2^14..2^15, if it is finite and not 0
      uint32_t most = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[s][e]) & 0x7FFFFFFFu);
      most = max(most, (uint32_t)__shfl_xor((int)most, 16));
      most = max(most, (uint32_t)__shfl_xor((int)most, 32));
      const int exponent = (int)(most >> 23);
      if (exponent > 0 && exponent < 255) {
        const int lift = 127 + 14 - exponent;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[s][e] = __builtin_ldexpf(v[s][e], lift);
        factor[m] = __builtin_ldexpf(scale, -lift);
      } else if (exponent == 255) {
        // beside what is not finite the others only must not become infinite
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (__builtin_isfinite(v[s][e])) v[s][e] = fminf(fmaxf(v[s][e], -65504.0f), 65504.0f);
      }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      halves<T>(v[s], &high[m][s], &low[m][s]);
      if (kPacked && group >= 2) high[m][s] = low[m][s];
    }
  }
  const uint16_t* b = p.b + (int64_t)tile.adapter * p.n * p.rank;
  const int row = (col >> 2) * 8 + (col & 3);
  for (int n0 = n_lo + wave * 64; n0 < n_hi; n0 += 256) {
    f32x4 sum[4][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) sum[j][m] = f32x4{0, 0, 0, 0};
    u32x4 held[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        held[m][h] = u32x4{0, 0, 0, 0};
        const int n = n0 + 32 * h + group * 8;
        if (p.base && n < n_hi) held[m][h] = load16(p.base + token[m] * p.base_stride + n);
      }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 bs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + (j >> 1) * 32 + (j & 1) * 4 + row;
        const int r0 = kPacked ? (group & 1) * 8 : 32 * s + group * 8;
        bs[j] = u32x4{0, 0, 0, 0};
        if (n < n_hi && r0 < rank) {
          bs[j] = load16(b + (int64_t)n * p.rank + r0);
          // past the adapter's own rank: zeros, as 0 x NaN is NaN
          if (r0 + 8 > rank) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (r0 + e >= rank) bs[j][e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          sum[j][m] = mfma<T>(bs[j], high[m][s], sum[j][m]);
          if constexpr (!kPacked) sum[j][m] = mfma<T>(bs[j], low[m][s], sum[j][m]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + 32 * h + group * 8;
        if (16 * m + col < tile.rows && n < n_hi) {
          f32x8 y = widen8<T>(held[m][h]);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = fmaf(sum[2 * h + e / 4][m][e % 4], factor[m], y[e]);
          *(u32x4*)(p.out + token[m] * p.out_stride + n) = narrow8<T>(y);
        }
      }
  }
}

template <typename T, int MT, int RB>
hipError_t launch(const LoraParams& p, hipStream_t stream) {
  down_kernel<T, MT, RB><<<dim3(p.tiles_most, p.splits), kLoraThreads, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  up_kernel<T, MT, RB><<<dim3(p.tiles_most, (p.n + p.columns - 1) / p.columns), kLoraThreads, 0, stream>>>(p);
  return hipGetLastError();
}
template <typename T, int MT>
hipError_t launch_rank(const LoraParams& p, hipStream_t stream) {
  switch (lora_rank_block(p.rank)) {
    case 16: return launch<T, MT, 16>(p, stream);
    case 32: return launch<T, MT, 32>(p, stream);
    case 64: return launch<T, MT, 64>(p, stream);
    default: return launch<T, MT, 128>(p, stream);
  }
}

}  // namespace

hipError_t launch_lora_plan(const LoraPlanParams& p, hipStream_t stream) {
  plan_kernel<<<1, kLoraPlanThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_lora(const LoraParams& p, int tile_rows, int dtype, hipStream_t stream) {
  if (dtype == W4A16_F16) return tile_rows == 64 ? launch_rank<F16, 4>(p, stream) : launch_rank<F16, 1>(p, stream);
  return tile_rows == 64 ? launch_rank<BF16, 4>(p, stream) : launch_rank<BF16, 1>(p, stream);
}

}  // namespace w4a16
