// Low-rank adapters of many requests beside a shared product:
//   out[t] = base[t] + scale_i sum_r v_r b[i, :, r],  v_r = sum_k x[t, k] a[i, r, k].
//
// A plan orders the tokens by adapter and cuts each adapter's into tiles of 16 or 64
// tokens. Two kernels follow it. The first (down) forms v: a workgroup takes a tile and a
// range of k, its waves parts of that range, and their sums meet in LDS; the ranges' sums
// go to scratch in fp32, where the last workgroup of a tile adds them in their order. It
// leaves v as two 16-bit parts, v = high + low: 16 bits of v in bf16 and 22 in fp16, each
// row scaled by a power of two in front of fp16 so that it stays in range. The second (up)
// takes a tile and a range of columns and multiplies both parts with b. For a few tokens
// one kernel does both. The products are small beside the bytes: what bounds them is
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
// within an adapter. 64 tokens 5 us, 8192 16 us, once for all products of a step.
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
        if (key == k) place(t, before + __popcll(same & ((1ull << lane) - 1)), k);
        __builtin_amdgcn_wave_barrier();
        if (lane == 0) l.count[wave][k] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        rest &= ~same;
      }
    }
  };
  over([](int, int, int) {});
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
    int adapter = kLoraUnused;
    int first = 0, left = 0;             // of the group's tokens in this tile
    if (i < used) {
      int g = 0, end = groups;           // the last group with tiles before <= i
      while (end - g > 1) {
        const int mid = (g + end) / 2;
        if (l.tiles[mid] <= i) g = mid; else end = mid;
      }
      adapter = g < p.adapters ? g : kLoraNone;
      first = (i - l.tiles[g]) * p.tile_rows;
      left = l.start[g + 1] - l.start[g] - first;
    }
    p.tile[i] = adapter;
    for (int r = max(left, 0); r < p.tile_rows; ++r) p.token[(int64_t)i * p.tile_rows + r] = -1;
  }
  over([&](int t, int at, int key) {
    const int in = at - l.start[key];
    const int tile = l.tiles[key] + in / p.tile_rows;
    p.token[(int64_t)tile * p.tile_rows + in % p.tile_rows] = t;
  });
}

// A row's token, or -1, whatever the plan holds; and the tile's adapter.
__device__ __forceinline__ int token_of(const LoraParams& p, int64_t row) {
  const int t = p.token[row];
  return t < p.tokens ? t : -1;
}
__device__ __forceinline__ int adapter_of(const LoraParams& p, int tile) {
  const int i = p.tile[tile];
  return i < p.adapters ? i : kLoraUnused;
}
__device__ __forceinline__ int rank_of(const LoraParams& p, int adapter) {
  return p.ranks ? min(max(p.ranks[adapter], 0), p.rank) : p.rank;
}

// A wave's LDS accesses take effect in order; this holds the compiler to it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Values that other workgroups read: 8 bytes at a time, past the caches that are not shared.
__device__ __forceinline__ void store_shared(float* to, const f32x4& v) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  __hip_atomic_store((uint64_t*)to, w.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store((uint64_t*)to + 1, w.y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x8 load_shared(const float* from) {
  typedef uint64_t u64x4 __attribute__((ext_vector_type(4)));
  u64x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __hip_atomic_load((const uint64_t*)from + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f32x8, w);
}
// This wave's stores are where everybody sees them.
__device__ __forceinline__ void wait_stores() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);    // vmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---- down: the sums v of MT parts of 16 tokens, RB ranks (padded), over a range of k, by a
// workgroup. Each wave takes a part of the range, and the waves' sums meet in LDS.
// Memory is read as whole lines, kLanes lanes a row, and turned in LDS into what the matrix
// instructions take (read straight into their layout, where neighbouring lanes hold different
// rows, 8192 tokens of 5120 with rank 64 took 45 us instead of 32).
template <typename T, int MT, int RB, int THREADS = kLoraDownThreads>
struct Down {
  static constexpr int kWaves = THREADS / 64, kRows = 16 * MT, RT = RB / 16;
  static constexpr int kStep = lora_step(MT, RB), kPieces = kStep / 32;
  static constexpr int kMeet = MT * RT < 4 ? MT * RT : 4;          // results that meet at a time
  static constexpr int kTurnA = RB < 64 ? RB : 64;                 // ranks that are turned at a time
  static constexpr int kStride = kStep + 8;                        // of a row in LDS
  static constexpr int kWaveTurn = (kRows > kTurnA ? kRows : kTurnA) * kStride;
  static constexpr int kMeetBytes = kWaves * kMeet * 64 * 16, kTurnBytes = kWaves * kWaveTurn * 2;
  static constexpr int kLdsBytes = kMeetBytes > kTurnBytes ? kMeetBytes : kTurnBytes;
  static constexpr int kLanes = kStep / 8, kRowsAt = 64 / kLanes;  // lanes of a row, rows of a load
  static constexpr int kLoadsX = kRows / kRowsAt, kLoadsA = RB / kRowsAt;
  struct Stage {
    u32x4 x[kLoadsX], a[kLoadsA];
  };

  // put(row, r, v): ranks r .. r + 3 of a row's sums (0 from the adapter's own rank on).
  template <typename Put>
  static __device__ __forceinline__ void sums(const LoraParams& p, char* lds, int64_t rows, int adapter, int rank,
                                              int k_lo, int k_hi, Put put) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, group = lane >> 4, line = lane / kLanes, piece = lane % kLanes;
    uint16_t* turn = (uint16_t*)lds + wave * kWaveTurn;
    // rows without a token take part with another's x: each row's sums are its own
    const uint16_t* x[kLoadsX];
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i)
      x[i] = p.x + (int64_t)max(token_of(p, rows + i * kRowsAt + line), 0) * p.x_stride;
    const uint16_t* a = p.a + (int64_t)adapter * p.rank * p.k;
    f32x4 sum[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r) sum[m][r] = f32x4{0, 0, 0, 0};

    // the waves' steps lie side by side, so that a row is read in runs of all of them
    constexpr int kTurn = kWaves * kStep;
    const int from = k_lo + wave * kStep, to = k_hi;
    auto load = [&](int k0, Stage& s) {
      const int k = k0 + piece * 8 < to ? k0 + piece * 8 : 0;
#pragma unroll
      for (int i = 0; i < kLoadsX; ++i) s.x[i] = load16(x[i] + k);
#pragma unroll
      for (int i = 0; i < kLoadsA; ++i) s.a[i] = load16(a + (int64_t)min(i * kRowsAt + line, p.rank - 1) * p.k + k);
    };
    auto multiply = [&](int k0, const Stage& s) {
      const bool in = k0 + piece * 8 < to;   // past the end: zeros on both sides, as 0 x NaN is NaN
      u32x4 xs[MT][kPieces];
#pragma unroll
      for (int i = 0; i < kLoadsX; ++i)
        *(u32x4*)&turn[(i * kRowsAt + line) * kStride + piece * 8] = in ? s.x[i] : u32x4{0, 0, 0, 0};
      wave_sync();
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < kPieces; ++j) xs[m][j] = *(const u32x4*)&turn[(16 * m + col) * kStride + 32 * j + group * 8];
      wave_sync();
#pragma unroll
      for (int h = 0; h < RB; h += kTurnA) {
#pragma unroll
        for (int i = 0; i < kTurnA / kRowsAt; ++i)
          *(u32x4*)&turn[(i * kRowsAt + line) * kStride + piece * 8] = in ? s.a[h / kRowsAt + i] : u32x4{0, 0, 0, 0};
        wave_sync();
        u32x4 as[kTurnA / 16][kPieces];
#pragma unroll
        for (int r = 0; r < kTurnA / 16; ++r)
#pragma unroll
          for (int j = 0; j < kPieces; ++j)
            as[r][j] = *(const u32x4*)&turn[(16 * r + col) * kStride + 32 * j + group * 8];
        wave_sync();
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < kTurnA / 16; ++r)
              sum[m][h / 16 + r] = mfma<T>(as[r][j], xs[m][j], sum[m][h / 16 + r]);
      }
    };
    if constexpr (THREADS > 512) {
#pragma unroll 1
      for (int k0 = from; k0 < to; k0 += kTurn) {
        Stage s;
        load(k0, s);
        multiply(k0, s);
      }
    } else if (from < to) {
      // the next step's loads are on their way while one is multiplied
      Stage s0, s1;
      int k0 = from;
      load(k0, s0);
      for (; k0 + 2 * kTurn < to; k0 += 2 * kTurn) {
        load(k0 + kTurn, s1);
        multiply(k0, s0);
        load(k0 + 2 * kTurn, s0);
        multiply(k0 + kTurn, s1);
      }
      if (k0 + kTurn < to) load(k0 + kTurn, s1);
      multiply(k0, s0);
      if (k0 + kTurn < to) multiply(k0 + kTurn, s1);
    }
    // the scratch holds the waves' sums from here on: a lane has ranks 16 r + 4 group .. + 3
    // of token 16 m + col
    f32x4 (*meet)[kMeet][64] = (f32x4 (*)[kMeet][64])lds;
#pragma unroll
    for (int first = 0; first < MT * RT; first += kMeet) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMeet; ++i) meet[wave][i][lane] = sum[(first + i) / RT][(first + i) % RT];
      __syncthreads();
      for (int i = wave; i < kMeet; i += kWaves) {
        f32x4 v = meet[0][i][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += meet[w][i][lane];
        const int m = (first + i) / RT, r = (first + i) % RT;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * r + 4 * group + e >= rank) v[e] = 0.0f;
        put(16 * m + col, 16 * r + 4 * group, v);
      }
    }
  }
};

// 8 ranks of a row's v as two 16-bit parts; what is not finite has no second one. The RB / 8
// lanes of a row are neighbours. Returns what the products are scaled by: `scale`, and in
// fp16 a power of two that brought the row's largest magnitude to 2^14..2^15.
template <typename T, int RB>
__device__ __forceinline__ float in_parts(f32x8 v, float scale, u32x4* high, u32x4* low) {
  if constexpr (T::kCode == W4A16_F16) {
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int s = 1; s < RB / 8; s <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, s));
    const int exponent = (int)(most >> 23);
    if (exponent > 0 && exponent < 255) {
      const int lift = 127 + 14 - exponent;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], lift);
      scale = __builtin_ldexpf(scale, -lift);
    } else if (exponent == 255) {
      // beside what is not finite the others only must not become infinite
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (__builtin_isfinite(v[e])) v[e] = fminf(fmaxf(v[e], -65504.0f), 65504.0f);
    }
  }
  f32x8 near = v;
  if constexpr (T::kCode != W4A16_F16) {
    // the last step below fp32's end would round to infinity
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (__builtin_isfinite(v[e])) near[e] = fminf(fmaxf(v[e], -0x1.FEp127f), 0x1.FEp127f);
  }
  const u32x4 h = narrow8<T>(near);
  const f32x8 wide = widen8<T>(h);
  f32x8 rest;
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = __builtin_isfinite(wide[e]) ? v[e] - wide[e] : 0.0f;
  *high = h;
  *low = narrow8<T>(rest);
  return scale;
}

// SUBS workgroups a tile and split. Where k is split over workgroups, the last one to arrive
// adds the splits, in their order: their sums are stored and loaded at the device's point of
// coherence (a release and acquire by fences writes back and invalidates a whole L2: 64
// tokens, 10 splits 48 us instead of 7).
template <typename T, int MT, int SUBS, int RB>
__global__ __launch_bounds__(kLoraDownThreads) void down_kernel(LoraParams p) {
  using D = Down<T, MT, RB>;
  constexpr int kRows = 16 * MT;
  __shared__ alignas(16) char lds[D::kLdsBytes];
  __shared__ alignas(16) float whole[kRows][RB];
  __shared__ int arrived;
  const int tid = threadIdx.x;
  const int64_t rows = (int64_t)blockIdx.x * kRows;
  const int adapter = adapter_of(p, blockIdx.x / SUBS);
  if (adapter < 0) return;
  const int split = blockIdx.y;
  const int64_t all_rows = (int64_t)p.tiles_most * SUBS * kRows;
  float* parts = p.parts + (split * all_rows + rows) * RB;
  const int k_lo = split * p.steps * kLoraStep;
  D::sums(p, lds, rows, adapter, rank_of(p, adapter), k_lo, min(p.k, k_lo + p.steps * kLoraStep),
          [&](int row, int r, const f32x4& v) {
            if (p.splits > 1)
              store_shared(parts + row * RB + r, v);
            else
              *(f32x4*)&whole[row][r] = v;
          });
  if (p.splits > 1) {
    wait_stores();
    __syncthreads();
    if (tid == 0) {
      arrived = __hip_atomic_fetch_add(p.counters + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == p.splits - 1)
        __hip_atomic_store(p.counters + blockIdx.x, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != p.splits - 1) return;
  } else {
    __syncthreads();
  }
  constexpr int kLanes = RB / 8;
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  for (int i = tid; i < kRows * kLanes; i += kLoraDownThreads) {
    const int row = i / kLanes, r0 = i % kLanes * 8;
    f32x8 v;
    if (p.splits > 1) {
      const float* at = p.parts + (rows + row) * RB + r0;
      v = load_shared(at);
      constexpr int kAhead = 5;
      for (int k = 1; k < p.splits; k += kAhead) {
        f32x8 next[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) next[j] = load_shared(at + min(k + j, p.splits - 1) * all_rows * RB);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + j < p.splits) v += next[j];
      }
    } else {
      v = *(const f32x8*)&whole[row][r0];
    }
    u32x4 high, low;
    const float factor = in_parts<T, RB>(v, scale, &high, &low);
    *(u32x4*)(p.high + (rows + row) * RB + r0) = high;
    *(u32x4*)(p.low + (rows + row) * RB + r0) = low;
    if (r0 == 0) p.factor[rows + row] = factor;
  }
}

// What is infinite in b meets both parts of v, and the second may be 0 or of the other sign: NaN in place of
// an infinite sum. Where a sum is NaN (asked here for a wave's) that of the first parts alone stands.
__device__ __forceinline__ bool any_nan(const f32x4 (&sum)[4]) {
  const f32x4 all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  const float any = (all.x + all.y) + (all.z + all.w);
  return __ballot(any != any) != 0;
}
__device__ __forceinline__ f32x4 where_nan(f32x4 sum, const f32x4& alone) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = sum[e] != sum[e] ? alone[e] : sum[e];
  return sum;
}

// ---- up, small tiles and ranks: a wave takes 64 columns of a tile of 16 tokens at a time. Rank
// blocks of 16 are one matrix instruction of depth 32, v's high parts in the first half and
// its low ones in the second; larger ones two for each 32 ranks. b is the left operand, its
// rows in the order that gives a lane 8 consecutive columns of its token.
template <typename T, int RB>
struct Few {
  static constexpr int KS = RB <= 16 ? 1 : RB / 32;
  static constexpr bool kPacked = RB <= 16;
  static constexpr int kParts = kPacked ? 1 : 2;       // operands of v for 32 ranks
  struct Held {
    u32x4 x[2];
  };
  struct Columns {
    u32x4 x[KS][4];
  };
  const uint16_t* base;                  // of the lane's token, at its first columns; null: 0
  uint16_t* out;
  const uint16_t* b;
  int token, group, row, rank, n_hi, rank_all;

  __device__ __forceinline__ Few(const LoraParams& p, int64_t row0, int adapter, int n_end) {
    const int lane = threadIdx.x & 63, col = lane & 15;
    token = token_of(p, row0 + col);
    group = lane >> 4;
    row = (col >> 2) * 8 + (col & 3);
    n_hi = n_end;
    rank_all = p.rank;
    rank = adapter >= 0 ? rank_of(p, adapter) : 0;
    base = p.base ? p.base + (int64_t)max(token, 0) * p.base_stride + group * 8 : nullptr;
    out = p.out + (int64_t)max(token, 0) * p.out_stride + group * 8;
    b = p.b + (int64_t)max(adapter, 0) * p.n * p.rank;
  }
  // First of the 8 ranks of the lane's operands of 32 ranks.
  __device__ __forceinline__ int rank_at(int s) const { return kPacked ? (group & 1) * 8 : 32 * s + group * 8; }
  __device__ __forceinline__ Held load_base(int n0) const {
    Held h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h.x[i] = u32x4{0, 0, 0, 0};
      if (base && token >= 0 && n0 + 32 * i + group * 8 < n_hi) h.x[i] = load16(base + n0 + 32 * i);
    }
    return h;
  }
  __device__ __forceinline__ void store_out(int n0, const Held& h) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (token >= 0 && n0 + 32 * i + group * 8 < n_hi) *(u32x4*)(out + n0 + 32 * i) = h.x[i];
  }
  // past the adapter's own rank: zeros, as 0 x NaN is NaN
  __device__ __forceinline__ u32x4 load_one(int n0, int s, int j) const {
    const int n = n0 + (j >> 1) * 32 + (j & 1) * 4 + row;
    return n < n_hi && rank_at(s) < rank ? load16(b + (int64_t)n * rank_all + rank_at(s)) : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void cut_one(u32x4& x, int s) const {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (rank_at(s) + e >= rank) x[e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
  }
  __device__ __forceinline__ Columns load_b(int n0) const {
    Columns c;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) c.x[s][j] = load_one(n0, s, j);
    return c;
  }
  __device__ __forceinline__ void cut_b(Columns& c) const {
    if ((rank & 7) == 0) return;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) cut_one(c.x[s][j], s);
  }
  // The lane's operands of v, from rows of RB high and RB low parts.
  __device__ __forceinline__ void load_v(const uint16_t* high, const uint16_t* low, u32x4 (&v)[KS][kParts]) const {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (kPacked) {
        v[s][0] = load16((group < 2 ? high : low) + rank_at(s));
      } else {
        v[s][0] = load16(high + rank_at(s));
        v[s][1] = load16(low + rank_at(s));
      }
    }
  }
  __device__ __forceinline__ Held add(int n0, Held h, const Columns& c, const u32x4 (&v)[KS][kParts], float factor) const {
    f32x4 sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < kParts; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = mfma<T>(c.x[s][j], v[s][i], sum[j]);
    if (__builtin_expect(any_nan(sum), 0)) {
      // (b once more from memory: its registers are free in all other steps)
      const bool low = kPacked && group >= 2;
      const u32x4 none{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 alone{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          u32x4 x = load_one(n0, s, j);
          cut_one(x, s);
          alone = mfma<T>(low ? none : x, low ? none : v[s][0], alone);
        }
        sum[j] = where_nan(sum[j], alone);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x8 y = widen8<T>(h.x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(sum[2 * i + e / 4][e % 4], factor, y[e]);
      h.x[i] = narrow8<T>(y);
    }
    return h;
  }
};

// b and base a step ahead. 64 tokens of 32 adapters, 17408 columns, rank 16: 6.4 us (3.5 TB/s
// of b, base and out; vector issue 43 %, waits 63 %).
template <typename T, int RB>
__global__ __launch_bounds__(kLoraThreads, 2) void up_kernel(LoraParams p) {
  using F = Few<T, RB>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = (int64_t)blockIdx.x * 16;
  const int adapter = adapter_of(p, blockIdx.x);
  if (adapter == kLoraUnused) return;
  const int n_lo = blockIdx.y * p.columns + wave * 64, n_hi = min(p.n, (int)(blockIdx.y + 1) * p.columns);
  const F f(p, row0, adapter, n_hi);
  if (adapter < 0) {
    if (p.base == p.out) return;
    for (int n0 = n_lo; n0 < n_hi; n0 += kUpColumns) f.store_out(n0, f.load_base(n0));
    return;
  }
  const int64_t row = row0 + (threadIdx.x & 15);
  u32x4 v[F::KS][F::kParts];
  f.load_v(p.high + row * RB, p.low + row * RB, v);
  const float factor = p.factor[row];
  typename F::Columns next = f.load_b(n_lo);
  typename F::Held held = f.load_base(n_lo);
  for (int n0 = n_lo; n0 < n_hi; n0 += kUpColumns) {
    typename F::Columns c = next;
    const typename F::Held now = held;
    f.cut_b(c);
    next = f.load_b(n0 + kUpColumns);
    held = f.load_base(n0 + kUpColumns);
    f.store_out(n0, f.add(n0, now, c, v, factor));
  }
}

// ---- both for a few tokens: every workgroup forms v for itself and multiplies it with its own
// columns, whose first b and base are on their way meanwhile. One launch in place of two, no
// scratch; a is read by each workgroup (the host's rule says where that pays). 64 tokens of 32
// adapters, k 5120, n 17408, rank 16: 12.7 us instead of 6.3 + 6.5, a call 11.5 instead of 14.3
// (with 512 threads and loads of 2 steps ahead 12.8, of 3 to 5 13.0 to 13.6). One token, k and
// n 4096, rank 8: 7.4 us instead of 4.8 + 3.3, a call 9.8 instead of 15.0.
template <typename T, int RB>
__global__ __launch_bounds__(lora_once_threads(RB)) void once_kernel(LoraParams p) {
  constexpr int kThreads = lora_once_threads(RB);
  using D = Down<T, 1, RB, kThreads>;
  using F = Few<T, RB>;
  __shared__ alignas(16) char lds[D::kLdsBytes];
  __shared__ alignas(16) float whole[16][RB];
  __shared__ alignas(16) uint16_t high[16][RB], low[16][RB];
  __shared__ float factors[16];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row0 = (int64_t)blockIdx.x * 16;
  const int adapter = adapter_of(p, blockIdx.x);
  if (adapter == kLoraUnused) return;
  const int n_lo = blockIdx.y * p.columns + wave * 64, n_hi = min(p.n, (int)(blockIdx.y + 1) * p.columns);
  const F f(p, row0, adapter, n_hi);
  if (adapter < 0) {
    if (p.base == p.out) return;
    for (int n0 = n_lo; n0 < n_hi; n0 += kThreads) f.store_out(n0, f.load_base(n0));
    return;
  }
  typename F::Held held = f.load_base(n_lo);
  typename F::Columns next = f.load_b(n_lo);
  D::sums(p, lds, row0, adapter, f.rank, 0, p.k, [&](int row, int r, const f32x4& v) { *(f32x4*)&whole[row][r] = v; });
  __syncthreads();
  constexpr int kLanes = RB / 8;
  if (tid < 16 * kLanes) {
    const int row = tid / kLanes, r0 = tid % kLanes * 8;
    u32x4 h, l;
    const float factor = in_parts<T, RB>(*(const f32x8*)&whole[row][r0], p.scales ? p.scales[adapter] : 1.0f, &h, &l);
    *(u32x4*)&high[row][r0] = h;
    *(u32x4*)&low[row][r0] = l;
    if (r0 == 0) factors[row] = factor;
  }
  __syncthreads();
  const int row = tid & 15;
  u32x4 v[F::KS][F::kParts];
  f.load_v(high[row], low[row], v);
  const float factor = factors[row];
  for (int n0 = n_lo; n0 < n_hi; n0 += kThreads) {
    typename F::Columns c = next;
    const typename F::Held now = held;
    f.cut_b(c);
    next = f.load_b(n0 + kThreads);
    held = f.load_base(n0 + kThreads);
    f.store_out(n0, f.add(n0, now, c, v, factor));
  }
}

// ---- up, tiles of 64 tokens, or ranks above 32: as above, in MT steps of 16 tokens with b of
// the columns in registers and v of the steps in LDS, and memory is read and written as
// whole lines, 8 lanes a row of 64 columns; b and the products are turned in LDS, each wave
// in a place of its own. Loads return in the order in which they were issued: base is loaded
// a step of columns ahead, and b of the next columns before the base that is needed after it.
// 8192 tokens, 17408 columns, rank 64: 123-127 us, 4.6 TB/s of base and out (a copy: 5.2); with
// operands read straight from memory, whose neighbouring lanes hold different rows, 162 us;
// with base two steps ahead 127-131. A third wave a SIMD has no registers for it (spills: 157).
template <typename T, int MT, int RB>
__global__ __launch_bounds__(kLoraThreads, 2) void up_lines_kernel(LoraParams p) {
  constexpr int KS = RB <= 16 ? 1 : RB / 32;
  constexpr bool kPacked = RB <= 16;
  constexpr int kRows = 16 * MT;
  constexpr int kParts = kPacked ? 1 : 2;              // loads of v for 32 ranks
  constexpr int kStride = 2 * RB + 8;                  // of v's rows in LDS: 16 bytes off the banks' period
  constexpr int kTurnB = RB < 64 ? RB : 64;            // ranks of b that are turned at a time
  constexpr int kStrideB = kTurnB + 8;                 // of b's rows
  constexpr int kStrideY = 64 + 4;                     // of the products', floats
  constexpr int kLanesB = kTurnB / 8, kRowsB = 64 / kLanesB, kLoadsB = 64 / kRowsB, kTurns = RB / kTurnB;
  constexpr int kBytes = 64 * kStrideB * 2 > 16 * kStrideY * 4 ? 64 * kStrideB * 2 : 16 * kStrideY * 4;
  __shared__ alignas(16) uint16_t vs[kRows * kStride];
  __shared__ float factors[kRows];
  __shared__ alignas(16) char turns[4][kBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, group = lane >> 4, line = lane >> 3, piece = lane & 7;
  const int64_t rows = (int64_t)blockIdx.x * kRows;
  int token[2 * MT];                       // of the lane's two rows of a step
#pragma unroll
  for (int m = 0; m < 2 * MT; ++m) token[m] = token_of(p, rows + 8 * m + line);
  const int adapter = adapter_of(p, blockIdx.x);
  if (adapter == kLoraUnused) return;
  const int n_lo = blockIdx.y * p.columns + wave * 64, n_hi = min(p.n, (int)(blockIdx.y + 1) * p.columns);
  struct Held {
    u32x4 x[2];
  };
  auto load_base = [&](int n0, int m) {
    Held h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h.x[i] = u32x4{0, 0, 0, 0};
      const int64_t at = (int64_t)token[2 * m + i] * p.base_stride + n0 + piece * 8;
      if (p.base && token[2 * m + i] >= 0 && n0 + piece * 8 < n_hi) h.x[i] = load16(p.base + at);
    }
    return h;
  };
  auto store_out = [&](int n0, int m, const Held& h) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = (int64_t)token[2 * m + i] * p.out_stride + n0 + piece * 8;
      if (token[2 * m + i] >= 0 && n0 + piece * 8 < n_hi) *(u32x4*)(p.out + at) = h.x[i];
    }
  };
  if (adapter < 0) {
    if (p.base == p.out) return;
    for (int n0 = n_lo; n0 < n_hi; n0 += kUpColumns) {
      Held h[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) h[m] = load_base(n0, m);
#pragma unroll
      for (int m = 0; m < MT; ++m) store_out(n0, m, h[m]);
    }
    return;
  }
  const int rank = rank_of(p, adapter);
  const uint16_t* b = p.b + (int64_t)adapter * p.n * p.rank;
  const int b_line = lane / kLanesB, b_piece = lane % kLanesB;
  struct Columns {
    u32x4 x[kTurns][kLoadsB];
  };
  // past the columns and the adapter's own rank: zeros, as 0 x NaN is NaN
  auto load_b = [&](int n0) {
    Columns c;
#pragma unroll
    for (int h = 0; h < kTurns; ++h)
#pragma unroll
      for (int i = 0; i < kLoadsB; ++i) {
        const int n = n0 + i * kRowsB + b_line, r0 = h * kTurnB + b_piece * 8;
        c.x[h][i] = u32x4{0, 0, 0, 0};
        if (n < n_hi && r0 < rank) c.x[h][i] = load16(b + (int64_t)n * p.rank + r0);
      }
    return c;
  };
  auto cut_b = [&](Columns& c) {
    if ((rank & 7) == 0) return;
#pragma unroll
    for (int h = 0; h < kTurns; ++h)
#pragma unroll
      for (int i = 0; i < kLoadsB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (h * kTurnB + b_piece * 8 + e >= rank) c.x[h][i][e / 2] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
  };
  constexpr int kLanesV = RB / 8;          // 16-byte pieces of a row's high (or low) parts
  for (int i = tid; i < 2 * kRows * kLanesV; i += kLoraThreads) {
    const int part = i / (kRows * kLanesV), at = i % (kRows * kLanesV);
    *(u32x4*)&vs[at / kLanesV * kStride + part * RB + at % kLanesV * 8] = load16((part ? p.low : p.high) + rows * RB + at * 8);
  }
  if (tid < kRows) factors[tid] = p.factor[rows + tid];
  Columns next = load_b(n_lo);
  Held held[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) held[m] = load_base(n_lo, m);
  __syncthreads();
  uint16_t* turn_b = (uint16_t*)turns[wave];
  float* turn_y = (float*)turns[wave];

  for (int n0 = n_lo; n0 < n_hi; n0 += kUpColumns) {
    cut_b(next);
    u32x4 bs[KS][4];
    constexpr int kDeep = KS / kTurns;     // of 32 ranks, a turn
#pragma unroll
    for (int h = 0; h < kTurns; ++h) {
#pragma unroll
      for (int i = 0; i < kLoadsB; ++i) *(u32x4*)&turn_b[(i * kRowsB + b_line) * kStrideB + b_piece * 8] = next.x[h][i];
      wave_sync();
#pragma unroll
      for (int s = 0; s < kDeep; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          bs[h * kDeep + s][j] =
              *(const u32x4*)&turn_b[(16 * j + col) * kStrideB + (kPacked ? (group & 1) * 8 : 32 * s + group * 8)];
      wave_sync();
    }
    next = load_b(n0 + kUpColumns);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f32x4 sum[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const u32x4 v = *(const u32x4*)&vs[(16 * m + col) * kStride + (kPacked ? group * 8 : i * RB + 32 * s + group * 8)];
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] = mfma<T>(bs[s][j], v, sum[j]);
        }
      // a lane holds columns 16 j + 4 group .. + 3 of token 16 m + col
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4*)&turn_y[col * kStrideY + 16 * j + 4 * group] = sum[j];
      if (__builtin_expect(any_nan(sum), 0)) {
        const bool low = kPacked && group >= 2;
        const u32x4 none{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 alone{0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const u32x4 v = *(const u32x4*)&vs[(16 * m + col) * kStride + (kPacked ? group * 8 : 32 * s + group * 8)];
            alone = mfma<T>(low ? none : bs[s][j], low ? none : v, alone);
          }
          f32x4& y = *(f32x4*)&turn_y[col * kStrideY + 16 * j + 4 * group];
          y = where_nan(y, alone);
        }
      }
      wave_sync();
      Held now = held[m];
      held[m] = load_base(n0 + kUpColumns, m);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 lo = *(const f32x4*)&turn_y[(8 * i + line) * kStrideY + piece * 8];
        const f32x4 hi = *(const f32x4*)&turn_y[(8 * i + line) * kStrideY + piece * 8 + 4];
        const float factor = factors[16 * m + 8 * i + line];
        f32x8 y = widen8<T>(now.x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(e < 4 ? lo[e & 3] : hi[e & 3], factor, y[e]);
        now.x[i] = narrow8<T>(y);
      }
      wave_sync();
      store_out(n0, m, now);
    }
  }
}

template <typename T, int MT, int RB>
hipError_t launch(const LoraParams& p, hipStream_t stream) {
  if constexpr (MT == 1 && RB <= 64) {
    if (p.splits == 0) {
      once_kernel<T, RB><<<dim3(p.tiles_most, (p.n + p.columns - 1) / p.columns), lora_once_threads(RB), 0, stream>>>(p);
      return hipGetLastError();
    }
  }
  constexpr int DOWN = MT == 4 ? kLoraDownParts : MT;
  down_kernel<T, DOWN, MT / DOWN, RB><<<dim3(p.tiles_most * (MT / DOWN), p.splits), kLoraDownThreads, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(p.tiles_most, (p.n + p.columns - 1) / p.columns);
  if constexpr (MT > 1 || RB > 32)
    up_lines_kernel<T, MT, RB><<<grid, kLoraThreads, 0, stream>>>(p);
  else
    up_kernel<T, RB><<<grid, kLoraThreads, 0, stream>>>(p);
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
