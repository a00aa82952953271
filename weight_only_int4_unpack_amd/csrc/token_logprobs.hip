// Log probabilities of given tokens, entropy, and the largest alternatives:
// one pass over each row of logits.
//
// A row is cut into `splits` parts, one workgroup each, whose four waves read
// tiles in turn, 64 bytes a lane, the next tile's loads on their way. Each lane
// keeps its own running reference m, s = sum e^(x - m) and t = sum e^(x - m) (x - m)
// in fp32 (e^ and t in base 2). From the joined sums
//   ln p_id = x_id - m - ln s,   entropy = ln s - ln 2 t / s
// (differences to m: no cancellation against a large maximum).
//
// Alternatives are ordered by one unsigned 64-bit key: the logit as an
// order-preserving integer above the complement of its index, so keys are
// all different, ties go to the lowest index, and "among the k largest" is an
// exact comparison against a bound. A wave's bound comes from its first tile: the
// k-th of its vectors' own largest logits is below the k largest of all, yet few
// logits pass it. Those that do go to the wave's list in LDS. The waves meet after
// the first tile, for a bound from all lists, and after the last; in between a
// tile costs one comparison a vector, and few logits of it pass.
//
// What bounds it: the stream alone (top_k = 0) runs at 3.7 TB/s and more, a copy at
// 5.2; its 10 instructions a logit are most of the difference. Selection adds
// a fixed chain of some 15 000 cycles per workgroup, of which every step
// waits for the one before (bound, list, meeting, hand-off, order), and all
// workgroups stand at the same place of it: 256 rows x 151667 bf16 take 20.9 us
// without alternatives and 33.5 us with 20 of them; 1 row 6 and 12 us.
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

constexpr int kWaves = kScoreThreads / 64;
constexpr int kWaveList = 256;           // keys of a wave's list
constexpr int kRound = 2;                // parts' keys that a thread takes at a time
constexpr int kList = kScoreMaxTop + kRound * kScoreThreads;  // keys of the workgroup's list
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  const float y = x == x ? x + 0.0f : -kInf;  // -0 as +0, NaN last
  const uint32_t u = __builtin_bit_cast(uint32_t, y);
  const uint32_t ordered = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return ((uint64_t)ordered << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  const uint32_t u = (o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o;
  return __builtin_bit_cast(float, u);
}

// log2 of e^(x - m). The difference first: x log2 e is past fp32's range for a logit masked
// by the lowest finite value, and a row may hold nothing else. (One multiply-add of x and
// of m log2 e instead: 256 rows x 151667 bf16 21.5 us instead of 22.5, with 20
// alternatives 35.1 instead of 35.9, and NaN for such a row.)
__device__ __forceinline__ float log2_of(float x, float m) { return (x - m) * kLog2e; }

// m a logit; t in units of log2.
struct Sums {
  float m, s, t;
};
// m = -inf stands for "nothing yet": its s and t are 0 (or NaN, which stays).
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == -kInf ? 0.0f : log2_of(a.m, m), db = b.m == -kInf ? 0.0f : log2_of(b.m, m);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  // 2^d d is 0 where 2^d is: the clamp keeps 0 * inf out
  const float ca = fmaxf(da, -1e4f), cb = fmaxf(db, -1e4f);
  return Sums{m, a.s * fa + b.s * fb, fa * (a.t + a.s * ca) + fb * (b.t + b.s * cb)};
}

// Logits of a type: Elem their bits, kNone a word of -inf. pack() undoes widen().
template <typename E>
struct Row;  // E: F16, BF16 or float
template <>
struct Row<float> {
  using Elem = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float one(uint32_t x) { return __uint_as_float(x); }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* x) {
    return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                 __float_as_uint(x[3])};
  }
};
template <typename T>
struct Row16 {
  using Elem = uint16_t;
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = T::kCode == W4A16_F16 ? 0xFC00FC00u : 0xFF80FF80u;
  static __device__ __forceinline__ float one(uint16_t x) { return widen1<T>(x); }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
    const f32x8 y = widen8<T>(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e];
  }
  static __device__ __forceinline__ u32x4 pack(const float* x) {
    return narrow8<T>(f32x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]});
  }
};
template <>
struct Row<F16> : Row16<F16> {};
template <>
struct Row<BF16> : Row16<BF16> {};

template <int VECS>
struct Lds {
  u32x4 held[kWaves][VECS][64];          // a tile in which logits passed
  uint64_t lists[kWaves][kWaveList];
  uint64_t list[kList + 16];
  Sums sums[kWaves];
  int32_t count[kWaves];
  int32_t last;
};

// How many of list[0..n) are larger than `key`; n rounded up to a multiple of
// 16 whose rest holds zeros (no key is larger than itself, 0 than none).
__device__ __forceinline__ int larger_than(const uint64_t* list, int n, uint64_t key) {
  int larger = 0;
#pragma unroll 1
  for (int j = 0; j < n; j += 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) larger += list[j + i] > key;
  }
  return larger;
}

// A wave's LDS accesses take effect in order; this holds the compiler to it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The largest 14 leading bits (sign, exponent, five of the mantissa) that at least k of
// the wave's N * 64 words reach, one bit a step; 0: fewer than k are not 0.
template <int N>
__device__ __forceinline__ uint32_t kth_leading(const uint32_t (&word)[N], int k) {
  uint32_t least = 0;
#pragma unroll 1
  for (uint32_t bit = 1u << 31; bit >= 1u << 18; bit >>= 1) {
    int reach = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) reach += __popcll(__ballot(word[i] >= (least | bit)));
    least |= reach >= k ? bit : 0;
  }
  return least;
}

// The k largest of the n keys of a list (room for 16 more), in order, at its
// start; returns how many there are. A key's place is the number of larger
// ones; of more than 64 those that cannot be among the k are dropped first.
// THREADS: the wave or workgroup whose threads (`at` of them) come here.
template <int THREADS, int MOST>
__device__ __forceinline__ int keep_largest(uint64_t* list, int at, int n, int k) {
  auto sync = [] {
    if constexpr (THREADS > 64)
      __syncthreads();
    else
      wave_sync();
  };
  constexpr int kEach = (MOST + THREADS - 1) / THREADS;
  uint64_t key[kEach];
  if (n > 64) {
    // every wave counts all keys, and moves those of its own chunks of 64
    constexpr int kChunks = (MOST + 63) / 64, kWaves = THREADS / 64;
    const int lane = at & 63, wave = at >> 6;
    uint32_t word[kChunks];
    int place[kEach];
    sync();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = c * 64 + lane;
      const uint64_t it = list[min(i, n - 1)];
      word[c] = i < n ? (uint32_t)(it >> 32) : 0;
      if (c % kWaves == wave) key[c / kWaves] = it;
    }
    const uint32_t least = kth_leading(word, k);
    n = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const bool in = word[c] != 0 && word[c] >= least;
      const uint64_t lanes = __ballot(in);
      if (c % kWaves == wave) place[c / kWaves] = in ? n + __popcll(lanes & ((1ull << lane) - 1)) : -1;
      n += __popcll(lanes);
    }
    sync();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i * kWaves + wave < kChunks && place[i] >= 0) list[place[i]] = key[i];
  }
  if (at < 16) list[n + at] = 0;
  sync();
  int place[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    place[i] = k;
    if ((at & ~63) + i * THREADS < n) {  // uniform over the wave
      key[i] = list[min(at + i * THREADS, n)];
      place[i] = at + i * THREADS < n ? larger_than(list, n, key[i]) : k;
    }
  }
  sync();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (place[i] < k) list[place[i]] = key[i];
  sync();
  return min(n, k);
}

// The value of the lane whose number differs in one bit (or, inside 8 and 16
// lanes, the mirrored one: enough where whole groups agree already).
template <int STEP>
__device__ __forceinline__ float other_lane(float x) {
  if constexpr (STEP >= 16) return __shfl_xor(x, STEP);
  constexpr int kCtrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xF, 0xF, true));
}
template <int STEP>
__device__ __forceinline__ Sums join_lanes(Sums a) {
  return join(a, Sums{other_lane<STEP>(a.m), other_lane<STEP>(a.s), other_lane<STEP>(a.t)});
}
__device__ __forceinline__ Sums join_wave(Sums a) {
  return join_lanes<32>(join_lanes<16>(join_lanes<8>(join_lanes<4>(join_lanes<2>(join_lanes<1>(a))))));
}

template <typename E>
__global__ __launch_bounds__(kScoreThreads, 4) void score_kernel(ScoreParams p) {
  using R = Row<E>;
  using Elem = typename R::Elem;
  constexpr int kVecs = 4, kPerLane = kVecs * R::kVec, kWaveTile = 64 * kPerLane;
  __shared__ Lds<kVecs> l;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = blockIdx.x / p.splits, part = blockIdx.x - row * p.splits;
  const Elem* x0 = (const Elem*)p.logits + row * p.row_stride;
  const int lo = part * p.part, hi = min(p.vocab, lo + p.part);
  const int k = p.top_k;
  // Vectors start at 16-byte boundaries of memory: `lead` logits before lo.
  const int lead = (int)(((uintptr_t)(x0 + lo) & 15) / sizeof(Elem));
  const int tiles = (hi - lo + lead + kWaveTile - 1) / kWaveTile;
  uint64_t* list = l.lists[wave];

  // First logit index of this lane's vector v of a tile.
  auto first_of = [&](int tile, int v) {
    return lo - lead + tile * kWaveTile + (v * 64 + lane) * R::kVec;
  };
  u32x4 raw[kVecs];
  auto load = [&](int tile) {
    const int i0 = lo - lead + tile * kWaveTile;
    if (i0 >= lo && i0 + kWaveTile <= hi) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) raw[v] = load16(x0 + first_of(tile, v));
      return;
    }
    // The part's ends: -inf in the places past them, which adds nothing.
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = first_of(tile, v);
      raw[v] = u32x4{R::kNone, R::kNone, R::kNone, R::kNone};
      if (i >= lo && i + R::kVec <= hi) raw[v] = load16(x0 + i);
    }
    // A vector across an end (the first, or the one with hi): one logit a lane, gathered
    // into the vector's lane.
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
      const int off = end == 0 ? 0 : hi - i0;
      if (end == 0 ? i0 >= lo : off >= kWaveTile) continue;
      const int i = i0 + off / R::kVec * R::kVec + lane;
      uint32_t bits = (Elem)R::kNone;
      if (lane < R::kVec && i >= lo && i < hi) bits = x0[i];
      u32x4 whole;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (sizeof(Elem) == 4)
          whole[w] = __builtin_amdgcn_readlane(bits, w);
        else
          whole[w] = __builtin_amdgcn_readlane(bits, 2 * w) |
                     __builtin_amdgcn_readlane(bits, 2 * w + 1) << 16;
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (v * 64 + lane == off / R::kVec) raw[v] = whole;
    }
  };

  // ahead of the stream, for whichever part finishes the row
  const int64_t id = p.ids[row];
  const bool known = id >= 0 && id < p.vocab;
  const float x_id = R::one(x0[known ? id : 0]);

  Sums sum{-kInf, 0.0f, 0.0f};
  int kept = 0;                          // keys in the wave's list
  uint64_t bound = 0;                    // keys below it are not among the k largest
  float x[kPerLane], most[kVecs];
  // Index of this lane's logit e of a tile.
  auto index_of = [&](int tile, int e) { return first_of(tile, e / R::kVec) + e % R::kVec; };

  auto stream = [&] {                    // x into most and sum
    // IEEE maximum: NaN where one is, which raises nothing and passes every bound
    float top = -kInf;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      most[v] = x[v * R::kVec];
#pragma unroll
      for (int e = 1; e < R::kVec; ++e)
        most[v] = __builtin_elementwise_maximum(most[v], x[v * R::kVec + e]);
      top = __builtin_elementwise_maximum(top, most[v]);
    }
    if (top > sum.m) sum = join(sum, Sums{top, 0.0f, 0.0f});
    const float ref = sum.m == -kInf ? 0.0f : sum.m;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const float d = log2_of(x[e], ref);
      const float w = __builtin_amdgcn_exp2f(d);
      sum.s += w;
      sum.t = fmaf(w, fmaxf(d, -1e4f), sum.t);
    }
  };
  // Which of the tile's logits may pass the bound, one bit each; they go to LDS, since
  // a register's number must be known and the n-th logit that passes is not.
  auto candidates = [&](int tile) {
    const float low = bound == 0 ? -kInf : value_of(bound);
    uint32_t mine = 0;                   // !(x < low): NaN is ordered as -inf
    bool any = false;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!__any(!(most[v] < low))) continue;
      any = true;
#pragma unroll
      for (int e = v * R::kVec; e < (v + 1) * R::kVec; ++e) mine |= !(x[e] < low) ? 1u << e : 0u;
    }
    if (!any) return 0u;
    const int i0 = lo - lead + tile * kWaveTile;
    if (i0 < lo || i0 + kWaveTile > hi) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {  // places past the ends are no logits
        const int i = first_of(tile, v);
        const int from = min(max(lo - i, 0), R::kVec), to = min(max(hi - i, 0), R::kVec);
        const uint32_t in = to > from ? ((1u << to) - 1) & ~((1u << from) - 1) : 0u;
        mine &= ~(((1u << R::kVec) - 1) << (v * R::kVec)) | in << (v * R::kVec);
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) l.held[wave][v][lane] = R::pack(x + v * R::kVec);
    wave_sync();
    return mine;
  };
  // Those that pass into the wave's list, one a lane at a time. It is cut back to k
  // whenever it could overflow, and to a lane a key where the waves meet afterwards.
  auto collect = [&](int tile, uint32_t mine, bool meets) {
    while (true) {
      const bool more = __any(mine != 0);
      if (kept > (more ? kWaveList - 16 - 64 : meets ? 64 : kWaveList)) {
        kept = keep_largest<64, kWaveList>(list, lane, kept, k);
        if (kept == k) bound = max(bound, list[k - 1]);
      }
      if (!more) break;
      uint64_t key = 0;
      if (mine != 0) {
        const int e = __builtin_ctz(mine);
        mine &= mine - 1;
        Elem it;
        __builtin_memcpy(&it, (const char*)&l.held[wave][e / R::kVec][lane] + e % R::kVec * sizeof(Elem),
                         sizeof(Elem));
        key = key_of(R::one(it), (uint32_t)index_of(tile, e));
      }
      const bool in = key != 0 && key >= bound;
      const uint64_t lanes = __ballot(in);
      if (in) list[kept + __popcll(lanes & ((1ull << lane) - 1))] = key;
      kept += __popcll(lanes);
    }
    wave_sync();                         // before `held` is written again
  };
  // Leading words of all waves' keys, a list in each register, and the bound they give.
  // `met` is the same in all waves, `bound` a wave's own where that is tighter.
  uint32_t words[kWaves], met = 0;
  auto meet = [&] {
    if (lane == 0) l.count[wave] = kept;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t word = (uint32_t)(l.lists[w][lane] >> 32);
      words[w] = lane < l.count[w] ? word : 0;
    }
    met = kth_leading(words, k);
    bound = max(bound, (uint64_t)met << 32);
  };

  // One copy of the code for the first tile and the others: cold instructions cost a
  // short row more than its arithmetic.
  const int rounds = (tiles + kWaves - 1) / kWaves;
#pragma unroll 1
  for (int r = -1; r < rounds; ++r) {
    const int tile = r * kWaves + wave;
    if (r >= 0 && tile < tiles) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) R::widen(raw[v], x + v * R::kVec);
    }
    if (tile + kWaves < tiles) load(tile + kWaves);
    if (r < 0) continue;
    uint32_t mine = 0;
    if (tile < tiles) {
      stream();
      if (k > 0) {
        if (r == 0) {                    // of the vectors' largest logits the k-th
          uint32_t best[kVecs];
#pragma unroll
          for (int v = 0; v < kVecs; ++v)
            best[v] = most[v] == most[v] ? (uint32_t)(key_of(most[v], 0) >> 32) : 0u;
          bound = (uint64_t)kth_leading(best, k) << 32;
        }
        mine = candidates(tile);
      }
    }
    if (k > 0) {
      const bool meets = r == 0 || r == rounds - 1;
      collect(tile, mine, meets);
      if (meets) meet();
      if (meets && r < rounds - 1) __syncthreads();  // all have read the lists
    }
  }
  if (k > 0) {                           // what passes the common bound, in order
    kept = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const bool in = words[w] != 0 && words[w] >= met;
      const uint64_t lanes = __ballot(in);
      if (w == wave && in) l.list[kept + __popcll(lanes & ((1ull << lane) - 1))] = list[lane];
      kept += __popcll(lanes);
    }
    __syncthreads();
    kept = keep_largest<kScoreThreads, kList>(l.list, tid, kept, k);
  }
  sum = join_wave(sum);
  if (lane == 0) l.sums[wave] = sum;
  __syncthreads();
  sum = l.sums[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum = join(sum, l.sums[w]);

  if (p.splits > 1) {
    // Hand-off: parts are written with device-scope stores; a full wait of
    // every wave makes them complete before the arrival is counted, and the
    // last workgroup to arrive reads them with device-scope loads. Parts are
    // joined in part order, so results do not depend on the arrival order.
    const int64_t bytes = score_part_bytes(k);
    char* rows = p.parts + (int64_t)row * p.splits * bytes;
    uint64_t* out = (uint64_t*)(rows + part * bytes);
    if (tid == 0) {
      const uint64_t a = __builtin_bit_cast(uint32_t, sum.m) |
                         ((uint64_t)__builtin_bit_cast(uint32_t, sum.s) << 32);
      __hip_atomic_store(out, a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(out + 1, (uint64_t)__builtin_bit_cast(uint32_t, sum.t), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    }
    if (tid < k)
      __hip_atomic_store(out + 2 + tid, tid < kept ? l.list[tid] : 0ull, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __syncthreads();
    if (tid == 0)
      l.last = __hip_atomic_fetch_add(p.counters + row * kScoreCounterStride, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
    __syncthreads();
    if (!l.last) return;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (tid == 0)
      __hip_atomic_store(p.counters + row * kScoreCounterStride, 0, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    auto word = [&](int s, int i) {
      return __hip_atomic_load((const uint64_t*)(rows + s * bytes) + i, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    };
    // Every wave joins the sums (one part per lane) and finds a bound: the k-th of
    // the parts' first keys, as many of each as there are lanes for.
    const int each = 64 / p.splits, of = lane / each;
    const uint64_t a = word(min(lane, p.splits - 1), 0), b = word(min(lane, p.splits - 1), 1);
    uint64_t key[kRound];
    auto fetch = [&](int from) {
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        const int i = from + j * kScoreThreads + tid;
        key[j] = i < p.splits * k ? word(i / k, 2 + i % k) : 0;
      }
    };
    if (k > 0) {
      const int rank = lane - of * each;
      const uint64_t first = of < p.splits && rank < k ? word(of, 2 + rank) : 0;
      fetch(0);
      const uint32_t words[1] = {(uint32_t)(first >> 32)};
      bound = (uint64_t)kth_leading(words, k) << 32;
    }
    sum = Sums{-kInf, 0.0f, 0.0f};
    if (lane < p.splits)
      sum = Sums{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)),
                 __uint_as_float((uint32_t)b)};
    sum = join_wave(sum);
    if (k > 0) {
      kept = 0;
#pragma unroll 1
      for (int from = 0;; from += kRound * kScoreThreads) {
        const bool more = from < p.splits * k;
        if (!more || kept > kScoreMaxTop) {
          kept = keep_largest<kScoreThreads, kList>(l.list, tid, kept, k);
          if (kept == k) bound = max(bound, l.list[k - 1]);
        }
        if (!more) break;
        if (from > 0) fetch(from);
        int place[kRound], mine = 0;
#pragma unroll
        for (int j = 0; j < kRound; ++j) {
          if (key[j] < bound) key[j] = 0;
          const uint64_t lanes = __ballot(key[j] != 0);
          place[j] = mine + __popcll(lanes & ((1ull << lane) - 1));
          mine += __popcll(lanes);
        }
        __syncthreads();
        if (lane == 0) l.count[wave] = mine;
        __syncthreads();
        int at = kept;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const int c = l.count[w];
          at += w < wave ? c : 0;
          kept += c;
        }
#pragma unroll
        for (int j = 0; j < kRound; ++j)
          if (key[j] != 0) l.list[at + place[j]] = key[j];
      }
    }
  }

  // All -inf: no softmax (m = -inf would otherwise give log 0).
  const float log_s = sum.m == -kInf ? __builtin_nanf("") : __log2f(sum.s);
  auto log_of = [&](float x) { return (x - sum.m) - kLn2 * log_s; };
  if (tid == 0) {
    p.logprobs[row] = known ? log_of(x_id) : __builtin_nanf("");
    p.entropy[row] = kLn2 * (log_s - sum.t / sum.s);
  }
  if (tid < k) {
    const uint64_t key = l.list[tid];
    p.top_logprobs[(int64_t)row * k + tid] = log_of(value_of(key));
    p.top_ids[(int64_t)row * k + tid] = 0xFFFFFFFFu - (uint32_t)key;
  }
}

}  // namespace

hipError_t launch_token_logprobs(const ScoreParams& p, int dtype, hipStream_t stream) {
  const dim3 grid((uint32_t)((int64_t)p.tokens * p.splits));
  if (dtype == W4A16_F16)
    hipLaunchKernelGGL(score_kernel<F16>, grid, dim3(kScoreThreads), 0, stream, p);
  else if (dtype == W4A16_BF16)
    hipLaunchKernelGGL(score_kernel<BF16>, grid, dim3(kScoreThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(score_kernel<float>, grid, dim3(kScoreThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace w4a16
