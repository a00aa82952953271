// Log probabilities of given tokens, entropy, and the largest alternatives:
// one pass over each row of logits.
//
// A row is cut into `splits` parts, one workgroup each, and a part into tiles
// of 8192 logits, 32 per thread. Each thread keeps its own running maximum m,
// s = sum e^(x - m) and t = sum e^(x - m) (x - m) in fp32, joined once at the
// end, so the stream has no reduction in it. From the joined sums
//   ln p_id = (x_id - m) - ln s,   entropy = ln s - t / s
// (differences to m: no cancellation against a large maximum).
//
// Alternatives are ordered by one unsigned 64-bit key: the logit as an
// order-preserving integer above the complement of its index, so keys are
// all different, ties go to the lowest index, and "among the k largest" is an
// exact comparison against a bound. The bound comes from the first tile: of
// 64 (or 256) threads' own largest keys the k-th largest is below the k
// largest keys of all, yet few keys pass it. Keys that pass go to a list in
// LDS; from then on a tile costs one comparison per thread unless one passes.
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

constexpr int kList = 1024;              // keys of the list in LDS
constexpr int kWaves = kScoreThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;
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

struct Sums {
  float m, s, t;
};
// m = -inf stands for "nothing yet": its s and t are 0 (or NaN, which stays).
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == -kInf ? 0.0f : a.m - m, db = b.m == -kInf ? 0.0f : b.m - m;
  const float fa = __builtin_amdgcn_exp2f(da * kLog2e), fb = __builtin_amdgcn_exp2f(db * kLog2e);
  // e^d d is 0 where e^d is: the clamp keeps 0 * inf out
  const float ca = fmaxf(da, -1e4f), cb = fmaxf(db, -1e4f);
  return Sums{m, a.s * fa + b.s * fb, fa * (a.t + a.s * ca) + fb * (b.t + b.s * cb)};
}

template <typename E>
struct Row;  // E: F16, BF16 or float
template <>
struct Row<float> {
  using Elem = float;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float one(float x) { return x; }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
  }
};
template <typename T>
struct Row16 {
  using Elem = uint16_t;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float one(uint16_t x) { return widen1<T>(x); }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
    const f32x8 y = widen8<T>(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e];
  }
};
template <>
struct Row<F16> : Row16<F16> {};
template <>
struct Row<BF16> : Row16<BF16> {};

struct Lds {
  uint64_t list[kList];
  uint64_t best[kScoreThreads];
  Sums sums[kWaves];
  uint64_t bound[kWaves];
  int32_t count[2][kWaves];
  int32_t last;
};

// The k largest of the n keys in the list, in order, at its start; returns
// how many there are. A key's place is the number of larger ones.
__device__ int keep_largest(Lds& l, int n, int k) {
  __syncthreads();
  uint64_t key[kList / kScoreThreads];
  int place[kList / kScoreThreads];
#pragma unroll
  for (int i = 0; i < kList / kScoreThreads; ++i) {
    const int at = threadIdx.x + i * kScoreThreads;
    place[i] = k;
    if (at < n) {
      key[i] = l.list[at];
      int larger = 0;
      for (int j = 0; j < n; ++j) larger += l.list[j] > key[i];
      place[i] = larger;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kList / kScoreThreads; ++i)
    if (place[i] < k) l.list[place[i]] = key[i];
  __syncthreads();
  return min(n, k);
}

template <typename E>
__global__ __launch_bounds__(kScoreThreads) void score_kernel(ScoreParams p) {
  using R = Row<E>;
  using Elem = typename R::Elem;
  constexpr int kVecs = kScorePerThread / R::kVec;
  __shared__ Lds l;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = blockIdx.x / p.splits, part = blockIdx.x - row * p.splits;
  const Elem* x0 = (const Elem*)p.logits + row * p.row_stride;
  const int lo = part * p.part, hi = min(p.vocab, lo + p.part);
  const int k = p.top_k;
  // Vectors start at 16-byte boundaries of memory: `lead` logits before lo.
  const int lead = (int)(((uintptr_t)(x0 + lo) & 15) / sizeof(Elem));
  const int tiles = (hi - lo + lead + kScoreTile - 1) / kScoreTile;

  // First logit index of this thread's vector v of a tile.
  auto first_of = [&](int tile, int v) {
    return lo - lead + tile * kScoreTile + (v * kScoreThreads + tid) * R::kVec;
  };
  u32x4 raw[kVecs];
  auto load = [&](int tile) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = first_of(tile, v);
      if (i >= lo && i + R::kVec <= hi) raw[v] = load16(x0 + i);
    }
  };

  Sums sum{-kInf, 0.0f, 0.0f};
  int kept = 0;                          // keys in the list, the same in every thread
  uint64_t bound = 0;                    // keys below it are not among the k largest
  load(0);
  for (int tile = 0; tile < tiles; ++tile) {
    float x[kScorePerThread];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = first_of(tile, v);
      if (i >= lo && i + R::kVec <= hi) {
        R::widen(raw[v], x + v * R::kVec);
      } else {                           // the row's ends, element by element
#pragma unroll
        for (int e = 0; e < R::kVec; ++e)
          x[v * R::kVec + e] = i + e >= lo && i + e < hi ? R::one(x0[i + e]) : -kInf;
      }
    }
    if (tile + 1 < tiles) load(tile + 1);

    float top = x[0];
#pragma unroll
    for (int e = 1; e < kScorePerThread; ++e) top = fmaxf(top, x[e]);
    if (top > sum.m) sum = join(sum, Sums{top, 0.0f, 0.0f});
    const float ref = sum.m == -kInf ? 0.0f : sum.m;
#pragma unroll
    for (int e = 0; e < kScorePerThread; ++e) {
      const float d = x[e] - ref;
      const float w = __builtin_amdgcn_exp2f(d * kLog2e);
      sum.s += w;
      sum.t = fmaf(w, fmaxf(d, -1e4f), sum.t);
    }
    if (k == 0) continue;

    auto key_at = [&](int e) -> uint64_t {  // 0: not a logit of this part
      const int i = first_of(tile, e / R::kVec) + e % R::kVec;
      return i >= lo && i < hi ? key_of(x[e], (uint32_t)i) : 0;
    };
    if (tile == 0) {
      uint64_t best = 0;
#pragma unroll
      for (int e = 0; e < kScorePerThread; ++e) best = max(best, key_at(e));
      l.best[tid] = best;
      __syncthreads();
      // up to 32 alternatives 64 threads' keys are enough (each wave finds a
      // bound of its own, the largest serves); above, the workgroup's 256
      const int from = k <= 32 ? wave * 64 : 0, n = k <= 32 ? 64 : kScoreThreads;
      int larger = 0;
      for (int j = from; j < from + n; ++j) larger += l.best[j] > best;
      if (lane == 0) l.bound[wave] = 0;
      __syncthreads();
      if (larger == k - 1 && best != 0) l.bound[wave] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) bound = max(bound, l.bound[w]);
    }
    const float low = bound == 0 ? -kInf : value_of(bound);
    int mine = 0;
    // !(top < low): a thread whose logits are NaN has top = NaN or its others' maximum
    if (!(top < low)) {
#pragma unroll
      for (int e = 0; e < kScorePerThread; ++e) {
        const uint64_t key = key_at(e);
        mine += key != 0 && key >= bound;
      }
    }
    int before = mine;                   // inclusive prefix over the wave
    if (__any(mine != 0)) {
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int o = __shfl_up(before, s);
        before += lane >= s ? o : 0;
      }
    }
    if (lane == 63) l.count[tile & 1][wave] = before;
    __syncthreads();
    int total = 0, base = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = l.count[tile & 1][w];
      base += w < wave ? c : 0;
      total += c;
    }
    if (total == 0) continue;
    if (kept + total <= kList) {
      int at = kept + base + before - mine;
      if (mine != 0) {
#pragma unroll
        for (int e = 0; e < kScorePerThread; ++e) {
          const uint64_t key = key_at(e);
          if (key != 0 && key >= bound) l.list[at++] = key;
        }
      }
      kept += total;
    } else {
      // More than the list holds (ascending or equal logits): one logit of
      // each thread at a time, the list cut back to k whenever it could
      // overflow. Unrolled: a logit's register has to be known.
#pragma unroll
      for (int e = 0; e < kScorePerThread; ++e) {
        if (kept + kScoreThreads > kList) {
          kept = keep_largest(l, kept, k);
          if (kept == k) bound = max(bound, l.list[k - 1]);
        }
        const uint64_t key = key_at(e);
        const bool in = key != 0 && key >= bound;
        const uint64_t lanes = __ballot(in);
        __syncthreads();
        if (lane == 0) l.count[0][wave] = __popcll(lanes);
        __syncthreads();
        int at = kept;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const int c = l.count[0][w];
          at += w < wave ? c : 0;
          kept += c;
        }
        if (in) l.list[at + __popcll(lanes & ((1ull << lane) - 1))] = key;
      }
      __syncthreads();                   // l.count is written again in the next tile
    }
    if (tile + 1 < tiles && kept > k) {
      kept = keep_largest(l, kept, k);
      bound = max(bound, l.list[k - 1]);
    }
  }
  if (k > 0) kept = keep_largest(l, kept, k);

#pragma unroll
  for (int s = 1; s < 64; s *= 2)
    sum = join(sum, Sums{__shfl_xor(sum.m, s), __shfl_xor(sum.s, s), __shfl_xor(sum.t, s)});
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
      l.last = __hip_atomic_fetch_add(p.counters + row, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
    __syncthreads();
    if (!l.last) return;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (tid == 0) __hip_atomic_store(p.counters + row, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    auto word = [&](int s, int i) {
      return __hip_atomic_load((const uint64_t*)(rows + s * bytes) + i, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    };
    // Every wave joins the sums (one part per lane) and finds the bound: the
    // largest of the parts' k-th keys.
    sum = Sums{-kInf, 0.0f, 0.0f};
    uint64_t kth = 0;
    if (lane < p.splits) {
      const uint64_t a = word(lane, 0);
      sum = Sums{__builtin_bit_cast(float, (uint32_t)a),
                 __builtin_bit_cast(float, (uint32_t)(a >> 32)),
                 __builtin_bit_cast(float, (uint32_t)word(lane, 1))};
      if (k > 0) kth = word(lane, 1 + k);
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      sum = join(sum, Sums{__shfl_xor(sum.m, s), __shfl_xor(sum.s, s), __shfl_xor(sum.t, s)});
      kth = max(kth, (uint64_t)__shfl_xor((unsigned long long)kth, s));
    }
    if (k > 0) {
      // 256 keys a round; the list is cut back whenever it could overflow.
      kept = 0;
      bound = kth;
      for (int from = 0; from < p.splits * k; from += kScoreThreads) {
        if (kept + kScoreThreads > kList) {
          kept = keep_largest(l, kept, k);
          if (kept == k) bound = max(bound, l.list[k - 1]);
        }
        const int i = from + tid;
        const uint64_t key = i < p.splits * k ? word(i / k, 2 + i % k) : 0;
        const bool in = key != 0 && key >= bound;
        const uint64_t lanes = __ballot(in);
        __syncthreads();
        if (lane == 0) l.count[0][wave] = __popcll(lanes);
        __syncthreads();
        int at = kept;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const int c = l.count[0][w];
          at += w < wave ? c : 0;
          kept += c;
        }
        if (in) l.list[at + __popcll(lanes & ((1ull << lane) - 1))] = key;
      }
      kept = keep_largest(l, kept, k);
    }
  }

  // All -inf: no softmax (m = -inf would otherwise give ln 0).
  const float log_s = sum.m == -kInf ? __builtin_nanf("") : logf(sum.s);
  if (tid == 0) {
    const int64_t id = p.ids[row];
    const bool known = id >= 0 && id < p.vocab;
    p.logprobs[row] = known ? (R::one(x0[known ? id : 0]) - sum.m) - log_s : __builtin_nanf("");
    p.entropy[row] = log_s - sum.t / sum.s;
  }
  if (tid < k) {
    const uint64_t key = l.list[tid];
    p.top_logprobs[(int64_t)row * k + tid] = (value_of(key) - sum.m) - log_s;
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
