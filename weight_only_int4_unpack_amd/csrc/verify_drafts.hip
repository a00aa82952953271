// Verification of drafted tokens against the model's logits, and the draw of the token
// after the accepted ones.
//
// Two kernels. The first weighs every row in fp32: a wave takes a chunk of 2048 (fp32: 1024)
// logits, finds its largest m and sums 2^((x - m) c), c = log2(e) / temperature. It is one
// pass over the logits. The second has one or more workgroups for a sequence: it joins the
// chunks' sums of the sequence's rows, weighs the drafted tokens, walks from node to node,
// and draws the last token from the last node's row, which it sums again in fp64, by spans of
// 1024: the span in which the cumulative sum passes the border from those sums, the logit
// from that span alone. All workgroups of a sequence walk alike and share the spans; whoever
// is last draws.
//
// What needs fp64: a draw is a border in a cumulative sum over 2^17 terms, and rounding moves
// one draw in 1 / (terms x rounding), a hundred with fp32 and 10^8 with sums that are right
// to 2^-46. The first kernel's sums are off by less than 2^-18: 56 half steps of fp32, 31 for a
// lane's additions, 23 for the three roundings of exponents that are log2 of the chunk, 11, in
// the mean over its weights at most, 2 for the exponential. A token is accepted by one comparison;
// where that sum is too near to tell (2^-16 of it), the row is summed in fp64 and compared again.
//
// Where a drawn token was rejected, the remainder R(S) = sum of max(w - S q, 0) is needed before S is
// known exactly. It is convex in S, and linear but for kinks where w = S q for a token: it is
// summed at two points around the first kernel's sum S', S' (1 -+ 2^-21), and taken between them on the
// chord. The slope at the upper one, the sum of q where w is above S q, says how far the chord may be off.
// Where that is above 2^-28 of the remainder, a sixteenth of the steps of a random number of 24
// bits (a draft that follows the model to 2^-20 in some of its mass, or a remainder of almost
// nothing), or a random number near 0 asks for more, the last workgroup sums the remainder
// again with the exact S, alone: 68 us more over 151667. Remainders below 2^-12 S come to that,
// for which few tokens are rejected; above it hardly any.
#include <climits>

#include "batch_internal.h"
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634074;

// Below 2^-1000 a weight is 0: there is no sum of weights that it would change.
constexpr double kLeast = -1000.0;

// 2^(d c) for kLeast <= d c <= 0: 2^n 2^f, n = d c rounded (by an addition that leaves it in
// the low bits), f = d c - n rounded once, |f| <= 1/2, n added to the exponent. The polynomial
// is the one of degree 9 with the least largest relative error, 2^-46 (exchange method).
__device__ __forceinline__ double exp2_of(double d, double c) {
  const double shifted = __builtin_fma(d, c, 0x1.8p52);
  const double f = __builtin_fma(d, c, -(shifted - 0x1.8p52));
  double p = 0x1.b3f421492867dp-24;
  p = __builtin_fma(p, f, 0x1.63edf1058a76ep-20);
  p = __builtin_fma(p, f, 0x1.ffce24611c0dap-17);
  p = __builtin_fma(p, f, 0x1.43088fca9a183p-13);
  p = __builtin_fma(p, f, 0x1.5d87fd9011eeep-10);
  p = __builtin_fma(p, f, 0x1.3b2ab72a1098dp-7);
  p = __builtin_fma(p, f, 0x1.c6b08d70d2003p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff81570dp-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa3752p-1);
  p = __builtin_fma(p, f, 1.0);
  typedef uint32_t Halves __attribute__((ext_vector_type(2)));
  Halves h = __builtin_bit_cast(Halves, p);
  h.y += __builtin_bit_cast(Halves, shifted).x << 20;
  return __builtin_bit_cast(double, h);
}

// How a sequence's logits are weighed: c = log2(e) / temperature, and the least difference
// that has a weight.
struct Scale {
  double c, least;
  bool greedy;
};
__device__ __forceinline__ Scale scale_of(const VerifyParams& p, int sequence) {
  Scale s{kLog2e, kLeast / kLog2e, false};
  if (p.temperatures) {
    const float t = p.temperatures[sequence];
    s.greedy = !(t > 0.0f);
    // an infinite temperature: every difference but an infinite one is 0
    s.c = s.greedy ? 1.0 : __builtin_fmax(kLog2e / (double)t, 1e-300);
    s.least = s.greedy ? 0.0 : __builtin_fmax(kLeast / kLog2e * (double)t, -1e303);
  }
  return s;
}
// Weight of a logit against the row's (or chunk's) largest, m finite; 0 for -infinity.
__device__ __forceinline__ double weigh(float x, double m, const Scale& s) {
  const double d = (double)x - m;
  const double w = exp2_of(__builtin_fmax(d, s.least), s.c);
  return d > s.least ? w : 0.0;
}
// The same with 2^-1000 in place of 0, for sums: those below kNothing are 0.
__device__ __forceinline__ double weigh_near(float x, double m, const Scale& s) {
  return exp2_of(__builtin_fmax((double)x - m, s.least), s.c);
}
constexpr double kNothing = 0x1p-900;
// The sign, the exponent and 20 bits of x.
__device__ __forceinline__ int leading(double x) {
  typedef int Halves __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(Halves, x).y;
}

// Drafted rows: how far the two points are, and what may be wrong of the remainder, and of it up to the border.
constexpr double kAside = 0x1p-21, kRemainder = 0x1p-28, kUpto = 0x1p-14;
// max(x, 0) of x <= 1, 0 for NaN: a modifier of the instruction that x comes from.
__device__ __forceinline__ double above_0(double x) { return __builtin_fmin(__builtin_fmax(x, 0.0), 1.0); }

// The value of the lane whose number differs in one bit (or, inside 8 and 16 lanes, the
// mirrored one: enough where whole groups agree already).
template <int STEP>
__device__ __forceinline__ int other_lane(int x) {
  if constexpr (STEP >= 16) return __shfl_xor(x, STEP);
  constexpr int kCtrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return __builtin_amdgcn_update_dpp(0, x, kCtrl, 0xF, 0xF, true);
}
template <int STEP>
__device__ __forceinline__ double add_lane(double x) {
  typedef int Halves __attribute__((ext_vector_type(2)));
  const Halves h = __builtin_bit_cast(Halves, x);
  return x + __builtin_bit_cast(double, Halves{other_lane<STEP>(h.x), other_lane<STEP>(h.y)});
}
// Sums over 16 lanes, in all of them, and over the wave.
__device__ __forceinline__ double row_sum(double x) { return add_lane<8>(add_lane<4>(add_lane<2>(add_lane<1>(x)))); }
__device__ __forceinline__ double wave_sum(double x) { return add_lane<32>(add_lane<16>(row_sum(x))); }
// Sum of the lanes up to this one.
__device__ __forceinline__ double wave_prefix(double x, int lane) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(x, s);
    if (lane >= s) x += y;
  }
  return x;
}
// NaN where one is.
template <int STEP>
__device__ __forceinline__ float max_lane(float x) {
  return __builtin_elementwise_maximum(x, __int_as_float(other_lane<STEP>(__float_as_int(x))));
}
__device__ __forceinline__ float row_max(float x) { return max_lane<8>(max_lane<4>(max_lane<2>(max_lane<1>(x)))); }
__device__ __forceinline__ float wave_max(float x) { return max_lane<32>(max_lane<16>(row_max(x))); }
template <int STEP>
__device__ __forceinline__ int min_lane(int x) {
  return min(x, other_lane<STEP>(x));
}
__device__ __forceinline__ int row_min(int x) { return min_lane<8>(min_lane<4>(min_lane<2>(min_lane<1>(x)))); }
__device__ __forceinline__ int wave_min(int x) { return min_lane<32>(min_lane<16>(row_min(x))); }

template <typename E>
struct Logits;  // E: F16, BF16 or float
template <>
struct Logits<float> {
  using Elem = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNoneWord = 0xFF800000u;
  static __device__ __forceinline__ float one(uint32_t x) { return __uint_as_float(x); }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
  }
};
template <typename T>
struct Logits16 {
  using Elem = uint16_t;
  static constexpr int kVec = 8;
  static constexpr uint32_t kNoneWord = T::kCode == W4A16_F16 ? 0xFC00FC00u : 0xFF80FF80u;
  static __device__ __forceinline__ float one(uint16_t x) { return widen1<T>(x); }
  static __device__ __forceinline__ void widen(u32x4 r, float* x) {
    const f32x8 y = widen8<T>(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e];
  }
};
template <>
struct Logits<F16> : Logits16<F16> {};
template <>
struct Logits<BF16> : Logits16<BF16> {};

// A chunk of a row: kEach logits a lane, -infinity in the places outside the row. Lane
// l's are the kVec from first + 64 kVec v on, v < 4.
template <typename E>
struct Chunk {
  using L = Logits<E>;
  using Elem = typename L::Elem;
  static constexpr int kVecs = 4, kEach = kVecs * L::kVec, kSize = 64 * kEach;
  u32x4 raw[kVecs];
  float x[kEach];
  int first;

  __device__ __forceinline__ static int lead(const Elem* row) { return (int)(((uintptr_t)row & 15) / sizeof(Elem)); }

  // fetch() starts the loads of a chunk, widen() takes them all.
  __device__ __forceinline__ void fetch(const Elem* row, int vocab, int chunk, int lane) {
    const int at = chunk * kSize - lead(row);
    first = at + lane * L::kVec;
    if (at >= 0 && at + kSize <= vocab) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) raw[v] = load16(row + index(v, 0));
      return;
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      raw[v] = u32x4{L::kNoneWord, L::kNoneWord, L::kNoneWord, L::kNoneWord};
      const int i = index(v, 0);
      if (i >= 0 && i + L::kVec <= vocab) raw[v] = load16(row + i);
    }
    // a vector across an end of the row: one logit a lane, gathered into the vector's lane
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
      const int i0 = across(row, vocab, end);
      if (i0 < at || i0 >= at + kSize) continue;
      const int i = i0 + lane;
      uint32_t bits = L::kNoneWord;
      if (lane < L::kVec && i >= 0 && i < vocab) bits = row[i];
      u32x4 whole;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (sizeof(Elem) == 4)
          whole[w] = __builtin_amdgcn_readlane(bits, w);
        else
          whole[w] = (__builtin_amdgcn_readlane(bits, 2 * w) & 0xFFFFu) | __builtin_amdgcn_readlane(bits, 2 * w + 1) << 16;
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (index(v, 0) == i0) raw[v] = whole;
    }
  }
  // First index of the vector that lies across the row's start or end (past both: none does).
  __device__ __forceinline__ static int across(const Elem* row, int vocab, int end) {
    const int before = lead(row);
    if (end == 0) return before > 0 ? -before : INT_MAX;
    const int rest = (vocab + before) % L::kVec;
    return rest > 0 && vocab - rest >= 0 ? vocab - rest : INT_MAX;
  }
  __device__ __forceinline__ void widen() {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) L::widen(raw[v], x + v * L::kVec);
  }
  // Index in the row of logit j of vector v.
  __device__ __forceinline__ int index(int v, int j) const {
    return first + v * (64 * L::kVec) + j;
  }
};

// One vector a lane of a chunk, and of a draft's row in the same places: -infinity, and 0,
// outside the row.
template <typename E, bool DRAFT>
struct Part {
  using C = Chunk<E>;
  using L = Logits<E>;
  static constexpr int kDrafts = DRAFT ? L::kVec / 4 : 1;
  u32x4 raw;
  f32x4 draft[kDrafts];
  int first;

  __device__ __forceinline__ void fetch(const typename L::Elem* row, const float* q, int vocab, int at, int lane) {
    typedef f32x4 Loose __attribute__((aligned(4)));
    first = at + lane * L::kVec;
    if (at >= 0 && at + 64 * L::kVec <= vocab) {
      raw = load16(row + first);
      if constexpr (DRAFT) {
#pragma unroll
        for (int j = 0; j < kDrafts; ++j) draft[j] = *(const Loose*)(q + first + 4 * j);
      }
      return;
    }
    raw = u32x4{L::kNoneWord, L::kNoneWord, L::kNoneWord, L::kNoneWord};
    const bool whole = first >= 0 && first + L::kVec <= vocab;
    if (whole) raw = load16(row + first);
#pragma unroll
    for (int j = 0; j < kDrafts; ++j) {
      draft[j] = f32x4{0, 0, 0, 0};
      if (DRAFT && whole) draft[j] = *(const Loose*)(q + first + 4 * j);
    }
    // a vector across an end of the row: one logit a lane, gathered into the vector's lane
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
      const int i0 = C::across(row, vocab, end);
      if (i0 < at || i0 >= at + 64 * L::kVec) continue;
      const int i = i0 + lane;
      uint32_t bits = L::kNoneWord;
      float mine = 0.0f;
      if (lane < L::kVec && i >= 0 && i < vocab) {
        bits = row[i];
        if (DRAFT) mine = q[i];
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t word = __builtin_amdgcn_readlane(bits, w);
        if constexpr (sizeof(typename L::Elem) == 2)
          word = (__builtin_amdgcn_readlane(bits, 2 * w) & 0xFFFFu) | __builtin_amdgcn_readlane(bits, 2 * w + 1) << 16;
        if (first == i0) raw[w] = word;
      }
      if constexpr (DRAFT) {
#pragma unroll
        for (int j = 0; j < L::kVec; ++j) {
          const float y = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), j));
          if (first == i0) draft[j / 4][j % 4] = y;
        }
      }
    }
  }
};

// The largest b with q_starts[b] <= row, of 0..sequences-1: 64 places are looked at a time.
__device__ __forceinline__ int sequence_of(const VerifyParams& p, int row, int lane) {
  int lo = 0, span = p.sequences;
  while (span > 1) {
    const int step = (span + 63) / 64;
    const int at = lane * step;
    const bool in = at < span && p.q_starts[lo + min(at, span - 1)] <= row;
    const int reach = __popcll(__ballot(in));
    const int go = max(reach - 1, 0) * step;
    lo += go;
    span = min(step, span - go);
  }
  return lo;
}

// Logits' weights in fp32 where the scale is an ordinary one; others (infinite and
// vanishing temperatures) in fp64. Bound by HBM and issue together: 288 rows of 151667 in
// bf16 17.5 us, 5.0 TB/s, vector issue 72 % (weighed in fp64, 40 us).
template <typename E>
__global__ __launch_bounds__(kVerifyThreads) void weigh_kernel(VerifyParams p) {
  using C = Chunk<E>;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kVerifyThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = (int)(unit / p.chunks), chunk = (int)(unit - (int64_t)row * p.chunks);
  if (row >= p.tokens) return;
  C c;
  c.fetch((const typename C::Elem*)p.logits + row * p.row_stride, p.vocab, chunk, lane);
  const Scale scale = scale_of(p, p.temperatures ? sequence_of(p, row, lane) : 0);
  c.widen();
  float m = c.x[0];
#pragma unroll
  for (int e = 1; e < C::kEach; ++e) m = __builtin_elementwise_maximum(m, c.x[e]);
  m = wave_max(m);
  VerifyChunk out{0.0, m, p.vocab};
  if (scale.greedy) {
    int at = p.vocab;
#pragma unroll
    for (int e = C::kEach - 1; e >= 0; --e)
      if (c.x[e] == m) at = c.index(e / C::L::kVec, e % C::L::kVec);
    out.first = wave_min(at);
    out.s = 1.0;
  } else if (m > -kInf && m < kInf) {
    if (scale.c > 1e-30 && scale.c < 1e30) {
      const float rate = (float)scale.c;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < C::kEach; ++e) s += __builtin_amdgcn_exp2f((c.x[e] - m) * rate);
      out.s = wave_sum((double)s);
    } else {
      double s = 0.0;
#pragma unroll
      for (int e = 0; e < C::kEach; ++e) s += weigh(c.x[e], (double)m, scale);
      out.s = wave_sum(s);
    }
  }
  if (lane == 0) p.parts[unit] = out;
}

// A sequence's nodes in LDS, for as many as a call may have.
struct Walk {
  double* weight;                        // of a node's token at its parent
  double* sum;                           // of the weights of a node's row
  double* mass;                          // of a row's spans
  float* most;                           // a row's largest logit; not finite: no softmax
  float* uniform;
  float* prob;
  int* parent;
  int* token;
  int* first;                            // greedy: where the row's largest logit stands; else -1: an fp64 sum
  int* path;
  int* gone;                             // tokens rejected at the last node, each once
};
constexpr int kNodeBytes = 2 * 8 + 8 * 4;
__host__ __device__ constexpr int walk_bytes(int nodes, int spans) { return nodes * kNodeBytes + spans * 8; }

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ void store_shared(double* to, double x) {
  __hip_atomic_store((uint64_t*)to, __builtin_bit_cast(uint64_t, x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double load_shared(const double* from) {
  return __builtin_bit_cast(double, __hip_atomic_load((const uint64_t*)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// A chain of loads and barriers: one sequence over 32000 logits 13 us. 64 chains over 151667
// with drafts 29.0, of which 58 MB of rows and drafts take 15.5 (HBM 11; a row's loads are two
// vectors ahead of the weighing: a chunk's at once take 3 us more; the remainder at S' alone 1.1 less).
template <typename E>
__global__ __launch_bounds__(kWalkThreads, 4) void walk_kernel(VerifyParams p) {
  using C = Chunk<E>;
  using L = typename C::L;
  using Elem = typename L::Elem;
  constexpr int kWaves = kWalkThreads / 64;
  extern __shared__ double lds[];
  __shared__ double sums_[kWaves], before_, target_;
  __shared__ int node_, len_, need_, dropped_, token_, arrived, span_, who_, last_[kWaves];
  __shared__ bool drawn_;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x / p.groups, group = blockIdx.x - b * p.groups;
  Walk w;
  {
    const int most = max(p.max_q, 1);
    w.weight = lds;
    w.sum = w.weight + most;
    w.mass = w.sum + most;
    w.most = (float*)(w.mass + p.spans);
    w.uniform = w.most + most;
    w.prob = w.uniform + most;
    w.parent = (int*)(w.prob + most);
    w.token = w.parent + most;
    w.first = w.token + most;
    w.path = w.first + most;
    w.gone = w.path + most;
  }
  const int64_t lo = min(max(p.q_starts[b], 0), p.tokens), hi = min(max(p.q_starts[b + 1], (int)lo), p.tokens);
  const int n = (int)min(hi - lo, (int64_t)p.max_q);
  const Scale scale = scale_of(p, b);
  const bool greedy = scale.greedy;
  const double border = (double)p.finals[b];
  const Elem* logits = (const Elem*)p.logits + lo * p.row_stride;
  int64_t* out_tokens = p.out_tokens + (int64_t)b * p.max_q;
  int32_t* out_path = p.path + (int64_t)b * p.max_q;
  if (n <= 0) {
    if (group > 0) return;
    for (int i = tid; i < p.max_q; i += kWalkThreads) {
      out_tokens[i] = -1;
      out_path[i] = -1;
    }
    if (tid == 0) p.counts[b] = 0;
    return;
  }

  // Nodes: what judges them, on its way while the rows are joined.
  constexpr int kEachNode = kVerifyMaxNodes / kWalkThreads;
  float x_node[kEachNode], uniform[kEachNode], prob[kEachNode];
  int parent_of[kEachNode], token_of[kEachNode];
#pragma unroll
  for (int e = 0; e < kEachNode; ++e) {
    const int i = tid + e * kWalkThreads;
    x_node[e] = -kInf;
    uniform[e] = prob[e] = 0.0f;
    parent_of[e] = token_of[e] = -1;
    if (i >= n) continue;
    int parent = i - 1;
    if (p.parents && i > 0) {
      parent = p.parents[lo + i];
      if (parent < 0 || parent >= i) parent = -1;
    }
    const int64_t id = p.ids[lo + i];
    const bool known = id >= 0 && id < p.vocab;
    const bool reads = known && parent >= 0;
    if (reads) x_node[e] = L::one(logits[parent * p.row_stride + id]);
    if (reads && p.probs) prob[e] = p.probs[(lo + parent) * p.probs_stride + id];
    uniform[e] = p.uniforms[lo + i];
    parent_of[e] = parent;
    token_of[e] = known ? (int)id : -1;
  }
  // Rows: their chunks joined, 16 lanes a row.
  {
    const int part_lane = lane & 15;
    for (int base = wave * 4; base < n; base += kWaves * 4) {
      const int i = base + (lane >> 4);
      const VerifyChunk* part = p.parts + (lo + min(i, n - 1)) * p.chunks;
      float m = -kInf;
      double s = 0.0;
      int first = p.vocab;
      constexpr int kAhead = 5;
      for (int k0 = part_lane; k0 < p.chunks; k0 += 16 * kAhead) {
        VerifyChunk c[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          c[j] = part[min(k0 + 16 * j, p.chunks - 1)];
          if (k0 + 16 * j >= p.chunks) c[j].m = -kInf;
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) top = __builtin_elementwise_maximum(top, c[j].m);
        if (top > m) first = p.vocab;
        if (greedy) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (c[j].m == top) first = min(first, c[j].first);
        } else if (top > -kInf && top < kInf) {
          s = m > -kInf ? s * weigh(m, (double)top, scale) : 0.0;
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (c[j].m > -kInf) s += c[j].s * weigh(c[j].m, (double)top, scale);
        }
        m = top;
      }
      const float top = row_max(m);
      const bool finite = top > -kInf && top < kInf;
      s = finite && m > -kInf ? s * weigh(m, (double)top, scale) : 0.0;
      if (m != top) first = p.vocab;
      s = row_sum(s);
      first = row_min(first);
      if (part_lane == 0 && i < n) {
        w.most[i] = top;
        w.sum[i] = !finite ? 0.0 : greedy ? 1.0 : s;
        w.first[i] = first;
      }
    }
  }
  if (tid == 0) {
    w.path[0] = 0;
    node_ = 0;
    len_ = 1;
    token_ = -1;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEachNode; ++e) {
    const int i = tid + e * kWalkThreads;
    if (i >= n) continue;
    const int parent = parent_of[e];
    double weight = 0.0;
    if (parent >= 0) {
      const float m = w.most[parent];
      if (m > -kInf && m < kInf)
        weight = greedy ? (token_of[e] == w.first[parent] ? 1.0 : 0.0) : weigh(x_node[e], (double)m, scale);
    }
    w.weight[i] = weight;
    w.parent[i] = parent;
    w.token[i] = token_of[e];
    w.uniform[i] = uniform[e];
    w.prob[i] = prob[e];
  }
  __syncthreads();

  // Sum of mass[0..spans), by one wave, in all its lanes; the lanes' own and what is before.
  auto sum_mass = [&](double* mine, double* upto) {
    const int each = (p.spans + 63) / 64;
    *mine = 0.0;
    for (int k = lane * each; k < min(p.spans, (lane + 1) * each); ++k) *mine += w.mass[k];
    *upto = wave_prefix(*mine, lane);
    return __shfl(*upto, 63);
  };

  // Stages that end in spans' sums, with one copy of code: the walk up to a row whose sum is
  // too near to tell; the last row; its remainder above a draft again, with the row's exact sum; that
  // row with all its weights, where the remainder is empty.
  enum { kWalking, kDrawing, kDrawingExact, kDrawingAll };
  constexpr int kNoSpan = -1, kInexact = -2;   // in place of a span: nothing is left; the remainder may be wrong
  int stage = kWalking, len = 1, last = 0;
  for (;;) {
    int node = 0, from = wave, step = kWaves, dropped = 0;
    const float* q = nullptr;
    if (stage == kWalking) {
      if (wave == 0) {
        int at = node_, count = len_, gone = 0, need = -1;
        bool drawn = false;
        for (;;) {
          const double total = w.sum[at];
          const bool rough = !greedy && w.first[at] >= 0;
          double removed = 0.0;
          int found = -1;
          gone = 0;
          drawn = false;
          for (int base = (at + 1) & ~63; base < n && found < 0 && need < 0; base += 64) {
            const int i = base + lane;
            uint64_t kids = __ballot(i > at && i < n && w.parent[min(i, n - 1)] == at);
            while (kids != 0) {
              const int c = base + __builtin_ctzll(kids);
              kids &= kids - 1;
              const double weight = w.weight[c], u = (double)w.uniform[c];
              const int token = w.token[c];
              if (!p.probs) {
                bool before = token < 0;
                for (int j = 0; j < gone; j += 64)
                  before |= __ballot(j + lane < gone && w.gone[min(j + lane, gone - 1)] == token) != 0;
                if (before) continue;
              }
              const double rate = p.probs ? u * (double)w.prob[c] : u;
              const double least = rate * (total - removed);
              if (rough && __builtin_fabs(least - weight) <= 0x1p-16 * rate * total) {
                need = at;
                break;
              }
              if (least < weight) {
                found = c;
                break;
              }
              drawn = p.probs != nullptr;
              if (!drawn) {
                if (lane == 0) w.gone[gone] = token;
                ++gone;
                removed += weight;
                wave_sync();
              }
            }
            if (p.probs) break;          // a chain: there are no others
          }
          if (found < 0) break;
          if (lane == 0) w.path[count] = found;
          ++count;
          at = found;
          wave_sync();
        }
        if (lane == 0) {
          node_ = at;
          len_ = count;
          need_ = need;
          dropped_ = gone;
          drawn_ = drawn;
        }
      }
      __syncthreads();
      node = need_;
      if (node < 0) {
        len = len_;
        last = w.path[len - 1];
        const bool sound = w.most[last] > -kInf && w.most[last] < kInf;
        if (greedy || !sound) {
          if (group > 0) return;
          if (tid == 0 && sound) token_ = w.first[last];
          break;
        }
        stage = kDrawing;
      }
    }
    if (stage != kWalking) node = last;
    const Elem* row = logits + node * p.row_stride;
    const double m = (double)w.most[node], near = w.sum[node];
    if (stage == kDrawing) {
      from = group * kWaves + wave;
      step = p.groups * kWaves;
      dropped = dropped_;
    }
    if ((stage == kDrawing || stage == kDrawingExact) && drawn_) q = p.probs + (lo + last) * p.probs_stride;
    double* shared = p.over + (int64_t)b * 3 * p.spans;

    // Of each span, by a wave: the sum of the weights without the rejected tokens, and, over
    // a draft, the remainder at two points around `near`, as the upper's and the difference; what
    // that is above the slope's is summed over the wave's spans. Loads of two vectors are on
    // their way while one is weighed.
    auto weigh_spans = [&](auto drafted) {
      constexpr bool kDraft = decltype(drafted)::value;
      using P = Part<E, kDraft>;
      constexpr int kVecs = kVerifySpan / (64 * L::kVec);
      const int count = from < p.spans ? (p.spans - from + step - 1) / step : 0;
      const double aside = stage == kDrawing ? kAside * near : 0.0, lower = near - aside, upper = near + aside;
      double s = 0.0, over = 0.0, over_lower = 0.0, bent = 0.0;
      float under = 0.0f;
      auto fetch = [&](P& part, int unit) {
        const int span = from + unit / kVecs * step;
        part.fetch(row, q, p.vocab, span * kVerifySpan - C::lead(row) + unit % kVecs * (64 * L::kVec), lane);
      };
      auto add = [&](const P& part) {
        float x[L::kVec];
        L::widen(part.raw, x);
        for (int j = 0; j < dropped; ++j) {
          const int at = w.gone[j] - part.first;
#pragma unroll
          for (int e = 0; e < L::kVec; ++e)
            if (e == at) x[e] = -kInf;
        }
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) {
          const double y = weigh_near(x[e], m, scale);
          s += y;
          if constexpr (kDraft) {
            const float d = part.draft[e / 4][e % 4];
            const double r = above_0(__builtin_fma(-upper, (double)d, y));
            over += r;
            over_lower += above_0(__builtin_fma(-lower, (double)d, y));
            under += leading(r) != 0 ? d : 0.0f;
          }
        }
      };
      auto finish = [&](int unit) {
        const int k = from + unit / kVecs * step;
        if (k >= p.spans) return;
        f32x2 slope{0.0f, 0.0f};
        if constexpr (kDraft) {
          const double step_up = over_lower - over;
          slope.x = (float)wave_sum(step_up);
          bent += __builtin_fma(-2.0 * aside, (double)under, step_up);
          if (k + step >= p.spans) slope.y = (float)wave_sum(bent);
          over = wave_sum(over);
          over = over > kNothing ? over : 0.0;
        }
        s = wave_sum(s);
        s = s > kNothing ? s : 0.0;
        if (lane == 0) {
          if (stage == kDrawing) {
            store_shared(shared + k, s);
            if constexpr (kDraft) {
              store_shared(shared + p.spans + k, over);
              store_shared(shared + 2 * p.spans + k, __builtin_bit_cast(double, slope));
            }
          } else {
            w.mass[k] = kDraft ? over : s;
          }
        }
        s = over = over_lower = 0.0;
        under = 0.0f;
      };
      P part[2];
#pragma unroll 1
      for (int unit = -2; unit < count * kVecs; unit += 2) {
        const bool more = unit + 2 < count * kVecs;
        if (unit >= 0) add(part[0]);
        if (more) fetch(part[0], unit + 2);
        if (kVecs == 1 && unit >= 0) finish(unit);
        if (unit >= 0) add(part[1]);
        if (more) fetch(part[1], unit + 3);
        if (unit >= 0 && (unit + 2) % kVecs == 0) finish(unit + 1);
      }
    };
    if (q)
      weigh_spans(std::bool_constant<true>{});
    else
      weigh_spans(std::bool_constant<false>{});
    double total = 0.0;
    if (stage == kDrawing) {
      // stores at the device's point of coherence, complete before this workgroup arrives
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __syncthreads();
      if (p.groups > 1) {
        if (tid == 0) {
          arrived = __hip_atomic_fetch_add(p.counters + b, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          if (arrived == p.groups - 1)
            __hip_atomic_store(p.counters + b, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (arrived != p.groups - 1) return;
      }
      constexpr int kEachSpan = (kVerifyMaxSpans + kWalkThreads - 1) / kWalkThreads;
      double over[kEachSpan];
      f32x2 slope[kEachSpan];
#pragma unroll
      for (int e = 0; e < kEachSpan; ++e) {
        const int k = tid + e * kWalkThreads;
        over[e] = 0.0;
        slope[e] = f32x2{0.0f, 0.0f};
        if (k >= p.spans) continue;
        w.mass[k] = load_shared(shared + k);
        if (q) {
          over[e] = load_shared(shared + p.spans + k);
          slope[e] = __builtin_bit_cast(f32x2, load_shared(shared + 2 * p.spans + k));
        }
      }
      __syncthreads();
      if (q) {
        if (wave == 0) {
          double mine, upto;
          const double all = sum_mass(&mine, &upto);
          if (lane == 0) target_ = all;
        }
        __syncthreads();
        total = target_;
        // what may be wrong: the difference to the slope, and as much as its 16 additions may hide
        const double by = 0.5 + (near - total) / (2.0 * kAside * near);
        double wrong = 0.0;
#pragma unroll
        for (int e = 0; e < kEachSpan; ++e) {
          const int k = tid + e * kWalkThreads;
          if (k < p.spans) w.mass[k] = __builtin_fma(by, (double)slope[e].x, over[e]);
          wrong += __builtin_fma(0x1p-20, (double)slope[e].x, (double)slope[e].y);
        }
        wrong = wave_sum(wrong);
        if (lane == 0) sums_[wave] = wrong;
      }
    } else if (stage == kDrawingExact) {
      total = near;
    }
    __syncthreads();
    if (wave == 0) {
      // the span whose sum passes the border; by rounding none may: the last with any
      double mine, upto;
      const double all = sum_mass(&mine, &upto), target = border * all;
      if (stage == kWalking) {
        if (lane == 0) {
          w.sum[node] = all;
          w.first[node] = -1;
        }
      } else {
        const int each = (p.spans + 63) / 64;
        uint64_t passing = __ballot(upto > target && mine > 0.0);
        const bool none = passing == 0;
        if (none) passing = __ballot(mine > 0.0);
        int span = kNoSpan;
        double before = 0.0;
        if (all > 0.0 && passing != 0) {
          const int owner = none ? 63 - __builtin_clzll(passing) : __builtin_ctzll(passing);
          double run = __shfl(upto - mine, owner);
          bool found = false;
          for (int k = owner * each; k < min(p.spans, (owner + 1) * each) && !found; ++k) {
            if (w.mass[k] > 0.0) {
              span = k;
              before = run;
              run += w.mass[k];
              found = !none && run > target;
            }
          }
        }
        if (stage == kDrawing && q) {
          double wrong = 0.0;
          for (int i = 0; i < kWaves; ++i) wrong += sums_[i];
          if (__builtin_fabs(near - total) > kAside * near || wrong > kRemainder * all || wrong > kUpto * target)
            span = kInexact;
          if (lane == 0) w.sum[node] = total;
        }
        if (lane == 0) {
          span_ = span;
          before_ = before;
          target_ = target;
        }
      }
    }
    __syncthreads();
    if (stage == kWalking) continue;
    if (span_ >= 0) {
      // that span by the whole workgroup, kFew consecutive logits a thread
      constexpr int kFew = kVerifySpan / kWalkThreads;
      const int first = span_ * kVerifySpan - C::lead(row) + tid * kFew;
      double r[kFew], sum = 0.0;
#pragma unroll
      for (int e = 0; e < kFew; ++e) {
        const int i = first + e, at = min(max(i, 0), p.vocab - 1);
        const float x = L::one(row[at]), draft = q ? q[at] : 0.0f;
        r[e] = weigh(i == at ? x : -kInf, m, scale);
        if (q) r[e] = i == at ? __builtin_fmax(__builtin_fma(-total, (double)draft, r[e]), 0.0) : 0.0;
      }
      for (int j = 0; j < dropped; ++j) {
        const int at = w.gone[j] - first;
#pragma unroll
        for (int e = 0; e < kFew; ++e)
          if (e == at) r[e] = 0.0;
      }
#pragma unroll
      for (int e = 0; e < kFew; ++e) sum += r[e];
      const double target = target_;
      const double upto = wave_prefix(sum, lane);
      if (lane == 63) sums_[wave] = upto;
      if (tid == 0) who_ = kWalkThreads;
      __syncthreads();
      double before = before_;
      for (int i = 0; i < wave; ++i) before += sums_[i];
      // the first thread that passes the border, or, by rounding, the last with anything
      const uint64_t lanes = __ballot(sum > 0.0 && before + upto > target), any = __ballot(sum > 0.0);
      if (lane == 0 && lanes != 0) atomicMin(&who_, tid + __builtin_ctzll(lanes));
      if (lane == 0) last_[wave] = any != 0 ? tid + 63 - __builtin_clzll(any) : -1;
      __syncthreads();
      int who = who_;
      const bool past = who == kWalkThreads;
      if (past)
        for (int i = 0; i < kWaves; ++i) who = last_[i] >= 0 ? last_[i] : who;
      if (tid == who) {
        double run = before + upto - sum;
        int token = -1;
        bool found = false;
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
          if (!found && r[e] > 0.0) {
            token = first + e;
            run += r[e];
            found = !past && run > target;
          }
        }
        token_ = token;
      }
    }
    __syncthreads();
    if (token_ >= 0 || stage == kDrawingAll) break;
    // (a span's remainder may be a rounding alone, of which no token has any)
    stage = stage == kDrawing && drawn_ && span_ != kNoSpan ? kDrawingExact : kDrawingAll;
  }
  __syncthreads();
  for (int i = tid; i < p.max_q; i += kWalkThreads) {
    out_tokens[i] = i + 1 < len ? (int64_t)w.token[w.path[i + 1]] : i + 1 == len ? (int64_t)token_ : -1;
    out_path[i] = i < len ? w.path[i] : -1;
  }
  if (tid == 0) p.counts[b] = len;
}

template <typename E>
hipError_t launch(const VerifyParams& p, hipStream_t stream) {
  const int64_t units = (int64_t)p.tokens * p.chunks;
  constexpr int kEach = kVerifyThreads / 64;
  if (units > 0) {
    weigh_kernel<E><<<(unsigned)((units + kEach - 1) / kEach), kVerifyThreads, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  walk_kernel<E><<<(unsigned)p.sequences * (unsigned)p.groups, kWalkThreads,
                   walk_bytes(p.max_q > 0 ? p.max_q : 1, p.spans), stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case W4A16_F16: return launch<F16>(p, stream);
    case W4A16_BF16: return launch<BF16>(p, stream);
    default: return launch<float>(p, stream);
  }
}

}  // namespace w4a16
