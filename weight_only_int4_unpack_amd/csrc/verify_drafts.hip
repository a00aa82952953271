// Verification of drafted tokens against the model's logits, and the draw of the token
// after the accepted ones.
//
// Two kernels. The first weighs every row: a wave takes a chunk of 2048 (fp32: 1024)
// logits, finds its largest m and sums 2^((x - m) c), c = log2(e) / temperature, in fp64.
// The second has one workgroup for a sequence: it joins the chunks' sums of the sequence's
// rows, weighs the drafted tokens, walks from node to node, and draws the last token: the
// chunk in which the cumulative sum passes the border from the chunks' sums, the logit from
// that chunk alone. Where a drawn token was rejected, the weights max(w / S - q, 0) are not
// yet summed: several workgroups take a sequence's chunks, and whoever is last draws.
//
// fp64, because a draw is a border in a cumulative sum over 2^17 terms: its rounding moves
// a draw once in 1 / (terms x rounding), a hundred draws with fp32 and 10^10 with fp64.
#include "batch_internal.h"
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634074;

// 2^t for t <= 0 (NaN and -inf: 0): 2^n 2^f, n = t rounded, |f| <= 1/2. The polynomial is
// the one of degree 10 with the least largest relative error, 2^-52 (exchange method);
// below 2^-1074 there is nothing to hold.
__device__ __forceinline__ double exp2_of(double t) {
  t = __builtin_fmax(t, -1100.0);
  const double n = __builtin_rint(t), f = t - n;
  double p = 0x1.e3991e644e6abp-28;
  p = __builtin_fma(p, f, 0x1.b6740fc28f781p-24);
  p = __builtin_fma(p, f, 0x1.62c157ee59177p-20);
  p = __builtin_fma(p, f, 0x1.ffcb55e82f22cp-17);
  p = __builtin_fma(p, f, 0x1.4309126056718p-13);
  p = __builtin_fma(p, f, 0x1.5d87fe9cc5d6fp-10);
  p = __builtin_fma(p, f, 0x1.3b2ab6fbde0f7p-7);
  p = __builtin_fma(p, f, 0x1.c6b08d703d48ap-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c3b9p-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa3a17p-1);
  p = __builtin_fma(p, f, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// Weight of a logit against the row's (or chunk's) largest, m finite.
__device__ __forceinline__ double weigh(float x, double m, double c) { return exp2_of(((double)x - m) * c); }

// log2(e) / temperature of a sequence; 0: greedy.
__device__ __forceinline__ double exponent_of(const VerifyParams& p, int sequence) {
  if (!p.temperatures) return kLog2e;
  const float t = p.temperatures[sequence];
  return t > 0.0f ? kLog2e / (double)t : 0.0;
}
__device__ __forceinline__ bool is_greedy(const VerifyParams& p, int sequence) {
  return p.temperatures && !(p.temperatures[sequence] > 0.0f);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
  return x;
}
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
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) x = __builtin_elementwise_maximum(x, __shfl_xor(x, s));
  return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) x = min(x, __shfl_xor(x, s));
  return x;
}

template <typename E>
struct Logits;  // E: F16, BF16 or float
template <>
struct Logits<float> {
  using Elem = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
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
  static constexpr uint16_t kNone = T::kCode == W4A16_F16 ? 0xFC00u : 0xFF80u;
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
// l's are first .. first + kEach - 1 (`packed`) or the kVec from first + 64 kVec v, v < 4.
template <typename E>
struct Chunk {
  using L = Logits<E>;
  using Elem = typename L::Elem;
  static constexpr int kVecs = 4, kEach = kVecs * L::kVec, kSize = 64 * kEach;
  float x[kEach];
  int first;

  __device__ __forceinline__ static int lead(const Elem* row) { return (int)(((uintptr_t)row & 15) / sizeof(Elem)); }

  template <bool PACKED>
  __device__ __forceinline__ void load(const Elem* row, int vocab, int chunk, int lane) {
    const int at = chunk * kSize - lead(row);
    first = at + lane * (PACKED ? kEach : L::kVec);
    u32x4 raw[kVecs];
    if (at >= 0 && at + kSize <= vocab) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) raw[v] = load16(row + index(PACKED, v, 0));
    } else {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int i = index(PACKED, v, 0);
        if (i >= 0 && i + L::kVec <= vocab) {
          raw[v] = load16(row + i);
        } else {
          Elem e[L::kVec];
#pragma unroll
          for (int j = 0; j < L::kVec; ++j) e[j] = i + j >= 0 && i + j < vocab ? row[i + j] : L::kNone;
          raw[v] = __builtin_bit_cast(u32x4, e);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) L::widen(raw[v], x + v * L::kVec);
  }
  // Index in the row of logit j of vector v.
  __device__ __forceinline__ int index(bool packed, int v, int j) const {
    return first + v * (packed ? L::kVec : 64 * L::kVec) + j;
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

template <typename E>
__global__ __launch_bounds__(kVerifyThreads) void weigh_kernel(VerifyParams p) {
  using C = Chunk<E>;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kVerifyThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= (int64_t)p.tokens * p.chunks) return;
  const int row = (int)(unit / p.chunks), chunk = (int)(unit - (int64_t)row * p.chunks);
  C c;
  c.template load<false>((const typename C::Elem*)p.logits + row * p.row_stride, p.vocab, chunk, lane);
  bool greedy = false;
  double scale = kLog2e;
  if (p.temperatures) {
    const int b = sequence_of(p, row, lane);
    greedy = is_greedy(p, b);
    scale = exponent_of(p, b);
  }
  float m = c.x[0];
#pragma unroll
  for (int e = 1; e < C::kEach; ++e) m = __builtin_elementwise_maximum(m, c.x[e]);
  m = wave_max(m);
  VerifyChunk out{0.0, m, p.vocab};
  if (greedy) {
    int at = p.vocab;
#pragma unroll
    for (int e = C::kEach - 1; e >= 0; --e)
      if (c.x[e] == m) at = c.index(false, e / C::L::kVec, e % C::L::kVec);
    out.first = wave_min(at);
    out.s = 1.0;
  } else if (m > -kInf && m < kInf) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < C::kEach; ++e) s += weigh(c.x[e], (double)m, scale);
    out.s = wave_sum(s);
  }
  if (lane == 0) p.parts[unit] = out;
}

struct Walk {
  double weight[kVerifyMaxNodes];        // of a node's token at its parent
  double sum[kVerifyMaxNodes];           // of the weights of a node's row
  float most[kVerifyMaxNodes];           // its largest logit; not finite: no softmax
  float uniform[kVerifyMaxNodes], prob[kVerifyMaxNodes];
  int parent[kVerifyMaxNodes], token[kVerifyMaxNodes], first[kVerifyMaxNodes], path[kVerifyMaxNodes];
  int gone[kVerifyMaxNodes];             // tokens rejected at the last node
  double mass[kVerifyMaxChunks];
  int len, dropped, last_token, arrived;
  bool drawn;                            // a drawn token was rejected
};

// r of the residual: what the model gives above the draft.
__device__ __forceinline__ double above(double weight, double sum, float q) {
  return __builtin_fmax(weight / sum - (double)q, 0.0);
}

template <typename E>
__global__ __launch_bounds__(kWalkThreads) void walk_kernel(VerifyParams p) {
  using C = Chunk<E>;
  using L = typename C::L;
  using Elem = typename L::Elem;
  __shared__ Walk w;
  constexpr int kWaves = kWalkThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x / p.groups, group = blockIdx.x - b * p.groups;
  const int64_t lo = min(max(p.q_starts[b], 0), p.tokens), hi = min(max(p.q_starts[b + 1], (int)lo), p.tokens);
  const int n = (int)min(hi - lo, (int64_t)p.max_q);
  const double scale = exponent_of(p, b);
  const bool greedy = is_greedy(p, b);
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

  // Nodes: what judges them. The weight is taken below, when the rows' largest are known.
  float x_node = 0.0f;
  if (tid > 0 && tid < n) {
    int parent = tid - 1;
    if (p.parents) {
      parent = p.parents[lo + tid];
      if (parent < 0 || parent >= tid) parent = -1;
    }
    const int64_t id = p.ids[lo + tid];
    const bool known = id >= 0 && id < p.vocab;
    w.parent[tid] = parent;
    w.token[tid] = known ? (int)id : -1;
    w.uniform[tid] = p.uniforms[lo + tid];
    const bool reads = known && parent >= 0;
    x_node = reads ? L::one(logits[parent * p.row_stride + id]) : -kInf;
    w.prob[tid] = reads && p.probs ? p.probs[(lo + parent) * p.probs_stride + id] : 0.0f;
  } else if (tid == 0) {
    w.parent[0] = -1;
    w.token[0] = -1;
  }
  // Rows: their chunks joined.
  for (int i = wave; i < n; i += kWaves) {
    const VerifyChunk* part = p.parts + (lo + i) * p.chunks;
    float m = -kInf;
    for (int k = lane; k < p.chunks; k += 64) m = __builtin_elementwise_maximum(m, part[k].m);
    m = wave_max(m);
    double s = 0.0;
    int first = p.vocab;
    if (m > -kInf && m < kInf) {
      for (int k = lane; k < p.chunks; k += 64) {
        const VerifyChunk c = part[k];
        if (greedy) {
          if (c.m == m) first = min(first, c.first);
        } else if (c.m > -kInf) {
          s += c.s * weigh(c.m, (double)m, scale);
        }
      }
      s = greedy ? 1.0 : wave_sum(s);
    }
    first = wave_min(first);
    if (lane == 0) {
      w.most[i] = m;
      w.sum[i] = s;
      w.first[i] = first;
    }
  }
  __syncthreads();
  if (tid > 0 && tid < n) {
    const int parent = w.parent[tid];
    double e = 0.0;
    if (parent >= 0) {
      const float m = w.most[parent];
      if (m > -kInf && m < kInf)
        e = greedy ? (w.token[tid] == w.first[parent] ? 1.0 : 0.0) : weigh(x_node, (double)m, scale);
    }
    w.weight[tid] = e;
  }
  __syncthreads();

  if (wave == 0) {
    int node = 0, len = 1, dropped = 0;
    bool drawn = false;
    if (lane == 0) w.path[0] = 0;
    for (;;) {
      const double total = w.sum[node];
      double removed = 0.0;
      int found = -1;
      dropped = 0;
      drawn = false;
      for (int base = (node + 1) & ~63; base < n && found < 0; base += 64) {
        const int i = base + lane;
        uint64_t kids = __ballot(i > node && i < n && w.parent[min(i, n - 1)] == node);
        while (kids != 0) {
          const int c = base + __builtin_ctzll(kids);
          kids &= kids - 1;
          const double weight = w.weight[c];
          const int token = w.token[c];
          if (p.probs) {
            if ((double)w.uniform[c] * (double)w.prob[c] * total < weight) {
              found = c;
              break;
            }
            drawn = true;
          } else {
            bool before = token < 0;
            for (int j = 0; j < dropped; j += 64)
              before |= __ballot(j + lane < dropped && w.gone[min(j + lane, dropped - 1)] == token) != 0;
            if (before) continue;
            if ((double)w.uniform[c] * (total - removed) < weight) {
              found = c;
              break;
            }
            if (lane == 0) w.gone[dropped] = token;
            ++dropped;
            removed += weight;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
          }
        }
      }
      if (found < 0) break;
      if (lane == 0) w.path[len] = found;
      ++len;
      node = found;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (lane == 0) {
      w.len = len;
      w.dropped = dropped;
      w.drawn = drawn;
    }
  }
  __syncthreads();
  const int len = w.len, last = w.path[len - 1];
  const float m = w.most[last];
  const double total = w.sum[last];
  const bool sound = m > -kInf && m < kInf;
  bool residual = w.drawn && sound && !greedy;
  if (!residual && group > 0) return;

  const Elem* row = logits + last * p.row_stride;
  const float* q = p.probs ? p.probs + (lo + last) * p.probs_stride : nullptr;
  const VerifyChunk* part = p.parts + (lo + last) * p.chunks;
  int dropped = w.dropped;

  // Weights of a chunk's logits, kEach consecutive ones a lane.
  auto chunk_weights = [&](int chunk, bool over, int drop, double* r) {
    C c;
    c.template load<true>(row, p.vocab, chunk, lane);
#pragma unroll
    for (int e = 0; e < C::kEach; ++e) {
      r[e] = weigh(c.x[e], (double)m, scale);
      const int i = c.first + e;
      if (over && i >= 0 && i < p.vocab) r[e] = above(r[e], total, q[i]);
    }
    for (int j = 0; j < drop; ++j) {
      const int at = w.gone[j] - c.first;
#pragma unroll
      for (int e = 0; e < C::kEach; ++e)
        if (e == at) r[e] = 0.0;
    }
    return c.first;
  };
  auto lane_sum = [&](const double* r) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < C::kEach; ++e) s += r[e];
    return s;
  };

  if (residual && p.groups > 1) {
    for (int k = group * kWaves + wave; k < p.chunks; k += p.groups * kWaves) {
      double r[C::kEach];
      chunk_weights(k, true, 0, r);
      const double s = wave_sum(lane_sum(r));
      if (lane == 0) p.over[(int64_t)b * p.chunks + k] = s;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      w.arrived = atomicAdd(p.counters + b, 1);
      if (w.arrived == p.groups - 1) p.counters[b] = 0;
    }
    __syncthreads();
    if (w.arrived != p.groups - 1) return;
    __threadfence();
  }
  if (tid == 0) w.last_token = -1;
  if (sound && greedy) {
    if (tid == 0) w.last_token = w.first[last];
  } else if (sound) {
    const double border = (double)p.finals[b];
    // a second time over all weights where the remainder is empty
    for (int turn = 0; turn < 2; ++turn) {
      __syncthreads();
      if (residual && p.groups > 1) {
        for (int k = tid; k < p.chunks; k += kWalkThreads) w.mass[k] = p.over[(int64_t)b * p.chunks + k];
      } else if (residual) {
        for (int k = wave; k < p.chunks; k += kWaves) {
          double r[C::kEach];
          chunk_weights(k, true, 0, r);
          const double s = wave_sum(lane_sum(r));
          if (lane == 0) w.mass[k] = s;
        }
      } else {
        for (int k = tid; k < p.chunks; k += kWalkThreads) {
          const VerifyChunk c = part[k];
          w.mass[k] = c.m > -kInf ? c.s * weigh(c.m, (double)m, scale) : 0.0;
        }
        __syncthreads();
        // chunks that lost tokens: summed again without them
        for (int j = wave; j < dropped; j += kWaves) {
          const int k = (w.gone[j] + C::lead(row)) / C::kSize;
          double r[C::kEach];
          chunk_weights(k, false, dropped, r);
          const double s = wave_sum(lane_sum(r));
          if (lane == 0) w.mass[k] = s;
        }
      }
      __syncthreads();
      if (wave == 0) {
        const int each = (p.chunks + 63) / 64;
        double mine = 0.0;
        for (int k = lane * each; k < min(p.chunks, (lane + 1) * each); ++k) mine += w.mass[k];
        const double upto = wave_prefix(mine, lane);
        const double all = __shfl(upto, 63);
        if (all > 0.0) {
          const double target = border * all;
          // the chunk whose sum passes the border; by rounding none may: the last with any
          uint64_t passing = __ballot(upto > target && mine > 0.0);
          const bool none = passing == 0;
          if (none) passing = __ballot(mine > 0.0);
          const int owner = none ? 63 - __builtin_clzll(passing) : __builtin_ctzll(passing);
          double before = __shfl(upto - mine, owner);
          int chunk = 0;
          {
            double run = before, at = before;
            bool found = false;
            for (int k = owner * each; k < min(p.chunks, (owner + 1) * each); ++k) {
              if (!found && w.mass[k] > 0.0) {
                chunk = k;
                at = run;
                run += w.mass[k];
                found = !none && run > target;
              }
            }
            before = at;
          }
          double r[C::kEach];
          const int first = chunk_weights(chunk, residual, residual ? 0 : dropped, r);
          const double sum = lane_sum(r);
          const double end = before + wave_prefix(sum, lane);
          uint64_t lanes = __ballot(end > target && sum > 0.0);
          const bool past = lanes == 0;
          if (past) lanes = __ballot(sum > 0.0);
          if (lanes != 0) {
            const int who = past ? 63 - __builtin_clzll(lanes) : __builtin_ctzll(lanes);
            double run = end - sum;
            int token = -1;
            bool found = false;
#pragma unroll
            for (int e = 0; e < C::kEach; ++e) {
              if (!found && r[e] > 0.0) {
                token = first + e;
                run += r[e];
                found = !past && run > target;
              }
            }
            if (lane == who) w.last_token = token;
          }
        }
      }
      __syncthreads();
      if (w.last_token >= 0) break;
      residual = false;
      dropped = 0;
    }
  }
  __syncthreads();
  for (int i = tid; i < p.max_q; i += kWalkThreads) {
    out_tokens[i] = i + 1 < len ? (int64_t)w.token[w.path[i + 1]] : i + 1 == len ? (int64_t)w.last_token : -1;
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
  walk_kernel<E><<<(unsigned)p.sequences * (unsigned)p.groups, kWalkThreads, 0, stream>>>(p);
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
