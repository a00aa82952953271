// Rotary positions and the paged key/value cache: rotate, quantise and write
// in one pass; read back.
//
// All of it is bound by HBM: a head's values are read once and written once,
// with a handful of operations each. A head is held by a group of 8, 16 or 32
// lanes, 8 dims (16 bytes) per lane, so that its row is one contiguous run of
// vector accesses, its partner dims are a second (cached) load, and its
// largest magnitude is found by shuffles inside the group.
#include <type_traits>

#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

// fp64 throughout: an fp32 angle p * f is off by up to p * 2^-24 radians
// (0.004 at p = 65536), an fp64 one by less than the rounding of the result.
__global__ __launch_bounds__(256) void rope_table_kernel(RopeTableParams p) {
  const int64_t n = p.positions * p.half;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n;
       at += (int64_t)gridDim.x * 256) {
    const int64_t row = at / p.half;
    const int i = (int)(at - row * p.half);
    double s, c;
    sincos((double)row * p.inv_freq[i], &s, &c);
    float* out = p.table + row * 2 * p.half;
    out[i] = (float)(p.amplitude * c);
    out[p.half + i] = (float)(p.amplitude * s);
  }
}

// How a lane's 8 dims meet their partners.
enum Pairing {
  kPlain,       // nothing is rotated
  kHalves,      // dims i and i + r/2, r/2 a multiple of 8: one aligned vector each
  kQuads,       // the same, r/2 a multiple of 4 only: two halves of a vector each
  kNeighbours,  // dims 2i and 2i + 1, r a multiple of 8: inside the lane
  kAny          // either, for other r: element by element
};

// Largest of the LPH lanes of a group, in all of them.
template <int LPH>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  auto dpp = [&](auto ctrl) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  dpp(std::integral_constant<int, 0xB1>{});    // lanes 1 0 3 2
  dpp(std::integral_constant<int, 0x4E>{});    // lanes 2 3 0 1
  dpp(std::integral_constant<int, 0x141>{});   // mirrored in 8
  if constexpr (LPH >= 16) dpp(std::integral_constant<int, 0x140>{});  // mirrored in 16
  if constexpr (LPH >= 32) x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  return x;
}

// One lane group takes `per_unit` (1 or 2) heads of a token in turn, so that the
// token's row of the table and its slot are read once for both. Bound by HBM:
// 16384 tokens x 48 heads into e4m3 79.8 us (4.75 TB/s; a large copy reaches
// 5.2), with one head a group 100 us, with 4 and 8 (longer waves) 90 and 126;
// a rotation of 8191 x 32 heads 25.6 us (5.3 TB/s).
template <typename T, int FMT, int LPH, Pairing PAIR>
__global__ __launch_bounds__(256) void rope_kv_kernel(RopeKvParams p) {
  const int lane = threadIdx.x % LPH;
  const int unit = blockIdx.x * (256 / LPH) + threadIdx.x / LPH;
  if (unit >= p.tokens * p.units_per_token) return;  // whole lane groups leave
  const int token = unit / p.units_per_token;
  const int first = (unit - token * p.units_per_token) * p.per_unit;
  const int last = min(first + p.per_unit, p.hq + 2 * p.hkv);
  const int d0 = 8 * lane;
  const bool live = d0 < p.dim;
  const int half = p.rot / 2;
  const bool turns = PAIR != kPlain && live && d0 < p.rot;
  // both at once, ahead of everything that waits for them
  const int64_t slot = last > p.hq ? p.slots[token] : 0;
  const int64_t pos = turns ? p.positions[token] : 0;

  // y[e] = own[e] x[e] + other[e] x[partner]; a position outside the table: NaN
  float own[8], other[8];
  if (turns) {
    const bool known = pos >= 0 && pos < p.table_rows;
    const float* row = p.table + (known ? pos : 0) * p.rot;
    const float bad = known ? 0.0f : __builtin_nanf("");
    const float flip = p.inverse ? -1.0f : 1.0f;
    if constexpr (PAIR == kHalves) {
      const int i0 = d0 < half ? d0 : d0 - half;
      const float sign = d0 < half ? -flip : flip;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const f32x4 c = *(const f32x4*)(row + i0 + e), s = *(const f32x4*)(row + half + i0 + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          own[e + j] = c[j] + bad;
          other[e + j] = sign * s[j];
        }
      }
    } else if constexpr (PAIR == kQuads) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const int d = min(d0 + e, p.rot - 4);
        const int i = d < half ? d : d - half;
        const f32x4 c = *(const f32x4*)(row + i), s = *(const f32x4*)(row + half + i);
        const float sign = d < half ? -flip : flip;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          own[e + j] = c[j] + bad;
          other[e + j] = sign * s[j];
        }
      }
    } else if constexpr (PAIR == kNeighbours) {
      const f32x4 c = *(const f32x4*)(row + d0 / 2), s = *(const f32x4*)(row + half + d0 / 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        own[e] = c[e / 2] + bad;
        other[e] = (e & 1 ? flip : -flip) * s[e / 2];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = min(d0 + e, p.rot - 1);
        const int i = p.interleaved ? d / 2 : d < half ? d : d - half;
        const bool low = p.interleaved ? (d & 1) == 0 : d < half;
        own[e] = row[i] + bad;
        other[e] = (low ? -flip : flip) * row[half + i];
      }
    }
  }
  // Loads of a head: its own vector, and with halves its partner's. All of a
  // head's lanes are in one wave, and its loads come before its stores in every
  // lane: the output may be the input.
  struct Raw {
    u32x4 own, other;
  };
  auto load = [&](const uint16_t* src) -> Raw {
    Raw r = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
    if (live) r.own = load16(src + d0);
    if constexpr (PAIR == kHalves)
      if (turns) r.other = load16(src + (d0 < half ? d0 + half : d0 - half));
    if constexpr (PAIR == kQuads)
      if (turns) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const int d = min(d0 + e, p.rot - 4);
          const u32x2 x = load8(src + (d < half ? d + half : d - half));
          r.other[e / 2] = x.x;
          r.other[e / 2 + 1] = x.y;
        }
      }
    if constexpr (PAIR == kAny)
      if (turns) {
        // elements past the rotated ones are their own partners, unused
        auto at = [&](int e) -> uint32_t {
          const int d = d0 + e;
          if (d >= p.rot) return 0;
          return src[p.interleaved ? d ^ 1 : d < half ? d + half : d - half];
        };
#pragma unroll
        for (int e = 0; e < 8; e += 2) r.other[e / 2] = at(e) | at(e + 1) << 16;
      }
    return r;
  };
  auto turn = [&](const Raw& r) -> f32x8 {
    const f32x8 x = widen8<T>(r.own);
    if constexpr (PAIR == kPlain) return x;
    const f32x8 y = PAIR == kNeighbours ? __builtin_shufflevector(x, x, 1, 0, 3, 2, 5, 4, 7, 6)
                                        : widen8<T>(r.other);
    f32x8 z = x;
    if (turns) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = fmaf(own[e], x[e], other[e] * y[e]);
        z[e] = (PAIR != kAny && PAIR != kQuads) || d0 + e < p.rot ? v : x[e];
      }
    }
    return z;
  };
  for (int h = first; h < min(last, p.hq); ++h) {
    const Raw r = load(p.q + token * p.q_token + h * p.q_head);
    const u32x4 y = turns ? narrow8<T>(turn(r)) : r.own;
    if (live) *(u32x4*)(p.q_out + token * p.out_token + h * p.out_head + d0) = y;
  }
  if (last <= p.hq) return;

  const bool kept = slot >= 0 && slot < (p.cache.pages << p.cache.page_shift);
  const int64_t page = slot >> p.cache.page_shift;
  // row of head 0's token inside its page; the next head's is a page's tokens on
  const int64_t at0 = ((page * p.cache.heads) << p.cache.page_shift) +
                      (slot & ((1 << p.cache.page_shift) - 1));
  auto write = [&](int h, const u32x4& raw, const f32x8& x, bool as_is, void* base, float* scales) {
    const int64_t at = at0 + ((int64_t)h << p.cache.page_shift);
    if constexpr (FMT == W4A16_KV_SAME) {
      const u32x4 y = as_is ? raw : narrow8<T>(x);
      if (live && kept) *(u32x4*)((uint16_t*)base + at * p.dim + d0) = y;
    } else {
      // Magnitudes compare like integers, infinities and NaN above all.
      uint32_t big = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(x[e]) & 0x7FFFFFFFu);
      big = group_max<LPH>(big);
      constexpr float kTop = FMT == W4A16_KV_E4M3 ? 448.0f : 127.0f;
      const float amax = __uint_as_float(big);
      const bool finite = big < 0x7F800000u;
      const bool some = finite && amax >= 0x1p-100f;
      const float inv = kTop / amax;
      const float scale = finite ? (some ? amax / kTop : 0.0f) : __builtin_nanf("");
      uint32_t code[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __builtin_amdgcn_fmed3f(x[e + j] * inv, -kTop, kTop);
        if constexpr (FMT == W4A16_KV_E4M3) {
          int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
          code[e / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
        } else {
          // 1.5 x 2^23 in front: the low byte of the sum is the rounded integer
          uint32_t c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(y[j] + 12582912.0f);
          code[e / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u),
                                              __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u),
                                              0x05040100u);
        }
        code[e / 4] = some ? code[e / 4] : 0u;
      }
      if (live && kept) *(u32x2*)((uint8_t*)base + at * p.dim + d0) = u32x2{code[0], code[1]};
      if (lane == 0 && kept) scales[at] = scale;
    }
  };
  for (int h = max(first, p.hq); h < min(last, p.hq + p.hkv); ++h) {
    const Raw r = load(p.k + token * p.k_token + (h - p.hq) * p.k_head);
    write(h - p.hq, r.own, turn(r), !turns, p.cache.k, p.cache.k_scale);
  }
  for (int h = max(first, p.hq + p.hkv); h < last; ++h) {
    const int hk = h - p.hq - p.hkv;
    u32x4 r = {0, 0, 0, 0};
    if (live) r = load16(p.v + token * p.v_token + hk * p.v_head + d0);
    write(hk, r, widen8<T>(r), true, p.cache.v, p.cache.v_scale);
  }
}

constexpr int kBatch = 4;  // heads whose loads a lane has in flight
static_assert(kBatch == kReadUnit, "a unit is one batch");

// Bound by HBM: 65536 tokens x 8 + 8 heads of e4m3 78.8 us (5.2 TB/s); a head at
// a time 99 us.
template <typename T, int FMT, int LPH>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadParams p) {
  const int lane = threadIdx.x % LPH;
  const int unit = blockIdx.x * (256 / LPH) + threadIdx.x / LPH;
  if (unit >= p.tokens * p.units_per_token) return;
  const int token = unit / p.units_per_token;
  const int first = (unit - token * p.units_per_token) * p.per_unit;
  const int last = min(first + p.per_unit, 2 * p.cache.heads);
  const int d0 = 8 * lane;
  if (d0 >= p.cache.dim) return;
  const int64_t slot = p.slots[token];
  const bool kept = slot >= 0 && slot < (p.cache.pages << p.cache.page_shift);
  const int64_t page = slot >> p.cache.page_shift;
  const int64_t at0 = ((page * p.cache.heads) << p.cache.page_shift) +
                      (slot & ((1 << p.cache.page_shift) - 1));
  for (int h = first; h < last; h += kBatch) {
    u32x4 raw[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      raw[i] = u32x4{0, 0, 0, 0};
      scale[i] = 0.0f;
      if (h + i < last && kept) {
        const bool is_v = h + i >= p.cache.heads;
        const int64_t at = at0 + ((int64_t)(h + i - (is_v ? p.cache.heads : 0)) << p.cache.page_shift);
        const void* base = is_v ? p.cache.v : p.cache.k;
        if constexpr (FMT == W4A16_KV_SAME) {
          raw[i] = load16((const uint16_t*)base + at * p.cache.dim + d0);
        } else {
          const u32x2 c = load8((const uint8_t*)base + at * p.cache.dim + d0);
          raw[i] = u32x4{c.x, c.y, 0, 0};
          scale[i] = (is_v ? p.cache.v_scale : p.cache.k_scale)[at];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i < last) {
        u32x4 y = raw[i];
        if constexpr (FMT != W4A16_KV_SAME) {
          const f32x4 lo = decode4<FMT>(raw[i].x) * scale[i], hi = decode4<FMT>(raw[i].y) * scale[i];
          y = kept ? narrow8<T>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)) : y;
        }
        const bool is_v = h + i >= p.cache.heads;
        const int hk = h + i - (is_v ? p.cache.heads : 0);
        *(u32x4*)((is_v ? p.v_out : p.k_out) +
                  ((int64_t)token * p.cache.heads + hk) * p.cache.dim + d0) = y;
      }
  }
}

template <typename T, int FMT, int LPH>
void (*rope_kv_of(Pairing pair))(RopeKvParams) {
  switch (pair) {
    case kPlain: return rope_kv_kernel<T, FMT, LPH, kPlain>;
    case kHalves: return rope_kv_kernel<T, FMT, LPH, kHalves>;
    case kQuads: return rope_kv_kernel<T, FMT, LPH, kQuads>;
    case kNeighbours: return rope_kv_kernel<T, FMT, LPH, kNeighbours>;
    default: return rope_kv_kernel<T, FMT, LPH, kAny>;
  }
}

template <typename T, int FMT>
hipError_t rope_kv_lanes(const RopeKvParams& p, hipStream_t stream) {
  const int lph = lanes_per_head(p.dim);
  const int64_t units = (int64_t)p.tokens * p.units_per_token;
  const dim3 grid((uint32_t)((units + 256 / lph - 1) / (256 / lph)));
  const Pairing pair = p.table == nullptr                      ? kPlain
                       : p.interleaved && p.rot % 8 == 0       ? kNeighbours
                       : !p.interleaved && p.rot % 16 == 0     ? kHalves
                       : !p.interleaved && p.rot % 8 == 0      ? kQuads
                                                               : kAny;
  const auto kernel = lph == 8    ? rope_kv_of<T, FMT, 8>(pair)
                      : lph == 16 ? rope_kv_of<T, FMT, 16>(pair)
                                  : rope_kv_of<T, FMT, 32>(pair);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <typename T, int FMT>
hipError_t kv_read_lanes(const KvReadParams& p, hipStream_t stream) {
  const int lph = lanes_per_head(p.cache.dim);
  const int64_t units = (int64_t)p.tokens * p.units_per_token;
  const dim3 grid((uint32_t)((units + 256 / lph - 1) / (256 / lph)));
  const auto kernel = lph == 8    ? kv_read_kernel<T, FMT, 8>
                      : lph == 16 ? kv_read_kernel<T, FMT, 16>
                                  : kv_read_kernel<T, FMT, 32>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_table(const RopeTableParams& p, hipStream_t stream) {
  const int64_t n = p.positions * p.half;
  const int64_t blocks = (n + 255) / 256;
  hipLaunchKernelGGL(rope_table_kernel, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_rope_kv(const RopeKvParams& p, int dtype, int format, hipStream_t stream) {
  if (dtype == W4A16_F16)
    return format == W4A16_KV_SAME   ? rope_kv_lanes<F16, W4A16_KV_SAME>(p, stream)
           : format == W4A16_KV_E4M3 ? rope_kv_lanes<F16, W4A16_KV_E4M3>(p, stream)
                                     : rope_kv_lanes<F16, W4A16_KV_INT8>(p, stream);
  return format == W4A16_KV_SAME   ? rope_kv_lanes<BF16, W4A16_KV_SAME>(p, stream)
         : format == W4A16_KV_E4M3 ? rope_kv_lanes<BF16, W4A16_KV_E4M3>(p, stream)
                                   : rope_kv_lanes<BF16, W4A16_KV_INT8>(p, stream);
}

hipError_t launch_kv_read(const KvReadParams& p, int dtype, int format, hipStream_t stream) {
  if (dtype == W4A16_F16)
    return format == W4A16_KV_SAME   ? kv_read_lanes<F16, W4A16_KV_SAME>(p, stream)
           : format == W4A16_KV_E4M3 ? kv_read_lanes<F16, W4A16_KV_E4M3>(p, stream)
                                     : kv_read_lanes<F16, W4A16_KV_INT8>(p, stream);
  return format == W4A16_KV_SAME   ? kv_read_lanes<BF16, W4A16_KV_SAME>(p, stream)
         : format == W4A16_KV_E4M3 ? kv_read_lanes<BF16, W4A16_KV_E4M3>(p, stream)
                                   : kv_read_lanes<BF16, W4A16_KV_INT8>(p, stream);
}

}  // namespace w4a16
