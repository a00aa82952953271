// Rotary positions and the paged key/value cache: rotate, quantise and write
// in one pass; read back.
//
// All of it is bound by HBM: a head's values are read once and written once,
// with a handful of operations each. A head is held by a group of 8, 16 or 32
// lanes, 8 dims (16 bytes) per lane, so that its row is one contiguous run of
// vector accesses, its partner dims are a second (cached) load, and its
// largest magnitude is found by shuffles inside the group.
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

// Factors of a lane's 8 dims d0..d0+7: y[e] = own[e] x[e] + other[e] x[partner].
struct Turn {
  float own[8], other[8];
};

template <typename T, int FMT, int LPH>
__global__ __launch_bounds__(256) void rope_kv_kernel(RopeKvParams p) {
  const int lane = threadIdx.x % LPH;
  const int unit = blockIdx.x * (256 / LPH) + threadIdx.x / LPH;
  if (unit >= p.tokens * p.units_per_token) return;  // whole lane groups leave
  const int token = unit / p.units_per_token;
  const int first = (unit - token * p.units_per_token) * p.per_unit;
  const int heads = p.hq + 2 * p.hkv;
  const int last = min(first + p.per_unit, heads);
  const int d0 = 8 * lane;
  const bool live = d0 < p.dim;
  const int half = p.rot / 2;
  // Whole vectors: a lane's 8 dims are rotated all or none, and their
  // partners are one aligned vector (halves) or the lane's own (neighbours).
  const bool vec = p.interleaved ? p.rot % 8 == 0 : half % 8 == 0;
  const bool turns = p.table != nullptr && live && d0 < p.rot;

  Turn w;
  if (turns) {
    const int64_t pos = p.positions[token];
    const bool known = pos >= 0 && pos < p.table_rows;
    const float* row = p.table + (known ? pos : 0) * p.rot;
    const float nan = __builtin_nanf("");
    if (vec && !p.interleaved) {
      const int i0 = d0 < half ? d0 : d0 - half;
      const float sign = (d0 < half) != (p.inverse != 0) ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const f32x4 c = *(const f32x4*)(row + i0 + e);
        const f32x4 s = *(const f32x4*)(row + half + i0 + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w.own[e + j] = known ? c[j] : nan;
          w.other[e + j] = known ? sign * s[j] : nan;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = min(d0 + e, p.rot - 1);
        const int i = p.interleaved ? d / 2 : d < half ? d : d - half;
        const bool low = p.interleaved ? (d & 1) == 0 : d < half;
        const float c = row[i], s = row[half + i];
        w.own[e] = known ? c : nan;
        w.other[e] = known ? (low != (p.inverse != 0) ? -s : s) : nan;
      }
    }
  }

  int64_t slot = 0;
  bool kept = false;
  if (p.hkv > 0) {
    slot = p.slots[token];
    kept = slot >= 0 && slot < (p.cache.pages << p.cache.page_shift);
  }

  for (int h = first; h < last; ++h) {
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const int hk = is_q ? 0 : is_v ? h - p.hq - p.hkv : h - p.hq;
    const uint16_t* src = is_q   ? p.q + token * p.q_token + h * p.q_head
                          : is_v ? p.v + token * p.v_token + hk * p.v_head
                                 : p.k + token * p.k_token + hk * p.k_head;
    u32x4 raw = {0, 0, 0, 0};
    if (live) raw = load16(src + d0);
    const bool turned = turns && !is_v;
    // The partner's load comes before any store of this wave, and every
    // partner of a head is in the same wave: q_out may be q itself.
    f32x8 x = widen8<T>(raw);
    if (turned) {
      f32x8 y = x;
      if (p.interleaved) {
        y = __builtin_shufflevector(x, x, 1, 0, 3, 2, 5, 4, 7, 6);
      } else if (vec) {
        y = widen8<T>(load16(src + (d0 < half ? d0 + half : d0 - half)));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          if (d < p.rot) y[e] = widen1<T>(src[d < half ? d + half : d - half]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float r = fmaf(w.own[e], x[e], w.other[e] * y[e]);
        x[e] = (vec || d0 + e < p.rot) ? r : x[e];
      }
    }
    if (is_q) {
      if (live)
        *(u32x4*)(p.q_out + token * p.out_token + h * p.out_head + d0) =
            turned ? narrow8<T>(x) : raw;
      continue;
    }
    // Row of this head's token inside its page.
    const int64_t page = slot >> p.cache.page_shift;
    const int64_t offset = slot & ((1 << p.cache.page_shift) - 1);
    const int64_t at = ((page * p.cache.heads + hk) << p.cache.page_shift) + offset;
    void* base = is_v ? p.cache.v : p.cache.k;
    if constexpr (FMT == W4A16_KV_SAME) {
      if (live && kept)
        *(u32x4*)((uint16_t*)base + at * p.dim + d0) = turned ? narrow8<T>(x) : raw;
    } else {
      // Magnitudes compare like integers, infinities and NaN above all.
      uint32_t big = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        big = max(big, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
      for (int s = 1; s < LPH; s *= 2) big = max(big, (uint32_t)__shfl_xor((int)big, s, LPH));
      constexpr float kTop = FMT == W4A16_KV_E4M3 ? 448.0f : 127.0f;
      const float amax = __builtin_bit_cast(float, big);
      const bool finite = big < 0x7F800000u;
      const bool some = finite && amax >= 0x1p-100f;
      const float inv = some ? kTop / amax : 0.0f;
      const float scale = finite ? (some ? amax / kTop : 0.0f) : __builtin_nanf("");
      uint32_t code[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = some ? fminf(fmaxf(x[e + j] * inv, -kTop), kTop) : 0.0f;
        if constexpr (FMT == W4A16_KV_E4M3) {
          int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
          code[e / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            code[e / 4] |= ((uint32_t)(int)__builtin_rintf(y[j]) & 0xFFu) << (8 * j);
        }
      }
      if (live && kept)
        *(u32x2*)((uint8_t*)base + at * p.dim + d0) = u32x2{code[0], code[1]};
      if (lane == 0 && kept) (is_v ? p.cache.v_scale : p.cache.k_scale)[at] = scale;
    }
  }
}

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
  const int64_t offset = slot & ((1 << p.cache.page_shift) - 1);
  for (int h = first; h < last; ++h) {
    const bool is_v = h >= p.cache.heads;
    const int hk = is_v ? h - p.cache.heads : h;
    const int64_t at = ((page * p.cache.heads + hk) << p.cache.page_shift) + offset;
    const void* base = is_v ? p.cache.v : p.cache.k;
    u32x4 y = {0, 0, 0, 0};
    if (kept) {
      if constexpr (FMT == W4A16_KV_SAME) {
        y = load16((const uint16_t*)base + at * p.cache.dim + d0);
      } else {
        const u32x2 c = load8((const uint8_t*)base + at * p.cache.dim + d0);
        const float s = (is_v ? p.cache.v_scale : p.cache.k_scale)[at];
        const f32x4 lo = decode4<FMT>(c.x) * s, hi = decode4<FMT>(c.y) * s;
        y = narrow8<T>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
    *(u32x4*)((is_v ? p.v_out : p.k_out) +
              ((int64_t)token * p.cache.heads + hk) * p.cache.dim + d0) = y;
  }
}

template <typename T, int FMT>
hipError_t rope_kv_lanes(const RopeKvParams& p, hipStream_t stream) {
  const int lph = lanes_per_head(p.dim);
  const int64_t units = (int64_t)p.tokens * p.units_per_token;
  const dim3 grid((uint32_t)((units + 256 / lph - 1) / (256 / lph)));
  if (lph == 8)
    hipLaunchKernelGGL((rope_kv_kernel<T, FMT, 8>), grid, dim3(256), 0, stream, p);
  else if (lph == 16)
    hipLaunchKernelGGL((rope_kv_kernel<T, FMT, 16>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((rope_kv_kernel<T, FMT, 32>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <typename T, int FMT>
hipError_t kv_read_lanes(const KvReadParams& p, hipStream_t stream) {
  const int lph = lanes_per_head(p.cache.dim);
  const int64_t units = (int64_t)p.tokens * p.units_per_token;
  const dim3 grid((uint32_t)((units + 256 / lph - 1) / (256 / lph)));
  if (lph == 8)
    hipLaunchKernelGGL((kv_read_kernel<T, FMT, 8>), grid, dim3(256), 0, stream, p);
  else if (lph == 16)
    hipLaunchKernelGGL((kv_read_kernel<T, FMT, 16>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((kv_read_kernel<T, FMT, 32>), grid, dim3(256), 0, stream, p);
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
