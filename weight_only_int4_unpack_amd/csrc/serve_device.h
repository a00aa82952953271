// Device helpers shared by the kernels around the weight products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_internal.h"

namespace w4a16 {
namespace serve {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct F16 {
  using Vec = f16x8;
  static constexpr int kCode = W4A16_F16;
};
struct BF16 {
  using Vec = bf16x8;
  static constexpr int kCode = W4A16_BF16;
};

template <typename T>
__device__ __forceinline__ f32x8 widen8(u32x4 x) {
  return __builtin_convertvector(__builtin_bit_cast(typename T::Vec, x), f32x8);
}
// Round to nearest even.
template <typename T>
__device__ __forceinline__ u32x4 narrow8(f32x8 x) {
  return __builtin_bit_cast(u32x4, __builtin_convertvector(x, typename T::Vec));
}
template <typename T>
__device__ __forceinline__ float widen1(uint16_t h) {
  if constexpr (T::kCode == W4A16_F16)
    return (float)__builtin_bit_cast(_Float16, h);
  else
    return __builtin_bit_cast(float, (uint32_t)h << 16);
}

__device__ __forceinline__ u32x4 load16(const void* p) { return *(const u32x4*)p; }
__device__ __forceinline__ u32x2 load8(const void* p) { return *(const u32x2*)p; }

// Four 8-bit codes of a word as fp32 (exact).
template <int FMT>
__device__ __forceinline__ f32x4 decode4(uint32_t w) {
  if constexpr (FMT == W4A16_KV_E4M3) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return f32x4{lo.x, lo.y, hi.x, hi.y};
  } else {
    return f32x4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16),
                 (float)(int8_t)(w >> 24)};
  }
}

}  // namespace serve
}  // namespace w4a16
