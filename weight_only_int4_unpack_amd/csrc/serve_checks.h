// Argument checks that the host sides of the operators around the weight products share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_internal.h"

namespace w4a16 {
namespace checks {

constexpr int64_t kMaxInt = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// Workgroups have 256 threads unless a kernel says otherwise, and a grid holds fewer than 2^32 threads.
constexpr int kServeThreads = 256;
constexpr int64_t kMaxGrid = ((int64_t)1 << 32) / kServeThreads - 1;
// CUs of a device that is not partitioned. Sizes are checked for it before there is a
// device to ask; scratch, once there is one, for that device's own.
constexpr int kWholeDevice = 256;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline w4a16_status launched(hipError_t e) {
  if (e == hipSuccess) return W4A16_OK;
  return report(W4A16_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

inline w4a16_status check_dtype(int32_t dtype) {
  if (dtype == W4A16_F16 || dtype == W4A16_BF16) return W4A16_OK;
  return report(W4A16_ERR_DTYPE, "dtype %d: only fp16 (0) and bf16 (1) are supported", (int)dtype);
}

inline w4a16_status check_dim(int32_t dim) {
  if (dim >= 8 && dim <= 256 && dim % 8 == 0) return W4A16_OK;
  return report(W4A16_ERR_SHAPE, "head_dim=%d must be a multiple of 8 in 8..256", (int)dim);
}

inline w4a16_status check_cache(const w4a16_kv_cache_t& c, KvView* view) {
  if (c.format != W4A16_KV_SAME && c.format != W4A16_KV_E4M3 && c.format != W4A16_KV_INT8)
    return report(W4A16_ERR_DTYPE, "cache format %d: 0 (same), 1 (e4m3) and 2 (int8) are supported",
                  (int)c.format);
  w4a16_status st = check_dim(c.head_dim);
  if (st != W4A16_OK) return st;
  // a lane of the attention kernels holds 16 dims of an 8-bit head, or of one above 128
  if (c.head_dim % 16 != 0 && (c.format != W4A16_KV_SAME || c.head_dim > 128))
    return report(W4A16_ERR_SHAPE,
                  "head_dim=%d must be a multiple of 16 above 128 and in a quantised cache",
                  (int)c.head_dim);
  int shift = 0;
  while ((1 << shift) < c.page_size && shift < 12) ++shift;
  if (c.page_size < 16 || c.page_size != (1 << shift))
    return report(W4A16_ERR_SHAPE, "page_size=%d must be a power of two in 16..4096",
                  (int)c.page_size);
  if (c.heads < 1 || c.heads > 4096 || c.pages < 0 || c.pages >= kMaxInt)
    return report(W4A16_ERR_SHAPE, "need 1..4096 cache heads and 0..2^31 pages (got %d, %lld)",
                  (int)c.heads, (long long)c.pages);
  if (c.pages > 0) {
    if (!c.k || !c.v) return report(W4A16_ERR_NULL, "the cache's k and v must be non-NULL");
    if (!aligned(c.k, 16) || !aligned(c.v, 16))
      return report(W4A16_ERR_ALIGN, "the cache's k and v must be 16-byte aligned");
    if (c.format != W4A16_KV_SAME) {
      if (!c.k_scale || !c.v_scale)
        return report(W4A16_ERR_NULL, "a quantised cache needs k_scale and v_scale");
      if (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))
        return report(W4A16_ERR_ALIGN, "the cache's scales must be 16-byte aligned");
    }
  }
  if (view)
    *view = KvView{c.k, c.v, c.k_scale, c.v_scale, c.pages, shift, c.heads, c.head_dim};
  return W4A16_OK;
}

inline w4a16_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return W4A16_OK;
  if (have < need)
    return report(W4A16_ERR_WORKSPACE, "the launch needs %lld bytes of workspace, %lld given",
                  (long long)need, (long long)have);
  if (!ws) return report(W4A16_ERR_NULL, "the launch needs a workspace and none was given");
  if (!aligned(ws, 16)) return report(W4A16_ERR_ALIGN, "workspace must be 16-byte aligned");
  return W4A16_OK;
}

}  // namespace checks
}  // namespace w4a16

#define CHECK(call)                       \
  do {                                    \
    const w4a16_status st_ = (call);      \
    if (st_ != W4A16_OK) return st_;      \
  } while (0)
