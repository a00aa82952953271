// Attention over a paged cache: fp16 activations, 16-bit cache.
#include "tree_attn_kernel.h"

namespace w4a16 {
hipError_t attn_f16_same(const AttnParams& p, AttnKind kind, hipStream_t stream) {
  return serve::launch_attn_shape<serve::F16, W4A16_KV_SAME>(p, kind, stream);
}
}  // namespace w4a16
