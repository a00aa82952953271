// Attention over a paged cache: fp16 activations, e4m3 cache.
#include "tree_attn_kernel.h"

namespace w4a16 {
hipError_t attn_f16_e4m3(const AttnParams& p, AttnKind kind, hipStream_t stream) {
  return serve::launch_attn_shape<serve::F16, W4A16_KV_E4M3>(p, kind, stream);
}
}  // namespace w4a16
