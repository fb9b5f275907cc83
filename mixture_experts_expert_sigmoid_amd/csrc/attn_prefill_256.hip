// Prompt attention kernels for head_dim 256.
#include "attn_prefill.h"

namespace moe {
hipError_t launch_prefill_256(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_prefill_d<256, kCausal>(a, fmt, s);
}
}  // namespace moe
