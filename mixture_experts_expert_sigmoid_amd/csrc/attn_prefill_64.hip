// Prompt attention kernels for head_dim 64.
#include "attn_prefill.h"

namespace moe {
hipError_t launch_prefill_64(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_prefill_d<64, kCausal>(a, fmt, s);
}
}  // namespace moe
