// Prompt attention kernels for head_dim 128.
#include "attn_prefill.h"

namespace moe {
hipError_t launch_prefill_128(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_prefill_d<128, kCausal>(a, fmt, s);
}
}  // namespace moe
