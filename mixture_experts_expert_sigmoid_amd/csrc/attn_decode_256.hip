// Single-token attention kernels for head_dim 256.
#include "attn_decode.h"

namespace moe {
hipError_t launch_decode_256(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_decode_d<256>(a, fmt, s);
}
}  // namespace moe
