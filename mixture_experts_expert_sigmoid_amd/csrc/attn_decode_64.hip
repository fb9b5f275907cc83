// Single-token attention kernels for head_dim 64.
#include "attn_decode.h"

namespace moe {
hipError_t launch_decode_64(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_decode_d<64>(a, fmt, s);
}
}  // namespace moe
