// Single-token attention kernels for head_dim 128.
#include "attn_decode.h"

namespace moe {
hipError_t launch_decode_128(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_decode_d<128>(a, fmt, s);
}
}  // namespace moe
