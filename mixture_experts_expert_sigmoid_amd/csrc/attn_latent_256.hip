// Latent attention kernels for vectors of 256 values.
#include "attn_latent.h"

namespace moe {
hipError_t launch_latent_256(const AttnArgs& a, int fmt, int grid, hipStream_t s) {
  return run_latent_d<256>(a, fmt, grid, s);
}
}  // namespace moe
