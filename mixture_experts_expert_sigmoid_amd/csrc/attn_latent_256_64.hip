// Latent attention for vectors of 256 values, 64 rows a workgroup.
#include "attn_latent.h"

namespace moe {
hipError_t launch_latent_256_64(const AttnArgs& a, int fmt, int grid, hipStream_t s) {
  return run_latent_d<256, 64>(a, fmt, grid, s);
}
}  // namespace moe
