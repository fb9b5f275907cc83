// Latent attention kernels for vectors of 512 values.
#include "attn_latent.h"

namespace moe {
hipError_t launch_latent_512(const AttnArgs& a, int fmt, int grid, hipStream_t s) {
  return run_latent_d<512>(a, fmt, grid, s);
}
}  // namespace moe
