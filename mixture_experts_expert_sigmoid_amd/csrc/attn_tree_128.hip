// Kernels of the attention of drafted trees for head_dim 128.
#include "attn_prefill.h"

namespace moe {
hipError_t launch_tree_128(const AttnArgs& a, int fmt, hipStream_t s) {
  return run_prefill_d<128, kTree>(a, fmt, s);
}
}  // namespace moe
