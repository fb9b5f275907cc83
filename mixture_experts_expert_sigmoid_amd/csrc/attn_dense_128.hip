// Kernels of the attention of prompts over dense rows of keys and values.
#include "attn_prefill.h"

namespace moe {
hipError_t launch_dense_128(const AttnArgs& a, int fmt, hipStream_t s) {
  return fmt == KV_BF16 ? run_prefill<true, false, kDenseDim, kDense>(a, s)
                        : run_prefill<false, false, kDenseDim, kDense>(a, s);
}
}  // namespace moe
