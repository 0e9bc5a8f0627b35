// Adapters of fp16 (see moe_adapters.cuh).
#include "moe_adapters.cuh"

namespace moe {

cudaError_t launch_adapters_f16(const AdapterParams& p, int blocks, cudaStream_t stream) {
  return launch_products<true>(p, blocks, stream);
}

}  // namespace moe
