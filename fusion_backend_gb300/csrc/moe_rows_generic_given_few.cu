// Row kernel instances for a routing that the caller brings, H <= 2048, at most
// four tokens (see moe_rows_generic_given.cu).
#include "moe_rows.cuh"

namespace moe {

cudaError_t launch_rows_generic_given_few(const LayerParams& p, cudaStream_t stream) {
  if (p.T == 1) {
    switch (p.wfmt) {
      case kWkQ4: return launch_rows_t<1, kWkQ4, false, 1, true>(p, stream);
      case kWkI8: return launch_rows_t<1, kWkI8, false, 1, true>(p, stream);
      default: return launch_rows_t<1, kWkBf16, false, 1, true>(p, stream);
    }
  }
  switch (p.wfmt) {
    case kWkQ4: return launch_rows_t<4, kWkQ4, false, 1, true>(p, stream);
    case kWkI8: return launch_rows_t<4, kWkI8, false, 1, true>(p, stream);
    default: return launch_rows_t<4, kWkBf16, false, 1, true>(p, stream);
  }
}

}  // namespace moe
