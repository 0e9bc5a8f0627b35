// Row kernel instances for a routing that the caller brings, the other decode
// shapes (see moe_rows_generic.cu).  Calls of one token and of up to four have
// instances of their own: the code of the eight-token instance does not fit the
// instruction caches, which a call of a few small experts pays for (T = 1,
// H = 1024, 4-bit: 45 us with it).
#include "moe_rows.cuh"

namespace moe {

cudaError_t launch_rows_generic_given_few(const LayerParams& p, cudaStream_t stream);

cudaError_t launch_rows_generic_given(const LayerParams& p, cudaStream_t stream) {
  if (p.H <= 2048) {
    if (p.T <= 4) return launch_rows_generic_given_few(p, stream);
    switch (p.wfmt) {
      case kWkQ4: return launch_rows_t<8, kWkQ4, false, 1, true>(p, stream);
      case kWkI8: return launch_rows_t<8, kWkI8, false, 1, true>(p, stream);
      default: return launch_rows_t<8, kWkBf16, false, 1, true>(p, stream);
    }
  }
  switch (p.wfmt) {
    case kWkQ4: return launch_rows_t<8, kWkQ4, false, 2, true>(p, stream);
    case kWkI8: return launch_rows_t<8, kWkI8, false, 2, true>(p, stream);
    default: return launch_rows_t<8, kWkBf16, false, 2, true>(p, stream);
  }
}

}  // namespace moe
