// Instances of the few-row base product for fp32 rows.
#include "base_direct.h"

namespace sgmv {

template <bool ZERO>
static hipError_t launch_i4(const BaseArgs& A, int s, hipStream_t stream) {
  if (s == 4) return launch_base_rows<false, true, ZERO, 4>(A, stream);
  if (s == 2) return launch_base_rows<false, true, ZERO, 2>(A, stream);
  return launch_base_rows<false, true, ZERO, 1>(A, stream);
}

hipError_t launch_base_direct_f32(const BaseArgs& A, int format, int s, hipStream_t stream) {
  if (format == SGMV_BASE_E2M1) return launch_base_rows<true, true, false, 4>(A, stream);
  return A.zero ? launch_i4<true>(A, s, stream) : launch_i4<false>(A, s, stream);
}

}  // namespace sgmv
