// Instances of the few-row base product for bf16 rows and I4 weights with zero points.
#include "base_direct.h"

namespace sgmv {

hipError_t launch_base_direct_i4z(const BaseArgs& A, int s, hipStream_t stream) {
  if (s == 4) return launch_base_rows<false, false, true, 4>(A, stream);
  if (s == 2) return launch_base_rows<false, false, true, 2>(A, stream);
  return launch_base_rows<false, false, true, 1>(A, stream);
}

}  // namespace sgmv
