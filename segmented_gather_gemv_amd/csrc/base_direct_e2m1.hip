// Instances of the few-row base product for bf16 rows and E2M1 weights.
#include "base_direct.h"

namespace sgmv {

hipError_t launch_base_direct_e2m1(const BaseArgs& A, hipStream_t stream) { return launch_base_rows<true, false, false, 4>(A, stream); }

}  // namespace sgmv
