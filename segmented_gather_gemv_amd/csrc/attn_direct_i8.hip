// Instances of the direct attention kernel for bf16 rows and an i8 cache.
#include "attn_direct.h"

namespace sgmv {

hipError_t launch_attn_direct_i8(const AttnArgs& A, hipStream_t stream) { return launch_direct_bf16<SGMV_KV_I8>(A, stream); }

}  // namespace sgmv
