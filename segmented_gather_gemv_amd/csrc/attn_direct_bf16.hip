// Instances of the direct attention kernel for bf16 rows and a bf16 cache.
#include "attn_direct.h"

namespace sgmv {

hipError_t launch_attn_direct_bf16(const AttnArgs& A, hipStream_t stream) { return launch_direct_bf16<SGMV_KV_BF16>(A, stream); }

}  // namespace sgmv
