// Instances of the direct attention kernel for bf16 rows and an e4m3 cache.
#include "attn_direct.h"

namespace sgmv {

hipError_t launch_attn_direct_e4m3(const AttnArgs& A, hipStream_t stream) { return launch_direct_bf16<SGMV_KV_E4M3>(A, stream); }

}  // namespace sgmv
