// Instances of the tiled attention kernel for a bf16 cache.
#include "attn_tiled.h"

namespace sgmv {

hipError_t launch_attn_tiled_bf16(const AttnArgs& A, hipStream_t stream) { return launch_tiled_dim<SGMV_KV_BF16>(A, stream); }

}  // namespace sgmv
