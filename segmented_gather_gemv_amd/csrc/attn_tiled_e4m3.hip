// Instances of the tiled attention kernel for an e4m3 cache.
#include "attn_tiled.h"

namespace sgmv {

hipError_t launch_attn_tiled_e4m3(const AttnArgs& A, hipStream_t stream) { return launch_tiled_dim<SGMV_KV_E4M3>(A, stream); }

}  // namespace sgmv
