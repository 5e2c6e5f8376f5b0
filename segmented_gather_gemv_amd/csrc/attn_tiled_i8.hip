// Instances of the tiled attention kernel for an i8 cache.
#include "attn_tiled.h"

namespace sgmv {

hipError_t launch_attn_tiled_i8(const AttnArgs& A, hipStream_t stream) { return launch_tiled_dim<SGMV_KV_I8>(A, stream); }

}  // namespace sgmv
