// Instances of the tiled attention kernel for a e4m3 cache.
#include "attn_tiled.h"

namespace sgmv {

hipError_t launch_attn_tiled_e4m3(const AttnArgs& A, unsigned slots, hipStream_t stream) {
  const dim3 g(slots * (unsigned)A.n_split[1] * (unsigned)A.kv.H);
  constexpr int F = SGMV_KV_E4M3;
  switch (A.kv.D) {
    case 64: attn_tiled_kernel<F, 64><<<g, tiled_waves(64) * WAVE, 0, stream>>>(A); break;
    case 96: attn_tiled_kernel<F, 96><<<g, tiled_waves(96) * WAVE, 0, stream>>>(A); break;
    case 128: attn_tiled_kernel<F, 128><<<g, tiled_waves(128) * WAVE, 0, stream>>>(A); break;
    case 192: attn_tiled_kernel<F, 192><<<g, tiled_waves(192) * WAVE, 0, stream>>>(A); break;
    case 256: attn_tiled_kernel<F, 256><<<g, tiled_waves(256) * WAVE, 0, stream>>>(A); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace sgmv
