// Instances of the direct attention kernel for fp32 rows.
#include "attn_direct.h"

namespace sgmv {

// fp32 operands take twice the registers of bf16 ones: head dimensions past 128 get one tile of rows.
template <int FMT, int R>
static hipError_t launch_dim(const AttnArgs& A, hipStream_t stream) {
  const int D = A.kv.D;
  if (D == 64) return launch_direct<true, FMT, 64, true, R, 4>(A, stream);
  if (D < 64) return launch_direct<true, FMT, 64, false, R, 4>(A, stream);
  if (D == 80) return launch_direct<true, FMT, 80, true, R, 4>(A, stream);
  if (D == 128) return launch_direct<true, FMT, 128, true, R, 4>(A, stream);
  if (D < 128) return launch_direct<true, FMT, 128, false, R, 4>(A, stream);
  if constexpr (R == 1) {
    if (D == 192) return launch_direct<true, FMT, 192, true, 1, 4>(A, stream);
    if (D == 256) return launch_direct<true, FMT, 256, true, 1, 4>(A, stream);
    return launch_direct<true, FMT, 256, false, 1, 4>(A, stream);
  }
  return hipErrorInvalidValue;
}

template <int FMT>
static hipError_t launch_fmt(const AttnArgs& A, hipStream_t stream) {
  return A.direct_tile == 16 ? launch_dim<FMT, 1>(A, stream) : launch_dim<FMT, 2>(A, stream);
}

hipError_t launch_attn_direct_f32(const AttnArgs& A, int fmt, hipStream_t stream) {
  if (fmt == SGMV_KV_E4M3) return launch_fmt<SGMV_KV_E4M3>(A, stream);
  if (fmt == SGMV_KV_I8) return launch_fmt<SGMV_KV_I8>(A, stream);
  return launch_fmt<SGMV_KV_F32>(A, stream);
}

}  // namespace sgmv
