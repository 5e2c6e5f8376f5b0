// Instances of the direct attention kernel for bf16 rows.
#include "attn_direct.h"

namespace sgmv {

template <int FMT>
static void launch_fmt(const AttnArgs& A, dim3 g, hipStream_t stream) {
  const dim3 b(256);
  const int D = A.kv.D;
  if (D == 64) attn_direct_kernel<false, FMT, 64, true><<<g, b, 0, stream>>>(A);
  else if (D < 64) attn_direct_kernel<false, FMT, 64, false><<<g, b, 0, stream>>>(A);
  else if (D == 128) attn_direct_kernel<false, FMT, 128, true><<<g, b, 0, stream>>>(A);
  else if (D < 128) attn_direct_kernel<false, FMT, 128, false><<<g, b, 0, stream>>>(A);
  else if (D == 256) attn_direct_kernel<false, FMT, 256, true><<<g, b, 0, stream>>>(A);
  else attn_direct_kernel<false, FMT, 256, false><<<g, b, 0, stream>>>(A);
}

hipError_t launch_attn_direct_bf16(const AttnArgs& A, int fmt, unsigned slots, hipStream_t stream) {
  const dim3 g(slots * (unsigned)A.n_split[0] * (unsigned)A.kv.H);
  if (fmt == SGMV_KV_E4M3) launch_fmt<SGMV_KV_E4M3>(A, g, stream);
  else if (fmt == SGMV_KV_I8) launch_fmt<SGMV_KV_I8>(A, g, stream);
  else launch_fmt<SGMV_KV_BF16>(A, g, stream);
  return hipGetLastError();
}

}  // namespace sgmv
