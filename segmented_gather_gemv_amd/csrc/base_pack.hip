// Packing a 4-bit base weight (load time): rows of codes into blocks of 16 n and 128 k in the order of the matrix
// cores' operands (base.h), scales and zero points beside them. Bound: eight bytes read one by one for each word
// written, from lines that a wave shares; 8192 x 8192 in 121 us, once.
#include "base.h"

namespace sgmv {

namespace {

// One word of the layout per thread.
__global__ __launch_bounds__(256) void base_pack_codes_kernel(BasePackArgs A) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tiles = (A.N + BASE_N - 1) / BASE_N;
  if (at >= tiles * A.blocks * 256) return;
  const int j = (int)(at & 3), lane = (int)(at >> 2 & 63);
  const int64_t block = at >> 8, tile = block / A.blocks;
  const int n = (int)(tile * BASE_N) + (lane & 15), k = (int)(block - tile * A.blocks) * BASE_K + 32 * j + 8 * (lane >> 4);
  uint32_t w = 0;
  if (n < A.N) {
    const uint8_t* row = A.codes + (int64_t)n * A.ldc;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < A.K) {
        const uint32_t c = row[(k + i) >> 1] >> (4 * ((k + i) & 1)) & 15u;
        w |= c << (A.e2m1 ? 4 * i : 8 * (i & 3) + 4 * (i >> 2));
      }
  }
  static_cast<uint32_t*>(A.codes_out)[at] = w;
}

// One scale (and zero point) of the layout per thread.
__global__ __launch_bounds__(256) void base_pack_scales_kernel(BasePackArgs A) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tiles = (A.N + BASE_N - 1) / BASE_N;
  if (at >= tiles * A.scale_rows * BASE_N * A.s) return;
  const int i = (int)(at % A.s);
  const int64_t rest = at / A.s;
  const int64_t row = rest / BASE_N, tile = row / A.scale_rows;
  const int64_t n = tile * BASE_N + rest % BASE_N, g = (row - tile * A.scale_rows) * A.s + i;
  const bool in = n < A.N && g < A.groups;
  const int64_t from = n * A.groups + g;
  if (A.scale_bytes == 4) static_cast<uint32_t*>(A.scale_out)[at] = in ? static_cast<const uint32_t*>(A.scale)[from] : 0u;
  else if (A.scale_bytes == 2) static_cast<uint16_t*>(A.scale_out)[at] = in ? static_cast<const uint16_t*>(A.scale)[from] : (uint16_t)0;
  else static_cast<uint8_t*>(A.scale_out)[at] = in ? static_cast<const uint8_t*>(A.scale)[from] : (uint8_t)0;
  if (A.zero) A.zero_out[at] = in ? A.zero[from] : (uint8_t)0;
}

}  // namespace

hipError_t launch_base_pack(const BasePackArgs& A, hipStream_t stream) {
  const int64_t tiles = (A.N + BASE_N - 1) / BASE_N;
  const int64_t words = tiles * A.blocks, scales = (tiles * A.scale_rows * BASE_N * A.s + 255) / 256;
  base_pack_codes_kernel<<<(unsigned)words, 256, 0, stream>>>(A);
  base_pack_scales_kernel<<<(unsigned)scales, 256, 0, stream>>>(A);
  return hipGetLastError();
}

}  // namespace sgmv
