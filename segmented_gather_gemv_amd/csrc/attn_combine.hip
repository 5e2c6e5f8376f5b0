// Joining the parts of rows whose tokens were split over workgroups: with each part's maximum m_i
// (of scores times log2 e), sum l_i and unnormalised output o_i,
//   m = max m_i,  out = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,  lse = (m + log2 of that sum) ln 2.
// One wave per (token, query head); it reads what the parts wrote (4 (D + 2) bytes each, still in
// the caches), and skips rows that were not split.
#include "attn.h"

namespace sgmv {

namespace {

template <bool F32>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs A) {
  const KvArgs& K = A.kv;
  const int lane = threadIdx.x & (WAVE - 1);
  const int64_t at = (int64_t)blockIdx.x * (256 / WAVE) + threadIdx.x / WAVE;
  const int token = (int)(at / A.Hq), head = (int)(at % A.Hq);
  if (token >= K.T) return;
  const int b = wave_find(K.B, token, [&](int i) { return min(max(K.q_start[i], 0), K.T); });
  const KvSeq s = kv_seq(K, b);
  const int tok = token - s.q0;
  if (tok < 0 || tok >= s.q_len) return;
  const int rows = s.q_len * A.G, row = tok * A.G + head % A.G;
  const int kernel = rows > A.direct_rows, tile = kernel ? tiled_rows(K.D) : AT_ROWS;
  const Span span = row_span(A, s, row / tile * tile, tile);
  const int used = span_splits(A, span, kernel);
  if (used == 1) return;

  const int64_t stride = (int64_t)K.T * A.Hq;
  float m = -INFINITY, l = 0.f;
  if (lane < used) {
    const f32x2_t v = *reinterpret_cast<const f32x2_t*>(A.part_ml + 2 * (lane * stride + at));
    m = v.x;
    l = v.y;
  }
  float top = m;
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float f = m == -INFINITY ? 0.f : exp2f(m - top);
  float sum = l * f;
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  const int d = 4 * lane;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < used; ++i) {
    const float w = __shfl(f, i);
    if (d < K.D) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(A.part_o + (i * stride + at) * K.D + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += w == 0.f ? 0.f : w * v[j];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (A.lse && lane == 0)
    A.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
  if (d < K.D)
    store_out<F32>(A, (int64_t)token * A.ldo_t + (int64_t)head * A.ldo_h + d, acc.x * inv, acc.y * inv,
                   acc.z * inv, acc.w * inv);
}

}  // namespace

hipError_t launch_attn_combine(const AttnArgs& A, hipStream_t stream) {
  const int64_t n = (int64_t)A.kv.T * A.Hq;
  const dim3 g((unsigned)((n + 3) / 4)), b(256);
  if (A.f32) attn_combine_kernel<true><<<g, b, 0, stream>>>(A);
  else attn_combine_kernel<false><<<g, b, 0, stream>>>(A);
  return hipGetLastError();
}

}  // namespace sgmv
