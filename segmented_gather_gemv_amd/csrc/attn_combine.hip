// Joining the parts of rows whose tokens were split over workgroups: with each part's maximum m_i
// (of scores times log2 e), sum l_i and unnormalised output o_i,
//   m = max m_i,  out = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,  lse = (m + log2 of that sum) ln 2.
// One launch for each kernel that may have split, one wave per row of its tiles; it reads what the
// parts wrote (4 (D + 2) bytes each, still in the caches), and skips rows that were not split.
#include "attn.h"

namespace sgmv {

namespace {

constexpr int JOIN_ROWS = 4;  // of a workgroup

template <bool F32>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs A, int kernel) {
  const KvArgs& K = A.kv;
  const int lane = threadIdx.x & (WAVE - 1);
  const int tile = kernel ? tiled_rows(K.D) : A.direct_tile, per_tile = tile / JOIN_ROWS;
  const int kvh = blockIdx.x % K.H, rest = blockIdx.x / K.H;
  const int slot = rest / per_tile;
  const auto first_slot = [&](int i) { return (int)((int64_t)min(max(K.q_start[i], 0), K.T) * A.G / tile) + i; };
  const bool one = !kernel && A.one_tile;
  const int b = one ? slot : __builtin_amdgcn_readfirstlane(wave_find(K.B, slot, first_slot));
  const int tile0 = one ? 0 : (slot - first_slot(b)) * tile;
  const KvSeq s = kv_seq(K, b);
  const int rows = s.q_len * A.G, row = tile0 + rest % per_tile * JOIN_ROWS + (int)threadIdx.x / WAVE;
  if (tile0 < 0 || row >= rows || (rows > A.direct_rows) != (kernel == 1)) return;
  const int used = span_splits(A, row_span(A, s, tile0, tile), kernel);
  if (used == 1) return;
  const int token = s.q0 + row / A.G, head = kvh * A.G + row % A.G;
  const int64_t at = (int64_t)token * A.Hq + head;

  const int64_t stride = A.part_rows[kernel], part = part_row(A, kernel, slot, kvh, row - tile0, at);
  const float *part_o = A.part_o[kernel], *part_ml = A.part_ml[kernel];
  float m = -INFINITY, l = 0.f;
  if (lane < used) {
    const f32x2_t v = *reinterpret_cast<const f32x2_t*>(part_ml + 2 * (lane * stride + part));
    m = v.x;
    l = v.y;
  }
  float top = m;
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float f = m == -INFINITY ? 1.f : exp2f(m - top);  // l = 0 and o = 0, or NaN
  float sum = l * f;
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  // lanes of a part: those that its D values take four each; several parts side by side
  const int width = K.D <= 64 ? 16 : K.D <= 128 ? 32 : 64;
  const int d = 4 * (lane & (width - 1)), side = lane / width, sides = WAVE / width;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int UNROLL = 8;  // loads in flight
  for (int i0 = 0; i0 < used; i0 += UNROLL * sides) {
    f32x4_t v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * sides + side;
      v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (i < used && d < K.D) v[u] = *reinterpret_cast<const f32x4_t*>(part_o + (i * stride + part) * K.D + d);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const float w = __shfl(f, min(i0 + u * sides + side, WAVE - 1));
      const bool in = i0 + u * sides + side < used;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += in ? w * v[u][j] : 0.f;
    }
  }
  for (int o = width; o < WAVE; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (A.lse && lane == 0)
    A.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
  if (side == 0 && d < K.D)
    store_out<F32>(A, (int64_t)token * A.ldo_t + (int64_t)head * A.ldo_h + d, acc.x * inv, acc.y * inv,
                   acc.z * inv, acc.w * inv);
}

}  // namespace

hipError_t launch_attn_combine(const AttnArgs& A, int kernel, hipStream_t stream) {
  const int tile = kernel ? tiled_rows(A.kv.D) : A.direct_tile;
  const dim3 g((unsigned)A.slots[kernel] * (unsigned)(tile / JOIN_ROWS) * (unsigned)A.kv.H), b(JOIN_ROWS * WAVE);
  if (A.f32) attn_combine_kernel<true><<<g, b, 0, stream>>>(A, kernel);
  else attn_combine_kernel<false><<<g, b, 0, stream>>>(A, kernel);
  return hipGetLastError();
}

}  // namespace sgmv
