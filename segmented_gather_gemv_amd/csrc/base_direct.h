// Product of few rows with a 4-bit base weight: the weight read once, straight into matrix-core operands.
//
// A workgroup takes NT * 16 columns n and 16 TM rows of x; its waves take every WAVES-th block of 128 k, each
// summing all of its tiles in fp32, and their sums are added in LDS in the waves' order. The weight's next block and the
// rows of x that go with it are in flight while one is multiplied.
#pragma once

#include "base.h"

namespace sgmv {

template <bool E2M1, bool F32, bool ZERO, int S, int NT, int TM, int WAVES>
__global__ __launch_bounds__(WAVES* WAVE, TM* NT >= 8 ? 2 : WAVES / 4) void base_direct_kernel(BaseArgs A) {
  constexpr int XW = F32 ? 2 : 1, ROWS = 16 * TM, COLS = 16 * NT, LD = COLS + 4;
  __shared__ float s_sum[WAVES][ROWS * LD];
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int r = lane & 15, quad = lane >> 4;
  const int tiles = (A.N + BASE_N - 1) / BASE_N;
  const int tile0 = blockIdx.x * NT, t0 = blockIdx.y * ROWS;

  // (rows and columns past the last ones are those again, and not stored)
  const char* x[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m)
    x[m] = static_cast<const char*>(A.x) + (int64_t)min(t0 + 16 * m + r, A.T - 1) * A.ldx * (F32 ? 4 : 2);
  int64_t tile[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) tile[n] = min(tile0 + n, tiles - 1);

  struct Block {
    u32x4_t w[NT], x[TM][4][XW];
    BaseScale<E2M1, F32, S> s[NT];
    BaseZero<ZERO, S> z[NT];
  };
  const auto load = [&](int kb, Block& b) {
    const int row = kb / A.per_group;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      b.w[n] = static_cast<const u32x4_t*>(A.codes)[(tile[n] * A.blocks + kb) * WAVE + lane];
      b.s[n] = BaseScale<E2M1, F32, S>::load(A.scale, tile[n] * A.scale_rows + row, r);
      if constexpr (!E2M1) b.z[n] = BaseZero<ZERO, S>::load(A.zero, tile[n] * A.scale_rows + row, r);
    }
    const bool whole = A.x_vec && (kb + 1) * BASE_K <= A.K;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < XW; ++e) {
          const int k = kb * BASE_K + 32 * j + 8 * quad + 4 * e;
          if (whole) {
            b.x[m][j][e] = load_u32x4(x[m] + (int64_t)k * (F32 ? 4 : 2));
          } else {
            u32x4_t v = {0u, 0u, 0u, 0u};
            if constexpr (F32) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k + i < A.K) v[i] = reinterpret_cast<const uint32_t*>(x[m])[k + i];
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (k + i < A.K) v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(x[m])[k + i] << (16 * (i & 1));
            }
            b.x[m][j][e] = v;
          }
        }
  };

  f32x4_t acc[NT][TM];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = f32x4_t{};
  const bf16x8_t ones = as_bf16x8(u32x4_t{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});

  const auto multiply = [&](const Block& b) {
#pragma unroll
    for (int g = 0; g < S; ++g) {
      f32x4_t part[NT][TM], sum[TM];
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        sum[m] = f32x4_t{};
#pragma unroll
        for (int n = 0; n < NT; ++n) part[n][m] = f32x4_t{};
      }
#pragma unroll
      for (int j = g * (4 / S); j < (g + 1) * (4 / S); ++j) {
        bf16x8_t p[TM][F32 ? 3 : 1];
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          if constexpr (F32) split3(b.x[m][j], p[m]);
          else p[m][0] = as_bf16x8(b.x[m][j][0]);
          if constexpr (!E2M1 && !F32) sum[m] = mfma_16x16x32_bf16(p[m][0], ones, sum[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4_t w;
          if constexpr (E2M1) w = base_floats(b.w[n][j], b.s[n].f[g]);
          else if constexpr (F32) w = base_less(base_codes(b.w[n][j]), b.z[n].f[g]);
          else w = base_codes(b.w[n][j]);
#pragma unroll
          for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int k = (F32 ? 3 : 1) - 1; k >= 0; --k) {  // the small parts first
              f32x4_t& to = E2M1 ? acc[n][m] : part[n][m];
              to = mfma_16x16x32_bf16(p[m][k], as_bf16x8(w), to);
            }
        }
      }
      if constexpr (!E2M1)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = F32 ? part[n][m][i] : fmaf(-b.z[n].f[g], sum[m][i], part[n][m][i]);
              acc[n][m][i] = fmaf(b.s[n].f[g], v, acc[n][m][i]);
            }
    }
  };

  int kb = wv;
  if (kb < A.blocks) {
    Block now, next;
    load(kb, now);
    for (; kb < A.blocks; kb += WAVES) {
      const bool more = kb + WAVES < A.blocks;
      if (more) load(kb + WAVES, next);
      multiply(now);
      if (more) now = next;
    }
  }

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_sum[wv][(16 * m + 4 * quad + i) * LD + 16 * n + r] = acc[n][m][i];
  __syncthreads();
  const int rows = min(A.T - t0, ROWS), cols = min(A.N - tile0 * BASE_N, COLS);
  for (int e = threadIdx.x; e < ROWS * COLS; e += WAVES * WAVE) {
    const int t = e / COLS, n = e - t * COLS;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += s_sum[w][t * LD + n];
    if (t >= rows || n >= cols) continue;
    const int64_t at = (int64_t)(t0 + t) * A.ldy + tile0 * BASE_N + n;
    if constexpr (F32) static_cast<float*>(A.y)[at] = v;
    else static_cast<uint16_t*>(A.y)[at] = (uint16_t)pack_bf16x2(v, 0.f);
  }
}

template <bool E2M1, bool F32, bool ZERO, int S, int NT, int TM, int WAVES>
hipError_t launch_base(const BaseArgs& A, hipStream_t stream) {
  const int tiles = (A.N + BASE_N - 1) / BASE_N;
  const dim3 g((unsigned)((tiles + NT - 1) / NT), (unsigned)((A.T + 16 * TM - 1) / (16 * TM)));
  base_direct_kernel<E2M1, F32, ZERO, S, NT, TM, WAVES><<<g, WAVES * WAVE, 0, stream>>>(A);
  return hipGetLastError();
}

template <bool E2M1, bool F32, bool ZERO, int S>
hipError_t launch_base_rows(const BaseArgs& A, hipStream_t stream) {
  if constexpr (F32) return launch_base<E2M1, F32, ZERO, S, 1, 1, 8>(A, stream);
  else {
    if (A.T <= 16) return launch_base<E2M1, F32, ZERO, S, 1, 1, 8>(A, stream);
    return launch_base<E2M1, F32, ZERO, S, 2, 2, 8>(A, stream);
  }
}

}  // namespace sgmv
