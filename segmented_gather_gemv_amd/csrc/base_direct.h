// Product of few rows with a 4-bit base weight: the weight read once, straight into matrix-core operands.
//
// A workgroup takes NT * 16 columns n and 16 TM rows of x; its waves take every WAVES-th block of 128 k, each
// summing all of its tiles in fp32, and their sums are added in LDS in the waves' order. Up to 4 rows go straight into
// operands (16 rows of the product's, the last of them again), and so do fp32 rows, whose parts are made in registers: a
// wave asks for its next block behind the products of one, and other waves' blocks are in flight meanwhile. More rows of
// bf16 are read as whole lines and pass through the wave's part of LDS (16 rows over 8192 x 8192: 12 us without); there
// the next block is in flight while one is multiplied. A wave's block is NT KB of the weight, so that 16 waves of one or
// two tiles have up to 16 or 32 KB of it in flight and 8 waves of four 32 KB; a unit holds two workgroups of unstaged bf16
// rows without zero points, and twice that.
//
// Bound: the weight's bytes, from some 16 rows on the conversions and products. Measured (I4, groups of 128, bf16 rows;
// floors by a large copy's 5.14 TB/s): one row over 8192 x 8192 8.0 us (35 MB, 4.3 TB/s; floor 6.8), over 28672 x 8192
// 26 (23.6); 16 rows 10.0 (6.8), 64 rows 18 (7.2); E2M1, 16 rows over 28672 x 8192 29 (24.7); fp32, one row over 8192 x
// 8192 12.8 (6.9), 64 over 4096 x 4096 12.9. 128 over 8192 x 8192 30 to 34 (14.4), 256 over 4096 x 4096 18 (7.2): each
// 16 or 32 rows convert the whole weight again.
#pragma once

#include "base.h"

namespace sgmv {

// Waves per SIMD to allocate registers for: one workgroup per compute unit, two where the registers of rows and zero
// points leave room or it has four waves (three of those a unit: 36 to 93 spilled registers, 10 to 200% slower). Of the
// instances below one spills: fp32, groups of 32 without zero points, one tile of columns, 2 registers.
constexpr int base_occupancy(bool zero, bool f32, int waves, bool staged) {
  if (!f32 && !staged && !zero) return 8;
  return waves >= 8 ? waves / 4 : 2;
}

template <bool E2M1, bool F32, bool ZERO, int S, int NT, int TM, int WAVES, bool STAGED>
__global__ __launch_bounds__(WAVES* WAVE, base_occupancy(ZERO, F32, WAVES, STAGED)) void base_direct_kernel(BaseArgs A) {
  constexpr int XW = F32 ? 2 : 1, ROWS = 16 * TM, COLS = 16 * NT, LD = COLS + 4;
  static_assert(!(STAGED && F32), "rows of bf16 are staged");
  constexpr int X_BYTES = STAGED ? ROWS * BASE_K * 2 : 0, SUM_BYTES = ROWS * LD * 4;
  __shared__ alignas(16) char s_all[WAVES * (X_BYTES > SUM_BYTES ? X_BYTES : SUM_BYTES)];
  float* const s_sum = reinterpret_cast<float*>(s_all);
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int r = lane & 15, quad = lane >> 4;
  const int tiles = (A.N + BASE_N - 1) / BASE_N, across = (tiles + NT - 1) / NT;
  const int down = blockIdx.x / across, tile0 = ((int)blockIdx.x - down * across) * NT, t0 = down * ROWS;

  // (rows and columns past the last ones are those again, and not stored)
  constexpr int E = F32 ? 4 : 2;
  int64_t tile[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) tile[n] = min(tile0 + n, tiles - 1);

  // 16 bytes of x [m][j][e] of a block: as operands row 16 m + r, k = 32 j + 8 quad + 4 e; staged, whole lines of row
  // 16 m + 4 j + quad, k = 8 r.
  const char* x[TM][STAGED ? 4 : 1];
  const auto k_of = [&](int j, int e) { return STAGED ? 8 * r : 32 * j + 8 * quad + 4 * e; };
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int j = 0; j < (STAGED ? 4 : 1); ++j)
      x[m][j] = static_cast<const char*>(A.x) + (int64_t)min(t0 + 16 * m + (STAGED ? 4 * j + quad : r), A.T - 1) * A.ldx * E;

  struct Weights {
    u32x4_t w[NT];
    BaseScale<E2M1, F32, S> s[NT];
    BaseZero<ZERO, S> z[NT];
  };
  struct Rows {
    u32x4_t x[TM][4][XW];
  };
  const auto load_weights = [&](int kb, Weights& b) {
    const int row = kb / A.per_group;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      b.w[n] = static_cast<const u32x4_t*>(A.codes)[(tile[n] * A.blocks + kb) * WAVE + lane];
      b.s[n] = BaseScale<E2M1, F32, S>::load(A.scale, tile[n] * A.scale_rows + row, r);
      if constexpr (!E2M1) b.z[n] = BaseZero<ZERO, S>::load(A.zero, tile[n] * A.scale_rows + row, r);
    }
  };
  const auto load_rows = [&](int kb, Rows& b) {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < XW; ++e) b.x[m][j][e] = load_row<F32>(x[m][STAGED ? j : 0] + ((int64_t)kb * BASE_K + k_of(j, e)) * E);
  };
  // Staged rows go to the wave's own part of LDS and come back as operands: pieces of 16 bytes, exchanged within a row so
  // that 16 rows' pieces of the same k lie in different banks.
  char* const own = s_all + wv * X_BYTES;
  const auto stage = [&](const Rows& b) {
    wave_lds_order();  // behind the reads of the block before
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 4 * j + quad;
        *reinterpret_cast<u32x4_t*>(own + (16 * m + row) * 256 + (r ^ row) * 16) = b.x[m][j][0];
      }
    wave_lds_order();  // other lanes read them
  };

  f32x4_t acc[NT][TM];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = f32x4_t{};
  const bf16x8_t ones = as_bf16x8(u32x4_t{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});

  const auto multiply = [&](const Weights& b, const Rows& rows) {
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
          if constexpr (F32) split3(rows.x[m][j], p[m]);
          else if constexpr (STAGED) p[m][0] = as_bf16x8(load_u32x4(own + (16 * m + r) * 256 + ((4 * j + quad) ^ r) * 16));
          else p[m][0] = as_bf16x8(rows.x[m][j][0]);
          if constexpr (!E2M1)
#pragma unroll
            for (int k = (F32 ? 3 : 1) - 1; k >= 0; --k) sum[m] = mfma_16x16x32_bf16(p[m][k], ones, sum[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4_t w;
          if constexpr (E2M1) w = base_floats(b.w[n][j], b.s[n].get(g));
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
              const float v = fmaf(-b.z[n].get(g), sum[m][i], part[n][m][i]);
              acc[n][m][i] = fmaf(b.s[n].get(g), v, acc[n][m][i]);
            }
    }
  };

  // Whole blocks; of staged ones the next is in flight while one is multiplied, else other waves' are. (No load depends
  // on whether it is the last: the compiler would move it behind the products that wait for it.)
  const int whole = A.K / BASE_K;
  Weights w;
  Rows rows;
  if (wv < whole) {
    load_weights(wv, w);
    load_rows(wv, rows);
    for (int kb = wv + WAVES; kb < whole; kb += WAVES) {
      if constexpr (STAGED) {
        const Weights now = w;
        stage(rows);
        load_weights(kb, w);
        load_rows(kb, rows);
        multiply(now, rows);
      } else {
        multiply(w, rows);
        load_weights(kb, w);
        load_rows(kb, rows);
      }
    }
    if constexpr (STAGED) stage(rows);
    multiply(w, rows);
  }
  if (whole < A.blocks && wv == whole % WAVES) {  // and what is left of K
    load_weights(whole, w);
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < XW; ++e) {
          const int k = whole * BASE_K + k_of(j, e);
          const char* at = x[m][STAGED ? j : 0] + (int64_t)k * E;
          if (A.K - k >= (F32 ? 4 : 8)) rows.x[m][j][e] = load_row<F32>(at);
          else rows.x[m][j][e] = load_rest<F32>(at, A.K - k);
        }
    if constexpr (STAGED) stage(rows);
    multiply(w, rows);
  }
  if constexpr (STAGED) __syncthreads();  // before the sums take the rows' place

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_sum[wv * (ROWS * LD) + (16 * m + 4 * quad + i) * LD + 16 * n + r] = acc[n][m][i];
  __syncthreads();
  const int n_rows = min(A.T - t0, ROWS), n_cols = min(A.N - tile0 * BASE_N, COLS);
  for (int e = threadIdx.x; e < ROWS * COLS; e += WAVES * WAVE) {
    const int t = e / COLS, n = e - t * COLS;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += s_sum[w * (ROWS * LD) + t * LD + n];
    if (t >= n_rows || n >= n_cols) continue;
    const int64_t at = (int64_t)(t0 + t) * A.ldy + tile0 * BASE_N + n;
    if constexpr (F32) static_cast<float*>(A.y)[at] = v;
    else static_cast<uint16_t*>(A.y)[at] = (uint16_t)pack_bf16x2(v, 0.f);
  }
}

template <bool E2M1, bool F32, bool ZERO, int S, int NT, int TM, int WAVES, bool STAGED>
hipError_t launch_base(const BaseArgs& A, hipStream_t stream) {
  const int tiles = (A.N + BASE_N - 1) / BASE_N;
  const unsigned g = (unsigned)((tiles + NT - 1) / NT) * (unsigned)((A.T + 16 * TM - 1) / (16 * TM));
  base_direct_kernel<E2M1, F32, ZERO, S, NT, TM, WAVES, STAGED><<<g, WAVES * WAVE, 0, stream>>>(A);
  return hipGetLastError();
}

// The instance of a call: the more columns and rows a workgroup takes, the less often rows of x are read and codes
// converted; but each compute unit wants a workgroup of its own, the weight's bytes having to be in flight. So the
// smallest whose workgroups run at once, one on each of 256 units, or the largest.
template <bool E2M1, bool F32, bool ZERO, int S>
hipError_t launch_base_rows(const BaseArgs& A, hipStream_t stream) {
  const int64_t tiles = (A.N + BASE_N - 1) / BASE_N;
  const auto at_once = [&](int nt, int tm) {  // (and of narrow weights no more columns than they have)
    return tiles <= nt || (tiles + nt - 1) / nt * ((A.T + 16 * tm - 1) / (16 * tm)) <= 256;
  };
  if constexpr (F32) {
    if (at_once(1, 1)) return launch_base<E2M1, F32, ZERO, S, 1, 1, 16, false>(A, stream);
    if (at_once(2, 1)) return launch_base<E2M1, F32, ZERO, S, 2, 1, 16, false>(A, stream);
    return launch_base<E2M1, F32, ZERO, S, 4, 1, 8, false>(A, stream);
  } else if (A.T <= 4) {
    if (tiles >= 512) return launch_base<E2M1, F32, ZERO, S, 2, 1, 16, false>(A, stream);
    return launch_base<E2M1, F32, ZERO, S, 1, 1, 16, false>(A, stream);
  } else {
    if (at_once(1, 1)) return launch_base<E2M1, F32, ZERO, S, 1, 1, 16, true>(A, stream);
    if (at_once(2, 1)) return launch_base<E2M1, F32, ZERO, S, 2, 1, 16, true>(A, stream);
    if (A.T <= 16) return launch_base<E2M1, F32, ZERO, S, 4, 1, 8, true>(A, stream);
    if (at_once(2, 2)) return launch_base<E2M1, F32, ZERO, S, 2, 2, 8, true>(A, stream);
    if (at_once(4, 2)) return launch_base<E2M1, F32, ZERO, S, 4, 2, 8, true>(A, stream);
    return launch_base<E2M1, F32, ZERO, S, 4, 2, 4, true>(A, stream);
  }
}

}  // namespace sgmv
