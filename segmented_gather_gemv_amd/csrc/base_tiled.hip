// Product of many rows with a 4-bit base weight: rows of x staged in LDS and shared by the workgroup's waves, codes
// converted in registers.
//
// A workgroup takes 64 rows and 256 columns, each of its four waves 64 of these, over all of K in blocks of 128: per block a
// wave loads 4 KB of the weight straight into operands (base.h) and multiplies them by the 16 operands of x that the
// workgroup has in LDS; rows of the next block are written to the other buffer meanwhile and those after it are on
// their way, so that one barrier a block is enough. LDS holds rows of 256 bytes whose 16-byte pieces are exchanged
// within a row, so that 16 rows' pieces of the same k lie in different banks.
//   I4    a group's sum is kept apart and scaled at its end: part = c x - z sum x, y += s part; sum x over the groups
//         comes from a first launch (of each wave by products with ones, it would be a fifth of all products).
//   E2M1  sums go straight on.
//   fp32  rows are three bf16 parts, small ones first, each a block of its own over the same codes: three times the
//         products, and the same kernel.
// Where that leaves compute units without a tile, K is split into ranges whose sums a last launch adds up.
//
// Bound: the matrix cores and the conversions beside them: per block a wave converts 128 words and scales 64 sums while it
// makes 64 products, which 2 waves a SIMD overlap in part (2048 rows over 11008 x 4096 with zero points: matrix cores
// busy 38% of the cycles, vector units 51%, at 2.06 GHz). Measured, bf16 rows: that 214 us (865 TFLOP/s; the
// library's bf16 product alone runs at 1197), 9 of them preparing rows; without zero points 196, groups of 64 217, groups
// of 32 with zero points 307, E2M1 166 (1115 TFLOP/s); 1000 rows over 8192 x 28672 460 us (1020). fp32 rows: 2048 over 8192 x
// 8192 with zero points 833 us, E2M1 639 (a library product of fp32: 1785). The instances of short groups with zero points
// spill: fp32 rows 11 registers (groups of 32) and 14 (64), bf16 rows 3 (64). Not kept: 128 rows a workgroup (one wave a
// SIMD: 329 us), 192 columns (224), loads straight to LDS (the compiler waits for all loads before each LDS read).
#include "base.h"

namespace sgmv {

namespace {

constexpr int TT = TILE_T / 16;  // tiles of rows
constexpr int TW = 4;            // waves
constexpr int TN = TILE_N / 16 / TW;  // tiles of columns of a wave

// Bytes of a block of rows, and of the sums over its groups behind them.
constexpr int block_bytes(int sums) { return TILE_T * (BASE_K * 2 + sums * 4); }

// Rows of x as the tiles stage them: blocks of 64 rows and 128 k, 256 bytes a row whose pieces of 16 are exchanged
// within it, zeros past the last row and the last k; and behind them the sums over each 128 / S values of the rows. A block
// per workgroup, 16 rows of it per wave, their loads in flight together.
template <bool F32, bool SUMS, int S>
__global__ __launch_bounds__(256) void base_rows_kernel(BaseArgs A) {
  constexpr int BLOCK_BYTES = block_bytes(SUMS ? S : 0), PARTS = F32 ? 3 : 1, E = F32 ? 4 : 2;
  const int lane = threadIdx.x & (WAVE - 1), r = lane & 15;
  const int band = (int)blockIdx.x / A.blocks, kb = (int)blockIdx.x - band * A.blocks, k = kb * BASE_K + 8 * r;
  u32x4_t v[4][E / 2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = (int64_t)band * TILE_T + threadIdx.x / WAVE * 16 + 4 * q + lane / 16;
    const int left = row < A.T ? A.K - k : 0;
    const char* p = static_cast<const char*>(A.x) + (row * A.ldx + k) * E;
#pragma unroll
    for (int h = 0; h < E / 2; ++h) {
      const int n = left - 4 * h;  // (of fp32 4 values a piece)
      v[q][h] = u32x4_t{0u, 0u, 0u, 0u};
      if (n >= (F32 ? 4 : 8)) v[q][h] = load_row<F32>(p + 16 * h);
      else if (n > 0) v[q][h] = load_rest<F32>(p + 16 * h, n);
    }
  }
  char* to = A.rows + (int64_t)blockIdx.x * PARTS * BLOCK_BYTES;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = threadIdx.x / WAVE * 16 + 4 * q + lane / 16;
    bf16x8_t part[PARTS];
    if constexpr (F32) split3(v[q], part);
    else part[0] = as_bf16x8(v[q][0]);
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      *reinterpret_cast<u32x4_t*>(to + i * BLOCK_BYTES + t * 256 + (r ^ (t & 15)) * 16) = __builtin_bit_cast(u32x4_t, part[PARTS - 1 - i]);
    if constexpr (SUMS) {  // with the last part
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float value = 0.f;  // (of its parts: what they lack of one below 2^-110 is missing here too)
#pragma unroll
        for (int k = PARTS - 1; k >= 0; --k) {
          const uint32_t w = __builtin_bit_cast(u32x4_t, part[k])[i / 2];
          value += __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
        }
        sum += value;
      }
#pragma unroll
      for (int o = 1; o < 16 / S; o <<= 1) sum += __shfl_xor(sum, o);
      if (r % (16 / S) == 0)
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
          *reinterpret_cast<float*>(to + i * BLOCK_BYTES + TILE_T * BASE_K * 2 + ((r / (16 / S)) * TILE_T + t) * 4) = i == PARTS - 1 ? sum : 0.f;
    }
  }
}

// The place of a workgroup's tile: each XCD takes a run of them, in squares of 8 by 8 that share rows and columns in its
// L2. False: none.
struct TilePlace {
  int at, t0, n0;
};

__device__ __forceinline__ bool tile_place(const BaseArgs& A, int block, TilePlace& p) {
  const int nt = (A.T + TILE_T - 1) / TILE_T, nn = (A.N + TILE_N - 1) / TILE_N;
  const int per = (nt * nn + 7) / 8;
  p.at = (block & 7) * per + (block >> 3);
  if ((block >> 3) >= per || p.at >= nt * nn) return false;
  const int band = p.at / (8 * nn), in = p.at - band * 8 * nn, wide = min(8, nt - 8 * band);
  p.t0 = (8 * band + in % wide) * TILE_T;
  p.n0 = in / wide * TILE_N;
  return true;
}

// 16 rows and 64 columns of a wave's results as rows of y: fp32 straight from its registers (64 bytes a row at once),
// bf16 through its 2 KB of LDS (16-byte pieces exchanged within the rows of 128, as above).
template <bool F32>
__device__ __forceinline__ void store_tile(const BaseArgs& A, char* own, int t0, int n0, const f32x4_t (&acc)[TN]) {
  const int lane = threadIdx.x & (WAVE - 1), r = lane & 15, quad = lane >> 4;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 4 * quad + i;
      float* y = static_cast<float*>(A.y) + (int64_t)t * A.ldy + n0 + r;
#pragma unroll
      for (int n = 0; n < TN; ++n)
        if (t < A.T && n0 + 16 * n + r < A.N) y[16 * n] = acc[n][i];
    }
    return;
  }
  wave_lds_order();
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * quad + i, c = 2 * n + (r >> 3);
      *reinterpret_cast<uint16_t*>(own + t * 128 + (c ^ (t & 7)) * 16 + (r & 7) * 2) = (uint16_t)pack_bf16x2(acc[n][i], 0.f);
    }
  wave_lds_order();
  constexpr int PIECES = 2 * TN;  // of a row
#pragma unroll
  for (int i = 0; i < (16 * PIECES + WAVE - 1) / WAVE; ++i) {
    const int e = i * WAVE + lane, t = e / PIECES, c = e - t * PIECES, left = A.N - n0 - 8 * c;
    if (t >= 16 || t0 + t >= A.T || left <= 0) continue;
    const u32x4_t v = load_u32x4(own + t * 128 + (c ^ (t & 7)) * 16);
    uint16_t* y = static_cast<uint16_t*>(A.y) + (int64_t)(t0 + t) * A.ldy + n0 + 8 * c;
    if (A.y_vec && left >= 8) {
      *reinterpret_cast<u32x4_t*>(y) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) y[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Place of a wave's 16 rows m in the parts of split `split`: TN registers of 4, lane by lane.
__device__ __forceinline__ float* part_of(const BaseArgs& A, int tiles, int split, int at, int wv, int m) {
  return A.parts + ((((int64_t)split * tiles + at) * TW + wv) * TT + m) * (TN * WAVE * 4);
}

// Sum of the parts of 16 rows and 64 columns, in the splits' order.
template <bool F32>
__global__ __launch_bounds__(TW* WAVE) void base_join_kernel(BaseArgs A) {
  __shared__ alignas(16) char s_y[TW][16 * 128];
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int tiles = ((A.T + TILE_T - 1) / TILE_T) * ((A.N + TILE_N - 1) / TILE_N);
  const int m = (int)blockIdx.x & (TT - 1);
  TilePlace p;
  if (!tile_place(A, (int)blockIdx.x / TT, p)) return;
  if (p.t0 + 16 * m >= A.T) return;
  f32x4_t acc[TN];
#pragma unroll
  for (int n = 0; n < TN; ++n) acc[n] = f32x4_t{};
  constexpr int AHEAD = 4;
  for (int s0 = 0; s0 < A.splits; s0 += AHEAD) {
    f32x4_t v[AHEAD][TN];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const float* from = part_of(A, tiles, min(s0 + i, A.splits - 1), p.at, wv, m) + lane * 4;
#pragma unroll
      for (int n = 0; n < TN; ++n) v[i][n] = *reinterpret_cast<const f32x4_t*>(from + n * WAVE * 4);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (s0 + i < A.splits)
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[n] += v[i][n];
  }
  store_tile<F32>(A, s_y[wv], p.t0 + 16 * m, p.n0 + wv * (16 * TN), acc);
}

// Workgroup barrier behind this wave's LDS accesses, with its loads from memory left in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <bool E2M1, bool F32, bool ZERO, int S>
__global__ __launch_bounds__(TW* WAVE, 2) void base_tiled_kernel(BaseArgs A) {
  constexpr int PARTS = F32 ? 3 : 1;  // steps of a block
  constexpr int BLOCK_BYTES = block_bytes(E2M1 ? 0 : S), ROW_BYTES = TILE_T * BASE_K * 2;
  __shared__ alignas(16) char s_x[2][BLOCK_BYTES];
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int r = lane & 15, quad = lane >> 4;
  const int tiles = (A.N + BASE_N - 1) / BASE_N;
  const int nt = (A.T + TILE_T - 1) / TILE_T, all = nt * ((A.N + TILE_N - 1) / TILE_N);
  const int run = (all + 7) / 8 * 8, split = blockIdx.x / run;
  TilePlace place;
  if (!tile_place(A, blockIdx.x - split * run, place)) return;
  const int t0 = place.t0, n0 = place.n0 + wv * (16 * TN);
  const int kb0 = split * A.split_blocks * PARTS, kb1 = min((split + 1) * A.split_blocks, A.blocks) * PARTS;

  int64_t tile[TN];  // (columns past the last ones are those again, and not stored)
#pragma unroll
  for (int n = 0; n < TN; ++n) tile[n] = min(n0 / 16 + n, tiles - 1);
  const char* const x = A.rows + (int64_t)(t0 / TILE_T) * A.blocks * PARTS * BLOCK_BYTES;

  struct Weights {
    u32x4_t w[TN];
    BaseScale<E2M1, F32, S> s[TN];
    BaseZero<ZERO, S> z[TN];
  };
  const auto load_weights = [&](int step, Weights& b) {
    const int kb = step / PARTS, row = kb / A.per_group;
#pragma unroll
    for (int n = 0; n < TN; ++n) b.w[n] = static_cast<const u32x4_t*>(A.codes)[(tile[n] * A.blocks + kb) * WAVE + lane];
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      b.s[n] = BaseScale<E2M1, F32, S>::load(A.scale, tile[n] * A.scale_rows + row, r);
      if constexpr (!E2M1) b.z[n] = BaseZero<ZERO, S>::load(A.zero, tile[n] * A.scale_rows + row, r);
    }
  };
  // A wave's quarter of a block of rows; of the sums 16 bytes a thread, the same ones of several (a branch here has the
  // compiler keep two sets of results).
  struct Rows {
    u32x4_t x[TT], sum;
  };
  const int own_row = wv * (ROW_BYTES / TW) + lane * 16, own_sum = ROW_BYTES + (int)(threadIdx.x % (S * TILE_T / 4)) * 16;
  const auto load_rows = [&](int kb, Rows& v) {
    const char* from = x + (int64_t)kb * BLOCK_BYTES;
#pragma unroll
    for (int i = 0; i < TT; ++i) v.x[i] = load_u32x4(from + own_row + i * 1024);
    if constexpr (!E2M1) v.sum = load_u32x4(from + own_sum);
  };
  const auto stage = [&](int buf, const Rows& v) {
#pragma unroll
    for (int i = 0; i < TT; ++i) *reinterpret_cast<u32x4_t*>(s_x[buf] + own_row + i * 1024) = v.x[i];
    if constexpr (!E2M1) *reinterpret_cast<u32x4_t*>(s_x[buf] + own_sum) = v.sum;
  };
  Rows rows;

  f32x4_t acc[TN][TT];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TT; ++m) acc[n][m] = f32x4_t{};

  const auto multiply = [&](int buf, const Weights& b) {
#pragma unroll
    for (int g = 0; g < S; ++g) {
      f32x4_t part[TN][TT], sum[TT];
      if constexpr (!E2M1)
#pragma unroll
        for (int m = 0; m < TT; ++m) sum[m] = *reinterpret_cast<const f32x4_t*>(s_x[buf] + ROW_BYTES + (g * TILE_T + 16 * m + 4 * quad) * 4);
#pragma unroll
      for (int j = g * (4 / S); j < (g + 1) * (4 / S); ++j) {
        bf16x8_t p[TT];
#pragma unroll
        for (int m = 0; m < TT; ++m)
          p[m] = as_bf16x8(load_u32x4(s_x[buf] + (16 * m + r) * 256 + ((4 * j + quad) ^ r) * 16));
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          u32x4_t w;
          if constexpr (E2M1) w = base_floats(b.w[n][j], b.s[n].get(g));
          else w = base_codes(b.w[n][j]);
#pragma unroll
          for (int m = 0; m < TT; ++m) {
            if constexpr (E2M1) {
              acc[n][m] = mfma_16x16x32_bf16(p[m], as_bf16x8(w), acc[n][m]);
            } else {
              f32x4_t from = part[n][m];
              if (j == g * (4 / S)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) from[i] = -b.z[n].get(g) * sum[m][i];
              }
              part[n][m] = mfma_16x16x32_bf16(p[m], as_bf16x8(w), from);
            }
          }
        }
        if constexpr (!E2M1) __builtin_amdgcn_sched_barrier(0x102);  // products stay in their step, for their operands' registers
      }
      if constexpr (!E2M1)
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int m = 0; m < TT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][m][i] = fmaf(b.s[n].get(g), part[n][m][i], acc[n][m][i]);
    }
  };

  // The weight comes two blocks ahead, into the registers of the block just multiplied, rows as those before them go to
  // LDS. (Past the last block it is asked for again: no wait then depends on what is left.)
  const int last = kb1 - 1;
  Weights w[2];
  load_rows(kb0, rows);
  load_weights(kb0, w[0]);
  stage(0, rows);
  load_rows(min(kb0 + 1, last), rows);
  load_weights(min(kb0 + 1, last), w[1]);
  const auto step = [&](int kb, int which) {
    lds_barrier();
    stage(which ^ 1, rows);
    load_rows(min(kb + 2, last), rows);
    multiply(which, w[which]);
    load_weights(min(kb + 2, last), w[which]);
  };
  int kb = kb0;
  for (; kb + 2 <= kb1; kb += 2) {
    step(kb, 0);
    step(kb + 1, 1);
  }
  if (kb < kb1) step(kb, 0);

  if (A.splits > 1) {
#pragma unroll
    for (int m = 0; m < TT; ++m) {
      float* to = part_of(A, all, split, place.at, wv, m) + lane * 4;
#pragma unroll
      for (int n = 0; n < TN; ++n) *reinterpret_cast<f32x4_t*>(to + n * WAVE * 4) = acc[n][m];
    }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < TT; ++m) {
    f32x4_t out[TN];
#pragma unroll
    for (int n = 0; n < TN; ++n) out[n] = acc[n][m];
    store_tile<F32>(A, s_x[0] + (wv * TT + m) * (16 * 128), t0 + 16 * m, n0, out);
  }
}

template <bool E2M1, bool F32, bool ZERO, int S>
hipError_t launch(const BaseArgs& A, hipStream_t stream) {
  const int64_t bands = (A.T + TILE_T - 1) / TILE_T, n = (bands * ((A.N + TILE_N - 1) / TILE_N) + 7) / 8 * 8;
  base_rows_kernel<F32, !E2M1, S><<<(unsigned)(bands * A.blocks), 256, 0, stream>>>(A);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  base_tiled_kernel<E2M1, F32, ZERO, S><<<(unsigned)(n * A.splits), TW * WAVE, 0, stream>>>(A);
  err = hipGetLastError();
  if (err != hipSuccess || A.splits == 1) return err;
  base_join_kernel<F32><<<(unsigned)(n * TT), TW * WAVE, 0, stream>>>(A);
  return hipGetLastError();
}

template <bool F32, bool ZERO>
hipError_t launch_i4(const BaseArgs& A, int s, hipStream_t stream) {
  return s == 4   ? launch<false, F32, ZERO, 4>(A, stream)
         : s == 2 ? launch<false, F32, ZERO, 2>(A, stream)
                  : launch<false, F32, ZERO, 1>(A, stream);
}

template <bool F32>
hipError_t launch_format(const BaseArgs& A, int format, int s, hipStream_t stream) {
  if (format == SGMV_BASE_E2M1) return launch<true, F32, false, 4>(A, stream);
  return A.zero ? launch_i4<F32, true>(A, s, stream) : launch_i4<F32, false>(A, s, stream);
}

}  // namespace

hipError_t launch_base_tiled(const BaseArgs& A, int format, int dtype, int s, hipStream_t stream) {
  return dtype == SGMV_F32 ? launch_format<true>(A, format, s, stream) : launch_format<false>(A, format, s, stream);
}

}  // namespace sgmv
