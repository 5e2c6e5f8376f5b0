// Attention of a step's new tokens over the paged cache: arguments and the steps that the kernels
// share. Row r of a sequence and key/value head is (new token r / G, query head r % G of the
// group), so that the G query heads of a key/value head share its tiles.
#pragma once

#include "kv_common.h"

namespace sgmv {

constexpr int AT_ROWS = 32;   // rows of one wave of the tiled kernel
constexpr int AT_TOKENS = 32; // granularity of a window's first token

struct AttnArgs {
  KvArgs kv;
  const void* q;
  void* out;
  float* lse;  // [T][Hq], may be null
  int64_t ldq_t, ldq_h, ldo_t, ldo_h;
  int32_t Hq, G;
  int32_t f32;         // q and out are fp32, else bf16
  int32_t q_vec;       // q rows may be read 16 bytes at a time
  int32_t o_vec;       // out rows may be written 8 bytes (bf16) or 16 (fp32) at a time
  float scale_log2;    // scale * log2(e)
  int32_t window;      // 0: none
  // rows of one sequence up to which the direct kernel takes it (the tiled kernel takes the
  // others; 0: all); INT32_MAX: the direct kernel takes all
  int32_t direct_rows;
  int32_t direct_tile; // rows of the direct kernel's workgroups: 16 or 32
  int32_t direct_waves;  // and their waves: 4 or 8
  int32_t one_tile;    // direct kernel: every sequence it takes has at most that many rows
  // split of a sequence's tokens over workgroups: `n_split` ranges of `chunk` tokens (a multiple
  // of the tile), the last one to the end
  int32_t chunk[2], n_split[2];  // [0] direct kernel, [1] tiled kernel
  int32_t slots[2];    // tiles of rows that the grid has room for (0: none)
  // parts of the ranges, for each kernel [n_split][part_rows][D] and [n_split][part_rows][2]: maximum (of
  // scores times log2(e)), sum. The row of a part: token and query head, or, where there are fewer of
  // those, row of the kernel's tiles (part_row).
  float* part_o[2];
  float* part_ml[2];
  int64_t part_rows[2];
  int32_t part_tile[2];  // rows of a tile, 0: by token and query head
};

// Whether the direct kernel has instances of two 16-row tiles per workgroup.
constexpr bool direct_two_tiles(int D, bool f32) { return D <= 128 || (D == 192 && !f32); }

// Whether it has instances of 8 waves per workgroup next to those of 4 (bf16 rows).
constexpr bool direct_eight_waves(int D, bool f32) { return D <= 128 && !f32; }

// The tiled kernel: head dimensions it has instances of, waves and rows of its workgroups.
constexpr bool tiled_dim(int D) { return D == 64 || D == 80 || D == 96 || D == 128 || D == 192 || D == 256; }
constexpr int tiled_waves(int D) { return D <= 128 ? 8 : 4; }
constexpr int tiled_rows(int D) { return tiled_waves(D) * AT_ROWS; }

// Rows of a sequence up to which a call with tiles of many rows takes it directly.
constexpr int tiled_direct_rows(int D) { return direct_two_tiles(D, false) ? 32 : 16; }

// Tokens that rows [row0, row0 + n) of a sequence look at: [begin, end), begin a multiple of 32.
struct Span {
  int begin, end;
};

__device__ __forceinline__ Span row_span(const AttnArgs& A, const KvSeq& s, int row0, int n) {
  const int rows = s.q_len * A.G;
  const int lo = row0 / A.G, hi = (min(row0 + n, rows) - 1) / A.G;
  const int first = s.kv_len - s.q_len;
  Span p;
  p.end = max(first + hi + 1, 0);
  // (a row before the first token sees nothing: no difference that passes 32 bits for the widest windows)
  p.begin = A.window ? max(max(first + lo + 1, 0) - A.window, 0) & ~(AT_TOKENS - 1) : 0;
  return p;
}

// Ranges that the tokens of a span are split into, for the direct (0) or the tiled (1) kernel.
__device__ __forceinline__ int span_splits(const AttnArgs& A, const Span& p, int kernel) {
  const int chunk = A.chunk[kernel];
  return min(max((p.end - p.begin + chunk - 1) / chunk, 1), A.n_split[kernel]);
}

// Row of the parts that belong to row `local` of a tile, of token and query head `at`.
__device__ __forceinline__ int64_t part_row(const AttnArgs& A, int kernel, int slot, int kvh, int local, int64_t at) {
  return A.part_tile[kernel] ? ((int64_t)slot * A.kv.H + kvh) * A.part_tile[kernel] + local : at;
}

__device__ __forceinline__ f32x16_t mfma_32x32_bf16(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// Token of register i of a 32x32 product's lane in half h.
__device__ __forceinline__ int reg_token(int i, int h) { return (i & 3) + 8 * (i >> 2) + 4 * h; }

// Four values of one output row from element `at` on.
template <bool F32>
__device__ __forceinline__ void store_out(const AttnArgs& A, int64_t at, float a, float b, float c, float d) {
  if constexpr (F32) {
    float* p = static_cast<float*>(A.out) + at;
    if (A.o_vec) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{a, b, c, d};
    } else {
      p[0] = a; p[1] = b; p[2] = c; p[3] = d;
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(A.out) + at;
    const u32x2_t w = {pack_bf16x2(a, b), pack_bf16x2(c, d)};
    if (A.o_vec) {
      *reinterpret_cast<u32x2_t*>(p) = w;
    } else {
      p[0] = (uint16_t)w.x; p[1] = (uint16_t)(w.x >> 16);
      p[2] = (uint16_t)w.y; p[3] = (uint16_t)(w.y >> 16);
    }
  }
}

__device__ __forceinline__ f32x4_t mfma_16x16x4_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

}  // namespace sgmv
