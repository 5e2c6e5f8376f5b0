// Shared definitions of the paged key/value cache: its layout on the device, the step's batch, and
// the conversions between stored codes and matrix-core operands.
//
// Tokens are stored in groups of 16 inside a page, per (page, head) one contiguous block:
//   K group  [D / c][16 tokens][c]   c = 16 bytes of elements
//   V group  [D][16 places]          place of token t: 8 * ((t / 4) % 2) + 4 * (t / 8) + t % 4
// A 32x32 product K Q^T leaves lane (column, half) with tokens 8 * (i / 4) + 4 * half + i % 4 of
// its column in register i. With V's places in that order, the 8 probabilities that a lane holds
// of one group are the k values of its half in the next product, V^T P^T, and the 8 elements of V
// that go with them are one contiguous load: the probabilities never leave their registers.
#pragma once

#include "common.h"

namespace sgmv {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int KV_GROUP = 16;

// Device view of a cache and a step's batch (passed by value).
struct KvArgs {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t ldp;
  int32_t pages, lps;  // lps: log2 of the page size
  int32_t table_pages;
  int32_t B, T, H, D;
};

// Rows [rows][H][D] beside the cache: read by the write call, written by the read call.
struct KvRows {
  void* k;
  void* v;
  int64_t ldk_t, ldk_h, ldv_t, ldv_h;
  const int32_t* out_start;  // read call: first row of each sequence
  int32_t rows;              // read call
  int32_t f32;               // rows are fp32, else bf16
  int32_t vec;               // rows may be accessed 16 bytes at a time
};

// One sequence of the batch, whatever the arrays hold: its first new token, its new tokens and
// its length, clamped so that nothing they lead to lies outside the arrays.
struct KvSeq {
  int q0, q_len, kv_len;
};

__device__ __forceinline__ KvSeq kv_seq(const KvArgs& A, int b) {
  KvSeq s;
  const int a = min(max(A.q_start[b], 0), A.T), e = min(max(A.q_start[b + 1], 0), A.T);
  s.q0 = a;
  s.q_len = max(e - a, 0);
  const int64_t most = (int64_t)A.table_pages << A.lps;
  s.kv_len = (int)min((int64_t)max(A.kv_len[b], 0), min(most, (int64_t)0x7fffff00));
  return s;
}

// Page of token t of a sequence, or -1 where there is none.
__device__ __forceinline__ int kv_page(const KvArgs& A, const int32_t* row, int t) {
  const int i = t >> A.lps;
  if (t < 0 || i >= A.table_pages) return -1;
  const int p = row[i];
  return (uint32_t)p < (uint32_t)A.pages ? p : -1;
}

// The last b in [0, B) with start(b) <= x, for a start that does not decrease: each round looks at
// 64 places at once, one per lane.
template <class F>
__device__ __forceinline__ int wave_find(int B, int x, F start) {
  const int lane = threadIdx.x & (WAVE - 1);
  int lo = 0, n = B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + WAVE - 1) / WAVE;
    const int at = lo + lane * step;
    const bool le = lane * step < n && start(at) <= x;
    const int c = __popcll(__ballot(le));
    const int k = max(c, 1) - 1;
    const int left = n - k * step;
    lo += k * step;
    n = min(step, left);
  }
  return lo;
}

// Maximum of a value over the two halves of the wave, in both.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Maximum and sum of a value over the lanes of equal lane % 16, in all of them.
__device__ __forceinline__ float quad_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

__device__ __forceinline__ float quad_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// ---------------------------------------------------------------------------------------
// stored formats
// ---------------------------------------------------------------------------------------
template <int FMT> struct KvFormat;  // sgmv_kv_format
template <> struct KvFormat<SGMV_KV_F32> { static constexpr int bytes = 4; static constexpr bool scaled = false; };
template <> struct KvFormat<SGMV_KV_BF16> { static constexpr int bytes = 2; static constexpr bool scaled = false; };
template <> struct KvFormat<SGMV_KV_E4M3> { static constexpr int bytes = 1; static constexpr bool scaled = true; };
template <> struct KvFormat<SGMV_KV_I8> { static constexpr int bytes = 1; static constexpr bool scaled = true; };

// Four codes of one 32-bit word as floats (exact).
template <int FMT>
__device__ __forceinline__ void codes4(uint32_t w, float (&f)[4]) {
  if constexpr (FMT == SGMV_KV_E4M3) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else {
    f[0] = (float)(int8_t)(w & 0xff);
    f[1] = (float)(int8_t)((w >> 8) & 0xff);
    f[2] = (float)(int8_t)((w >> 16) & 0xff);
    f[3] = (float)((int32_t)w >> 24);
  }
}

// Eight codes as bf16 (exact: e4m3 has 4 significant bits, int8 at most 8).
template <int FMT>
__device__ __forceinline__ u32x4_t codes8_bf16(u32x2_t w) {
  u32x4_t r;
  if constexpr (FMT == SGMV_KV_E4M3) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.f, true));
  } else {
    float a[4], b[4];
    codes4<FMT>(w.x, a);
    codes4<FMT>(w.y, b);
    // exact values: the upper halves of the floats
    r.x = __builtin_amdgcn_perm(__float_as_uint(a[1]), __float_as_uint(a[0]), 0x07060302u);
    r.y = __builtin_amdgcn_perm(__float_as_uint(a[3]), __float_as_uint(a[2]), 0x07060302u);
    r.z = __builtin_amdgcn_perm(__float_as_uint(b[1]), __float_as_uint(b[0]), 0x07060302u);
    r.w = __builtin_amdgcn_perm(__float_as_uint(b[3]), __float_as_uint(b[2]), 0x07060302u);
  }
  return r;
}

}  // namespace sgmv
