// Writing new tokens into the paged key/value cache, quantised on the way, and reading tokens back.
//
// A row is one (token, head): D values. For the 8-bit formats, with F = 448 (e4m3) or 127 (int8):
//   amax = max |x|,  scale = amax / F,  code = round(x * F / amax) to the format, ties to even;
//   a row of zeros has scale 0 and codes 0; a row with a non-finite value has scale NaN and codes
//   0, so that it reads back as NaN whatever the format can hold.
// The code is that of the exact quotient; y = x * (F / amax) in fp32 is within 2^-23 of it.
//   bf16 rows: the quotient of 8-bit significands and F is a border between two codes or at least 2^-16 of
//   it away (their difference, times both denominators, is a whole number). y rounded to 19 bits is that border
//   or on the quotient's side of it, so its code is the quotient's, ties to even with it.
//   fp32 rows: where a little more and a little less than y round to the same code, that is it, and only where
//   they do not (two values in a hundred thousand) the quotient is formed in fp64, rounded to odd first.
// The maximum is taken of the bits, two bf16 at once. So done, a write as e4m3 takes no longer than one of
// bf16 (64 sequences' 100 tokens: 12.4 us both; with an exact division of bf16 values on a border as well, which
// half of all waves have at any step, 18.1).
//
// A wave takes 16 rows, lane r of each quarter (quad) row r, and of every row the pieces of K that are
// 16 bytes in the cache, quad by quad, all of them loaded before the first is stored. K is stored as it is
// held. V has tokens innermost: of 8-bit codes 16 lanes exchange a 16x16 block, after which each holds one d
// of their tokens, 16 bytes of the cache (4x4 blocks and words of 4 bytes took 4% longer); of bf16 four
// exchange a 4x4 block. The 16 rows are the tokens of one group and head (a group, or of bf16 a quad of
// tokens, that is not written whole is stored element by element, so that the others keep theirs), or, where
// sequences bring few tokens, whichever rows follow each other (then a wave of V takes one row). K and V are
// separate waves.
//
// Bound: the rows' bytes; one token per sequence: the chain of loads from the sequence to its page.
// Measured, 8 heads of 128: 256 sequences' new tokens written as e4m3 5.6 us and read back 4.2 us; 16 prompts'
// chunks (8.9 thousand tokens) written as int8 16.0 us (55 MB, 11 us of a large copy: all waves are resident at once,
// so that loads, quantising and stores follow each other), 41 thousand tokens read back as bf16 57 us (258 MB,
// 4.5 TB/s; a large copy: 5.1). Fp32 rows written as e4m3 or int8 19.4 us (floor 17.9), read back 143 (84); rows that
// are held as they are: bf16 written in 13.9 us (14.2), read in 75 (67), fp32 25 (28) and 181 (133).
#include "kv_common.h"

namespace sgmv {

namespace {

constexpr int RW_WAVES = 4;

// fp32 nearest to d, rounded to odd: a later rounding to fewer bits then equals a single one.
__device__ __forceinline__ float to_odd(double d) {
  const float f = __double2float_rz(d);
  return (double)f == d ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// What quantising a row needs: its maximum; a power of two that keeps the parts of a quotient in range, and F
// over the maximum so scaled (0: codes 0); its scale.
struct RowScale {
  float amax, s, inv, scale;
};

// top: bits of the row's maximum of |x| (as integers they order as the values do, infinity and NaN last)
template <int FMT>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
  if (top == 0u || top >= 0x7f800000u) return {0.f, 1.f, 0.f, top ? __uint_as_float(0x7fc00000u) : 0.f};
  const float amax = __uint_as_float(top), s = amax > 0x1p100f ? 0x1p-32f : amax < 0x1p-90f ? 0x1p64f : 1.f;
  return {amax, s, F / (amax * s), amax / F};
}

// Four values rounded to codes. int8: the low bits of 1.5 * 2^23 + q are those of q rounded.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float (&q)[4]) {
  if constexpr (FMT == SGMV_KV_E4M3) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  } else {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 0x1.8p23f);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
  }
}

// Codes of four values of a row.
template <int FMT, class T>
__device__ __forceinline__ uint32_t quantise4(const float (&x)[4], const RowScale& S) {
  constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
  uint32_t w;
  float q[4];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __uint_as_float((__float_as_uint(x[i] * S.s * S.inv) + 16u) & ~31u);
    w = encode4<FMT>(q);
  } else {
    float hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = x[i] * S.s * S.inv;
      q[i] = y * (1.f - 0x1p-22f);
      hi[i] = y * (1.f + 0x1p-22f);
    }
    w = encode4<FMT>(q);
    if (__any(w != encode4<FMT>(hi))) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = to_odd((double)x[i] * (double)F / (double)S.amax);
      w = encode4<FMT>(q);
    }
  }
  return S.inv == 0.f ? 0u : w;
}

// Transposes a 4x4 block of bytes held by 4 neighbouring lanes, one row each.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int lane) {
  uint32_t t = __builtin_amdgcn_mov_dpp(w, 0xb1, 0xf, 0xf, true);  // lane ^ 1
  w = __builtin_amdgcn_perm(t, w, lane & 1 ? 0x03070105u : 0x06020400u);
  t = __builtin_amdgcn_mov_dpp(w, 0x4e, 0xf, 0xf, true);  // lane ^ 2
  return __builtin_amdgcn_perm(t, w, lane & 2 ? 0x03020706u : 0x05040100u);
}

// Transposes a 16x16 block of bytes held by 16 neighbouring lanes, one row each: words between lanes 8 and 4
// apart, then bytes between neighbours.
__device__ __forceinline__ void transpose_16x16(u32x4_t& c, int lane) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // lane ^ 8: a rotation by half of the 16
    const bool up = lane & 8;
    const uint32_t x = c[k], y = c[k + 2], got = __builtin_amdgcn_mov_dpp(up ? x : y, 0x128, 0xf, 0xf, true);
    c[k] = up ? got : x;
    c[k + 2] = up ? y : got;
  }
#pragma unroll
  for (int k = 0; k < 4; k += 2) {  // lane ^ 4: mirrored in 8 (^ 7), then in 4 (^ 3)
    const bool up = lane & 4;
    const uint32_t x = c[k], y = c[k + 1];
    const uint32_t got = __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(up ? x : y, 0x141, 0xf, 0xf, true), 0x1b, 0xf, 0xf, true);
    c[k] = up ? got : x;
    c[k + 1] = up ? y : got;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = transpose_bytes(c[k], lane);
}

// The same of 4x4 16-bit elements, a row in two words.
__device__ __forceinline__ void transpose_halves(uint32_t& a, uint32_t& b, int lane) {
  const bool up = lane & 2, odd = lane & 1;
  const uint32_t other = __builtin_amdgcn_mov_dpp(up ? a : b, 0x4e, 0xf, 0xf, true);
  const uint32_t keep = up ? b : a;
  const uint32_t x = up ? other : keep, y = up ? keep : other;  // of lanes 0 and 2, or 1 and 3
  const uint32_t tx = __builtin_amdgcn_mov_dpp(x, 0xb1, 0xf, 0xf, true);
  const uint32_t ty = __builtin_amdgcn_mov_dpp(y, 0xb1, 0xf, 0xf, true);
  const uint32_t sel = odd ? 0x03020706u : 0x05040100u;  // high halves, low halves
  a = __builtin_amdgcn_perm(tx, x, sel);
  b = __builtin_amdgcn_perm(ty, y, sel);
}

// 4 C bytes (C values of T) of a row, as words; element by element where rows are not aligned.
template <class T, int N>
__device__ __forceinline__ void load_words(const T* p, bool vec, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    u32x4_t v;
    if (vec) {
      v = load_u32x4(reinterpret_cast<const char*>(p) + 16 * i);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const T* e = p + (4 * i + j) * 4 / sizeof(T);
        if constexpr (sizeof(T) == 4) v[j] = *reinterpret_cast<const uint32_t*>(e);
        else v[j] = e[0] | (uint32_t)e[1] << 16;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
  }
}

template <class T, int N>
__device__ __forceinline__ void store_words(T* p, bool vec, const uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    if (vec) {
      *reinterpret_cast<u32x4_t*>(reinterpret_cast<char*>(p) + 16 * i) = u32x4_t{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        T* e = p + (4 * i + j) * 4 / sizeof(T);
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<uint32_t*>(e) = w[4 * i + j];
        } else {
          e[0] = (uint16_t)w[4 * i + j];
          e[1] = (uint16_t)(w[4 * i + j] >> 16);
        }
      }
    }
  }
}

// Value e of a unit held as words of T.
template <class T, int N>
__device__ __forceinline__ float word_value(const uint32_t (&w)[N], int e) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
  return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
}

// The larger |value| of a word of T and of `top`, as bits; 16-bit values in both halves.
template <class T>
__device__ __forceinline__ uint32_t word_top(uint32_t top, uint32_t w) {
  if constexpr (sizeof(T) == 4) return max(top, w & 0x7fffffffu);
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, top),
                                                                __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu)));
}

// That of the lanes of equal lane % 16, as fp32 bits.
template <class T>
__device__ __forceinline__ uint32_t quad_top(uint32_t top) {
  if constexpr (sizeof(T) == 2) top = max(top & 0xffff0000u, top << 16);
  auto r = __builtin_amdgcn_permlane16_swap(top, top, false, false);
  top = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(top, top, false, false);
  return max(r[0], r[1]);
}

// Where the row of this lane goes to or comes from.
struct Place {
  bool ok;        // there is such a row
  bool quad_ok;   // and its three neighbours' (the same quad of tokens) are there too
  bool whole;     // and all 16 of the group
  int64_t row;    // row beside the cache
  int b, pos;     // sequence, position in it
  int head;
};

// [pages][H][page size] index of a place, or -1: no page.
__device__ __forceinline__ int64_t token_of(const KvArgs& K, const Place& P) {
  const int page = kv_page(K, K.table + (int64_t)P.b * K.ldp, P.pos);
  return page < 0 ? -1 : ((int64_t)page * K.H + P.head) * (1 << K.lps) + (P.pos & ((1 << K.lps) - 1));
}

// Place of token r of a group, and token at place r.
__device__ __forceinline__ int place_of(int r) { return 8 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }

// GROUPED: slot `w` of 16 tokens: the groups of sequence b take the slots from first(b) = (rows
// before b) / 16 + 2 b on; n rows touch at most (n + 14) / 16 + 1 groups. start: rows of each sequence,
// the last ones of it.
// by_place: lane r of 16 has the token at place r, not token r.
__device__ __forceinline__ bool group_place(const KvArgs& K, const int32_t* start, int total, bool by_place, Place& P) {
  const int lane = threadIdx.x & (WAVE - 1), r = by_place ? place_of(lane & 15) : lane & 15;
  const int slot = blockIdx.x * RW_WAVES + threadIdx.x / WAVE;
  const int b = wave_find(K.B, slot, [&](int i) { return min(max(start[i], 0), total) / 16 + 2 * i; });
  const int r0 = min(max(start[b], 0), total), r1 = min(max(start[b + 1], 0), total);
  const int n = max(r1 - r0, 0), kv_len = kv_seq(K, b).kv_len;
  const int first = kv_len - n;  // position of the first row; may be negative
  const int g0 = (first >> 4) + (slot - (r0 / 16 + 2 * b));
  const int t_lo = max(16 * g0, first), t_hi = min(16 * g0 + 16, kv_len);
  if (t_lo >= t_hi) return false;
  const int t = 16 * g0 + r, t4 = t & ~3;
  P.head = blockIdx.y;
  P.ok = t >= t_lo && t < t_hi;
  P.quad_ok = t4 >= t_lo && t4 + 4 <= t_hi;
  P.whole = t_lo == 16 * g0 && t_hi == 16 * g0 + 16;
  P.row = P.ok ? r0 + (t - first) : r0;
  P.b = b;
  P.pos = t;
  return true;
}

// Not grouped: row `at` of the rows (token, head) in order, each lane its own; total: rows of tokens,
// those of sequence b start[b] .. start[b + 1], the last ones of it.
__device__ __forceinline__ void row_place(const KvArgs& K, const int32_t* starts, int total, int at, Place& P) {
  const int token_at = at / K.H;
  const bool in = token_at < total;
  const int token = in ? token_at : 0;
  P.head = at - token_at * K.H;
  // the sequence: as if all had the same number of tokens, else by search
  int b = min((int)(((float)token + 0.5f) * ((float)K.B / (float)total)), K.B - 1);
  const auto start = [&](int i) { return min(max(starts[i], 0), total); };
  int s0 = start(b), s1 = start(b + 1);
  uint64_t left = __ballot(in && !(s0 <= token && token < s1));
  while (left) {
    const int t = __builtin_amdgcn_readlane(token, __ffsll((unsigned long long)left) - 1);
    const int found = wave_find(K.B, t, start);
    if (token == t) {
      b = found;
      s0 = start(b);
      s1 = start(b + 1);
    }
    left &= ~__ballot(token == t);
  }
  P.ok = in && s0 <= token && token < s1;
  P.quad_ok = P.whole = false;
  P.row = token;
  P.b = b;
  P.pos = P.ok ? kv_seq(K, b).kv_len - s1 + token : -1;
}

template <int FMT, class T> struct Unit {
  static constexpr int bytes = KvFormat<FMT>::bytes;
  static constexpr int C = 16 / bytes;                          // values of d
  static constexpr int words = C * sizeof(T) / 4;               // of a row beside the cache
  static constexpr int most = SGMV_KV_MAX_HEAD_DIM / C / 4;     // of one lane
};

// Bytes of V that hold value e of unit u for a token of a group.
template <int BYTES>
__device__ __forceinline__ int64_t v_at(int d, int place) { return (int64_t)(d * 16 + place) * BYTES; }

// 16 rows of K (or, grouped, of V) per wave.
template <int FMT, class T, bool GROUPED>
__device__ __forceinline__ void write_rows(const KvArgs& K, const KvRows& A, bool is_v, const Place& place16) {
  using U = Unit<FMT, T>;
  constexpr int BYTES = U::bytes, C = U::C;
  constexpr bool SCALED = KvFormat<FMT>::scaled;
  const int lane = threadIdx.x & (WAVE - 1), quad = lane >> 4;
  Place P = place16;
  if (!__any(P.ok)) return;
  const int D = K.D, units = D / C;
  const T* src = static_cast<const T*>(is_v ? A.v : A.k) + P.row * (is_v ? A.ldv_t : A.ldk_t) +
                 P.head * (is_v ? A.ldv_h : A.ldk_h);
  uint32_t w[U::most][U::words];
#pragma unroll
  for (int n = 0; n < U::most; ++n) {
    if (4 * n >= units) break;
    const int u = quad + 4 * n;
#pragma unroll
    for (int i = 0; i < U::words; ++i) w[n][i] = 0u;
    if (P.ok && u < units) load_words(src + u * C, A.vec, w[n]);
  }
  const int64_t at = token_of(K, P), token = max(at, (int64_t)0);  // the page's load beside the row's
  P.ok = P.ok && at >= 0;
  const int r = (int)(token & 15);
  char* dst = static_cast<char*>(const_cast<void*>(is_v ? K.v : K.k)) + (token & ~(int64_t)15) * D * BYTES;
  RowScale S = {};
  if constexpr (SCALED) {
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < U::most; ++n) {
      if (4 * n >= units) break;
#pragma unroll
      for (int i = 0; i < U::words; ++i) top = word_top<T>(top, w[n][i]);
    }
    S = row_scale<FMT>(quad_top<T>(top));
    if (P.ok && quad == 0) const_cast<float*>(is_v ? K.v_scale : K.k_scale)[token] = S.scale;
  }
#pragma unroll
  for (int n = 0; n < U::most; ++n) {
    if (4 * n >= units) break;
    const int u = quad + 4 * n;
    const bool in = u < units;
    u32x4_t c;  // the unit as it is in the cache
    if constexpr (SCALED) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = word_value<T>(w[n], 4 * k + j);
        c[k] = quantise4<FMT, T>(x, S);
      }
    } else {
      c = u32x4_t{w[n][0], w[n][1], w[n][2], w[n][3]};
    }
    if (!GROUPED || !is_v) {
      if (P.ok && in) *reinterpret_cast<u32x4_t*>(dst + (u * 16 + r) * 16) = c;
      continue;
    }
    if constexpr (BYTES == 4) {  // 16 tokens are 64 bytes
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (P.ok && in) *reinterpret_cast<uint32_t*>(dst + v_at<4>(u * 4 + j, place_of(r))) = c[j];
      continue;
    }
    const bool apart = BYTES == 1 ? !P.whole : !P.quad_ok;  // stored element by element
    if (__any(P.ok && apart)) {
      if (P.ok && apart && in)
#pragma unroll
        for (int e = 0; e < C; ++e) {
          if constexpr (BYTES == 1) dst[v_at<1>(u * C + e, place_of(r))] = (char)(c[e / 4] >> (8 * (e % 4)));
          else *reinterpret_cast<uint16_t*>(dst + v_at<2>(u * C + e, place_of(r))) = (uint16_t)(c[e / 2] >> (16 * (e % 2)));
        }
    }
    if constexpr (BYTES == 1) {
      transpose_16x16(c, lane);
      if (P.whole && P.ok && in) *reinterpret_cast<u32x4_t*>(dst + v_at<1>(u * 16 + (lane & 15), 0)) = c;
    }
    if constexpr (BYTES == 2) {
      const bool put = P.ok && P.quad_ok && in;
      const int j = lane & 3, place = place_of(r & ~3);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t a = c[2 * k], b = c[2 * k + 1];
        transpose_halves(a, b, lane);
        if (put) *reinterpret_cast<u32x2_t*>(dst + v_at<2>(u * 8 + 4 * k + j, place)) = u32x2_t{a, b};
      }
    }
  }
}

// One row of V per wave: its places in the cache are 16 elements apart, and lanes side by side in d
// share cache lines (16 rows per wave, every lane in another line, took twice as long).
template <int FMT, class T>
__device__ __forceinline__ void write_v_row(const KvArgs& K, const KvRows& A, const Place& P) {
  constexpr int BYTES = KvFormat<FMT>::bytes, MOST = SGMV_KV_MAX_HEAD_DIM / WAVE;
  const int lane = threadIdx.x & (WAVE - 1), D = K.D;
  if (!P.ok) return;
  const T* src = static_cast<const T*>(A.v) + P.row * A.ldv_t + P.head * A.ldv_h;
  T e[MOST];
  float x[MOST];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    e[i] = lane + WAVE * i < D ? src[lane + WAVE * i] : T(0);
    if constexpr (sizeof(T) == 4) x[i] = e[i];
    else x[i] = bf16_bits_to_f32(e[i]);
    top = word_top<float>(top, __float_as_uint(x[i]));
  }
  const int64_t token = token_of(K, P);
  if (token < 0) return;
  char* dst = static_cast<char*>(const_cast<void*>(K.v)) + (token & ~(int64_t)15) * D * BYTES;
  const int place = place_of((int)(token & 15));
  uint32_t c = 0;
  if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    const RowScale S = row_scale<FMT>(quad_top<float>(top));
    c = quantise4<FMT, T>(x, S);
    if (lane == 0) const_cast<float*>(K.v_scale)[token] = S.scale;
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int d = lane + WAVE * i;
    if (d >= D) break;
    if constexpr (BYTES == 1) dst[v_at<1>(d, place)] = (char)(c >> (8 * i));
    else *reinterpret_cast<T*>(dst + v_at<BYTES>(d, place)) = e[i];
  }
}

template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_write_groups_kernel(KvArgs K, KvRows A) {
  Place P;
  if (group_place(K, K.q_start, K.T, blockIdx.z && KvFormat<FMT>::bytes == 1, P)) write_rows<FMT, T, true>(K, A, blockIdx.z, P);
}

// Workgroups [0, for_v) take V, the others K.
template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_write_rows_kernel(KvArgs K, KvRows A, int for_v) {
  const int wv = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
  Place P;
  if ((int)blockIdx.x < for_v) {
    row_place(K, K.q_start, K.T, (int)blockIdx.x * RW_WAVES + wv, P);
    write_v_row<FMT, T>(K, A, P);
  } else {
    row_place(K, K.q_start, K.T, (((int)blockIdx.x - for_v) * RW_WAVES + wv) * 16 + (lane & 15), P);
    write_rows<FMT, T, false>(K, A, false, P);
  }
}

// 16 rows of K (or, grouped, of V) per wave.
template <int FMT, class T, bool GROUPED>
__device__ __forceinline__ void read_rows(const KvArgs& K, const KvRows& A, bool is_v, const Place& P) {
  using U = Unit<FMT, T>;
  constexpr int BYTES = U::bytes, C = U::C;
  const int lane = threadIdx.x & (WAVE - 1), quad = lane >> 4;
  const int D = K.D, units = D / C;
  const int64_t at = token_of(K, P), token = max(at, (int64_t)0);
  const bool there = at >= 0;
  const int r = (int)(token & 15);
  const char* src = static_cast<const char*>(is_v ? K.v : K.k) + (token & ~(int64_t)15) * D * BYTES;
  T* dst = static_cast<T*>(is_v ? A.v : A.k) + P.row * (is_v ? A.ldv_t : A.ldk_t) + P.head * (is_v ? A.ldv_h : A.ldk_h);
  float scale = 1.f;
  if constexpr (KvFormat<FMT>::scaled) {
    if (there) scale = (is_v ? K.v_scale : K.k_scale)[token];
  }
  u32x4_t all[U::most];  // of every unit before the first store
#pragma unroll
  for (int n = 0; n < U::most; ++n) {
    if (4 * n >= units) break;
    const int u = quad + 4 * n;
    u32x4_t c = {0u, 0u, 0u, 0u};
    if (there && u < units) {
      if (!GROUPED || !is_v) {
        c = load_u32x4(src + (u * 16 + r) * 16);
      } else {
        const int j = lane & 3, place = place_of(r & ~3);
        if constexpr (BYTES == 1) c = load_u32x4(src + v_at<1>(u * 16 + (lane & 15), 0));
        if constexpr (BYTES == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const uint32_t*>(src + v_at<4>(u * 4 + k, place_of(r)));
        }
        if constexpr (BYTES == 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const u32x2_t x = *reinterpret_cast<const u32x2_t*>(src + v_at<2>(u * 8 + 4 * k + j, place));
            c[2 * k] = x.x;
            c[2 * k + 1] = x.y;
          }
        }
      }
    }
    all[n] = c;
  }
#pragma unroll
  for (int n = 0; n < U::most; ++n) {
    if (4 * n >= units) break;
    const int u = quad + 4 * n;
    u32x4_t c = all[n];
    if (GROUPED && is_v) {
      if constexpr (BYTES == 1) transpose_16x16(c, lane);
      if constexpr (BYTES == 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t a = c[2 * k], b = c[2 * k + 1];
          transpose_halves(a, b, lane);
          c[2 * k] = a;
          c[2 * k + 1] = b;
        }
      }
    }
    uint32_t w[U::words];
    if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
        codes4<FMT>(c[k], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = there ? f[j] * scale : 0.f;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[4 * k + j] = __float_as_uint(f[j]);
        } else {
          w[2 * k] = pack_bf16x2(f[0], f[1]);
          w[2 * k + 1] = pack_bf16x2(f[2], f[3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = c[k];
    }
    if (P.ok && u < units) store_words(dst + u * C, A.vec, w);
  }
}

// One row of V per wave (see write_v_row).
template <int FMT, class T>
__device__ __forceinline__ void read_v_row(const KvArgs& K, const KvRows& A, const Place& P) {
  constexpr int BYTES = KvFormat<FMT>::bytes, MOST = SGMV_KV_MAX_HEAD_DIM / WAVE;
  const int lane = threadIdx.x & (WAVE - 1), D = K.D;
  if (!P.ok) return;
  T* dst = static_cast<T*>(A.v) + P.row * A.ldv_t + P.head * A.ldv_h;
  const int64_t at = token_of(K, P), token = max(at, (int64_t)0);
  const char* src = static_cast<const char*>(K.v) + (token & ~(int64_t)15) * D * BYTES;
  const int place = place_of((int)(token & 15));
  float scale = 1.f;
  if constexpr (KvFormat<FMT>::scaled) scale = K.v_scale[token];
  T e[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int d = min(lane + WAVE * i, D - 1);
    if constexpr (BYTES == 1) {
      float f[4];
      codes4<FMT>(static_cast<const uint8_t*>(static_cast<const void*>(src))[d * 16 + place], f);
      if constexpr (sizeof(T) == 4) e[i] = f[0] * scale;
      else e[i] = (T)pack_bf16x2(f[0] * scale, 0.f);
    } else {
      e[i] = *reinterpret_cast<const T*>(src + v_at<BYTES>(d, place));
    }
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    if (lane + WAVE * i < D) dst[lane + WAVE * i] = at < 0 ? T(0) : e[i];
}

template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_read_groups_kernel(KvArgs K, KvRows A) {
  Place P;
  if (group_place(K, A.out_start, A.rows, blockIdx.z && KvFormat<FMT>::bytes == 1, P)) read_rows<FMT, T, true>(K, A, blockIdx.z, P);
}

template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_read_rows_kernel(KvArgs K, KvRows A, int for_v) {
  const int wv = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
  Place P;
  if ((int)blockIdx.x < for_v) {
    row_place(K, A.out_start, A.rows, (int)blockIdx.x * RW_WAVES + wv, P);
    read_v_row<FMT, T>(K, A, P);
  } else {
    row_place(K, A.out_start, A.rows, (((int)blockIdx.x - for_v) * RW_WAVES + wv) * 16 + (lane & 15), P);
    read_rows<FMT, T, false>(K, A, false, P);
  }
}

// Slots of 16-token groups for `tokens` rows of B sequences (see group_place).
dim3 group_grid(const KvArgs& K, int64_t tokens) {
  const int64_t slots = tokens / 16 + 2 * (int64_t)K.B;
  return dim3((unsigned)((slots + RW_WAVES - 1) / RW_WAVES), (unsigned)K.H, 2);
}

// Row by row while groups would be mostly empty: workgroups for V and in all (0: by groups).
struct RowGrid {
  int for_v;
  unsigned all;
};
RowGrid row_grid(const KvArgs& K, int64_t tokens, bool few) {
  const int64_t rows = tokens * K.H, for_v = (rows + RW_WAVES - 1) / RW_WAVES;
  if (!few || rows > 0x3000000) return {0, 0};  // (a launch takes fewer than 2^32 work items, 68 of each row)
  return {(int)for_v, (unsigned)(for_v + (rows + 16 * RW_WAVES - 1) / (16 * RW_WAVES))};
}

template <int FMT, class T>
void launch_write(const KvArgs& K, const KvRows& R, int max_q, hipStream_t stream) {
  const RowGrid g = row_grid(K, K.T, max_q <= 8);
  if (g.all) kv_write_rows_kernel<FMT, T><<<g.all, RW_WAVES * WAVE, 0, stream>>>(K, R, g.for_v);
  else kv_write_groups_kernel<FMT, T><<<group_grid(K, K.T), RW_WAVES * WAVE, 0, stream>>>(K, R);
}

template <int FMT, class T>
void launch_read(const KvArgs& K, const KvRows& R, hipStream_t stream) {
  const RowGrid g = row_grid(K, R.rows, R.rows <= 4 * (int64_t)K.B);
  if (g.all) kv_read_rows_kernel<FMT, T><<<g.all, RW_WAVES * WAVE, 0, stream>>>(K, R, g.for_v);
  else kv_read_groups_kernel<FMT, T><<<group_grid(K, R.rows), RW_WAVES * WAVE, 0, stream>>>(K, R);
}

}  // namespace

hipError_t launch_kv_write(const KvArgs& K, const KvRows& R, int fmt, int max_q, hipStream_t stream) {
  if (fmt == SGMV_KV_F32) launch_write<SGMV_KV_F32, float>(K, R, max_q, stream);
  else if (fmt == SGMV_KV_BF16) launch_write<SGMV_KV_BF16, uint16_t>(K, R, max_q, stream);
  else if (fmt == SGMV_KV_E4M3 && R.f32) launch_write<SGMV_KV_E4M3, float>(K, R, max_q, stream);
  else if (fmt == SGMV_KV_E4M3) launch_write<SGMV_KV_E4M3, uint16_t>(K, R, max_q, stream);
  else if (R.f32) launch_write<SGMV_KV_I8, float>(K, R, max_q, stream);
  else launch_write<SGMV_KV_I8, uint16_t>(K, R, max_q, stream);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs& K, const KvRows& R, int fmt, hipStream_t stream) {
  if (fmt == SGMV_KV_F32) launch_read<SGMV_KV_F32, float>(K, R, stream);
  else if (fmt == SGMV_KV_BF16) launch_read<SGMV_KV_BF16, uint16_t>(K, R, stream);
  else if (fmt == SGMV_KV_E4M3 && R.f32) launch_read<SGMV_KV_E4M3, float>(K, R, stream);
  else if (fmt == SGMV_KV_E4M3) launch_read<SGMV_KV_E4M3, uint16_t>(K, R, stream);
  else if (R.f32) launch_read<SGMV_KV_I8, float>(K, R, stream);
  else launch_read<SGMV_KV_I8, uint16_t>(K, R, stream);
  return hipGetLastError();
}

}  // namespace sgmv
