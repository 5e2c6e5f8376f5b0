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
// Measured, 8 heads of 128, passes over one set of tensors and over eight in turn, which the memory-side cache does not
// hold (floors by a large copy's 5.1 TB/s): 256 sequences' new tokens written as e4m3 5.0 and 5.5 us; 16 prompts' chunks
// (8.9 thousand tokens) of bf16 as int8 or e4m3 13.1 and 17.2 us (55 MB, floor 11: all waves are resident at once, so
// that loads, quantising and stores follow each other; with the page asked for behind the row 14.1 and 19.0), as they
// are 14.1 and 20.6 (14); of fp32 as 8 bits 18.9 and 26.5 (18), as they are 24.9 and 39.9 (28). Read back, over one set
// and over four: the new tokens 4.2 and 4.8 us; 41 thousand tokens of int8 as bf16 46 and 53 us (258 MB, 50), of bf16
// 75 and 75 (67), of e4m3 as fp32 142 and 147 (84), of fp32 188 and 178 (133).
//
// The append turns K on its way, (a, b) -> (a c - b s, b c + a s) with the cosine and sine of the token's position, every
// product and sum rounded to fp32, and the queries, which it writes as rows. V goes as above. K takes lanes of its
// own: 4 values and the 4 that they are paired with in one lane, rows side by side in a wave, so that values and
// angles are loaded once whatever the rotation and the head size; a group's 16 rows are four loads in flight and four
// stores (16 rows a wave in pieces of 16 bytes, as above, needs the pairs' other halves and the angles of 16 values at
// once: 150 registers, or each loaded twice; the chunks below took 54 us, and tokens of D = 256 that bring one each 9.4
// us, now 4.0). The queries are workgroups of the same launch, behind the others (between them, 55 us).
// Bound: the rows' bytes; of few tokens, the chain of loads. Measured with 32 query and 8 key heads of 128: one token 3.2
// us, 16 prompts' chunks (8.6 thousand tokens) into int8 48 us (206 MB, 4.2 TB/s), the queries' part alone 30 (as
// long as a copy of them), K and V 20 (floor 11); 256 tokens of 64 and 8 heads into e4m3 6.4.
#include <algorithm>

#include "quantise.h"

namespace sgmv {

namespace {

constexpr int RW_WAVES = 4;

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

// The page table's entry of a place, whatever it is (-1: the table has none).
__device__ __forceinline__ int page_entry(const KvArgs& K, const Place& P) {
  const int i = P.pos >> K.lps;
  return P.pos < 0 || i >= K.table_pages ? -1 : K.table[(int64_t)P.b * K.ldp + i];
}

// [pages][H][page size] index of a place in the page of an entry, or -1: no page.
__device__ __forceinline__ int64_t token_in(const KvArgs& K, const Place& P, int page) {
  if ((uint32_t)page >= (uint32_t)K.pages) return -1;
  return ((int64_t)page * K.H + P.head) * (1 << K.lps) + (P.pos & ((1 << K.lps) - 1));
}

__device__ __forceinline__ int64_t token_of(const KvArgs& K, const Place& P) { return token_in(K, P, page_entry(K, P)); }

// Place of token r of a group, and token at place r.
__device__ __forceinline__ int place_of(int r) { return 8 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }

// A group of 16 tokens, the first at a multiple of 16: those of its rows that are there.
struct Group {
  int b, head;
  int t0, lo, hi;  // position of the first token, and those of the first row and behind the last
  int64_t row;     // row of position 0
};

// GROUPED: slot `w` of 16 tokens: the groups of sequence b take the slots from first(b) = (rows
// before b) / 16 + 2 b on; n rows touch at most (n + 14) / 16 + 1 groups. start: rows of each sequence,
// the last ones of it.
__device__ __forceinline__ bool find_group(const KvArgs& K, const int32_t* start, int total, int slots, int head, Group& G) {
  const int slot = slots * RW_WAVES + threadIdx.x / WAVE;
  const int b = wave_find(K.B, slot, [&](int i) { return min(max(start[i], 0), total) / 16 + 2 * i; });
  const int r0 = min(max(start[b], 0), total), r1 = min(max(start[b + 1], 0), total);
  const int n = max(r1 - r0, 0), kv_len = kv_seq(K, b).kv_len;
  const int first = kv_len - n;  // position of the first row; may be negative
  const int g0 = (first >> 4) + (slot - (r0 / 16 + 2 * b));
  G = {b, head, 16 * g0, max(16 * g0, first), min(16 * g0 + 16, kv_len), (int64_t)r0 - first};
  return G.lo < G.hi;
}

// Token r of a group.
__device__ __forceinline__ Place place_in(const Group& G, int r) {
  const int t = G.t0 + r, t4 = t & ~3;
  Place P;
  P.head = G.head;
  P.ok = t >= G.lo && t < G.hi;
  P.quad_ok = t4 >= G.lo && t4 + 4 <= G.hi;
  P.whole = G.lo == G.t0 && G.hi == G.t0 + 16;
  P.row = G.row + (P.ok ? t : G.lo);
  P.b = G.b;
  P.pos = t;
  return P;
}

// by_place: lane r of 16 has the token at place r, not token r.
__device__ __forceinline__ bool group_place(const KvArgs& K, const int32_t* start, int total, int slots, int head,
                                            bool by_place, Place& P) {
  const int lane = threadIdx.x & (WAVE - 1);
  Group G;
  if (!find_group(K, start, total, slots, head, G)) return false;
  P = place_in(G, by_place ? place_of(lane & 15) : lane & 15);
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

// N floats of the table of cosines and sines, whose rows start anywhere.
template <int N>
__device__ __forceinline__ void load_angles(const float* p, float (&f)[N]) {
  typedef f32x2_t any8_t __attribute__((aligned(4)));
  typedef f32x4_t any16_t __attribute__((aligned(4)));
  if constexpr (N == 2) {
    const f32x2_t v = *reinterpret_cast<const any8_t*>(p);
    f[0] = v.x;
    f[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4_t v = *reinterpret_cast<const any16_t*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[i + j] = v[j];
    }
  }
}

// Cosines and sines i .. i + N - 1 of a position; past the table they are NaN, so that what they turn is.
template <int N>
__device__ __forceinline__ void angles(const KvTurn& R, int pos, int i, float (&c)[N], float (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] = s[j] = __uint_as_float(0x7fc00000u);
  if ((uint32_t)pos >= (uint32_t)R.positions) return;  // (a row before the first token is not written anyway)
  const float* row = R.cos_sin + pos * R.ld + i;       // (nothing waits for the loads here)
  load_angles(row, c);
  load_angles(row + R.rotary / 2, s);
}

// A pair turned by its angle: two products and their sum, each rounded to fp32.
__device__ __forceinline__ float turn_low(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return a * c - b * s;
}
__device__ __forceinline__ float turn_high(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return b * c + a * s;
}

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
  const int page = page_entry(K, P);  // (loaded beside the row)
  uint32_t w[U::most][U::words];
#pragma unroll
  for (int n = 0; n < U::most; ++n) {
    if (4 * n >= units) break;
    const int u = quad + 4 * n;
#pragma unroll
    for (int i = 0; i < U::words; ++i) w[n][i] = 0u;
    if (P.ok && u < units) load_words(src + u * C, A.vec, w[n]);
  }
  const int64_t at = token_in(K, P, page), token = max(at, (int64_t)0);
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

// Rows of K that are turned, side by side in a wave: a lane takes 8 values of one, two times 4 that are each other's
// pairs (of neighbours, and of what is not turned, 8 in a row), so that values, cosines and sines are loaded once.
// turned_lanes: of a row, as many as a power of two.
__host__ __device__ inline int turned_lanes(int D) {
  int lanes = 2;
  while (lanes * 8 < D) lanes *= 2;
  return lanes;
}

template <class T>
struct TurnedPiece {
  uint32_t a[sizeof(T)], b[sizeof(T)];  // 4 values each
  float c[4], s[4];
};

template <class T, bool NEIGHBOURS>
__device__ __forceinline__ void piece_places(const KvTurn& R, int piece, int& d0, int& d1) {
  const bool halves = !NEIGHBOURS && 8 * piece < R.rotary;
  d0 = halves ? 4 * piece : 8 * piece;
  d1 = d0 + (halves ? R.rotary / 2 : 4);
}

template <class T>
__device__ __forceinline__ void load4(const T* p, uint32_t (&w)[sizeof(T)]) {
  typedef u32x2_t any8_t __attribute__((aligned(2)));
  typedef u32x4_t any16_t __attribute__((aligned(4)));
  if constexpr (sizeof(T) == 2) {
    const u32x2_t v = *reinterpret_cast<const any8_t*>(p);
    w[0] = v[0], w[1] = v[1];
  } else {
    const u32x4_t v = *reinterpret_cast<const any16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  }
}

template <class T, bool NEIGHBOURS>
__device__ __forceinline__ void load_turned(const KvArgs& K, const KvRows& A, const KvTurn& R, const Place& P, int piece,
                                            TurnedPiece<T>& t) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) t.a[i] = t.b[i] = 0u;
  if (!P.ok || 8 * piece >= K.D) return;
  const T* src = static_cast<const T*>(A.k) + P.row * A.ldk_t + P.head * A.ldk_h;
  int d0, d1;
  piece_places<T, NEIGHBOURS>(R, piece, d0, d1);
  load4(src + d0, t.a);
  load4(src + d1, t.b);
  if (8 * piece < R.rotary) angles(R, P.pos, 4 * piece, t.c, t.s);
}

// The largest of 2, 4, 8, 16 or 32 lanes side by side, in all of them.
__device__ __forceinline__ uint32_t side_top(uint32_t top, int lanes) {
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp(top, 0xb1, 0xf, 0xf, true));                 // lane ^ 1
  if (lanes > 2) top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp(top, 0x4e, 0xf, 0xf, true));   // lane ^ 2
  if (lanes > 4) top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp(top, 0x141, 0xf, 0xf, true));  // 8 lanes reversed
  if (lanes > 8) top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp(top, 0x140, 0xf, 0xf, true));  // 16 lanes reversed
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(top, top, false, false);
    top = max(r[0], r[1]);
  }
  return top;
}

// All lanes of a wave call it; `token` negative: the row is not written.
template <int FMT, class T, bool NEIGHBOURS>
__device__ __forceinline__ void write_turned(const KvArgs& K, const KvTurn& R, int64_t token, int lanes, int piece,
                                             const TurnedPiece<T>& t) {
  constexpr int BYTES = KvFormat<FMT>::bytes, C = 16 / BYTES;
  float x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = word_value<T>(t.a, i);
    y[i] = word_value<T>(t.b, i);
  }
  if (8 * piece < R.rotary) {
    if constexpr (NEIGHBOURS) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = x[2 * i], b = y[2 * i];
        x[2 * i] = turn_low(a, x[2 * i + 1], t.c[i], t.s[i]);
        x[2 * i + 1] = turn_high(a, x[2 * i + 1], t.c[i], t.s[i]);
        y[2 * i] = turn_low(b, y[2 * i + 1], t.c[2 + i], t.s[2 + i]);
        y[2 * i + 1] = turn_high(b, y[2 * i + 1], t.c[2 + i], t.s[2 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[i];
        x[i] = turn_low(a, y[i], t.c[i], t.s[i]);
        y[i] = turn_high(a, y[i], t.c[i], t.s[i]);
      }
    }
  }
  uint32_t cx = 0, cy = 0;
  if constexpr (KvFormat<FMT>::scaled) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = word_top<float>(word_top<float>(top, __float_as_uint(x[i])), __float_as_uint(y[i]));
    const RowScale S = row_scale<FMT>(side_top(top, lanes));
    cx = quantise4<FMT, float>(x, S);
    cy = quantise4<FMT, float>(y, S);
    if (piece == 0 && token >= 0) const_cast<float*>(K.k_scale)[token] = S.scale;
  }
  if (token < 0 || 8 * piece >= K.D) return;
  char* dst = static_cast<char*>(const_cast<void*>(K.k)) + (token & ~(int64_t)15) * K.D * BYTES;
  const auto store = [&](int d, uint32_t c, const float (&v)[4]) {
    char* to = dst + ((d / C * 16 + (int)(token & 15)) * C + d % C) * BYTES;
    if constexpr (BYTES == 1) *reinterpret_cast<uint32_t*>(to) = c;
    else if constexpr (BYTES == 2) *reinterpret_cast<u32x2_t*>(to) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[0], v[1], v[2], v[3]};
  };
  int d0, d1;
  piece_places<T, NEIGHBOURS>(R, piece, d0, d1);
  store(d0, cx, x);
  store(d1, cy, y);
}

// The rows of a group; all of its loads are in flight at once but for long rows'.
template <int FMT, class T, bool NEIGHBOURS>
__device__ __forceinline__ void write_turned_group(const KvArgs& K, const KvRows& A, const KvTurn& R, const Group& G) {
  const int lane = threadIdx.x & (WAVE - 1), lanes = turned_lanes(K.D);
  const int piece = lane & (lanes - 1), first = lane / lanes, step = WAVE / lanes;
  Place at = place_in(G, 0);
  const int page = page_entry(K, at);
  for (int r0 = 0; r0 < 16; r0 += 4 * step) {
    TurnedPiece<T> t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i * step + first;
      Place P = place_in(G, r);
      P.ok = P.ok && r < 16;
      load_turned<T, NEIGHBOURS>(K, A, R, P, piece, t[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r0 + i * step >= 16) break;
      const int r = r0 + i * step + first;
      const Place P = place_in(G, r);
      write_turned<FMT, T, NEIGHBOURS>(K, R, P.ok && r < 16 ? token_in(K, P, page) : -1, lanes, piece, t[i]);
    }
  }
}

template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_write_groups_kernel(KvArgs K, KvRows A) {
  Place P;
  if (group_place(K, K.q_start, K.T, blockIdx.x, blockIdx.y, blockIdx.z && KvFormat<FMT>::bytes == 1, P))
    write_rows<FMT, T, true>(K, A, blockIdx.z, P);
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

constexpr int TURN_HEADS = 4;  // that a lane of the queries' waves takes, at most

// How the queries' rows are laid over waves: a lane takes one piece of a head, 16 values that make 8 pairs (of
// neighbours 8, of what is not turned 8 to copy), of `each` heads `side` apart.
struct TurnGrid {
  int turned, pieces;  // pieces of a head that are turned, and all (with those to copy)
  int side, each;      // heads side by side in a wave, and of a lane
  int waves;           // of a token
};

__host__ __device__ inline TurnGrid turn_grid(const KvTurn& R, int T, int D) {
  TurnGrid g;
  g.turned = R.rotary / (R.interleaved ? 8 : 16);
  const bool same = R.q == R.q_out && R.ldq_t == R.ldo_t && R.ldq_h == R.ldo_h;
  g.pieces = g.turned + (same ? 0 : (D - R.rotary) / 8);
  g.side = WAVE / g.pieces;
  // few tokens do not fill the card with waves of several heads a lane
  const int waves = (R.heads + g.side - 1) / g.side;
  g.each = (int64_t)waves * T <= 4096 ? 1 : TURN_HEADS;
  g.waves = (waves + g.each - 1) / g.each;
  return g;
}

// One wave of the queries. A lane reads all that it turns before it writes, so that rows may be turned in place.
template <class T>
__device__ __forceinline__ void turn_queries(const KvArgs& K, const KvTurn& R, int wave) {
  constexpr int W = 2 * sizeof(T);  // words of 8 values
  const int lane = threadIdx.x & (WAVE - 1);
  const TurnGrid G = turn_grid(R, K.T, K.D);
  const int token = wave / G.waves;
  if (token >= K.T) return;
  Place P;
  row_place(K, K.q_start, K.T, token * K.H, P);  // (the same in all lanes)
  if (!P.ok || P.pos < 0) return;
  const int at = lane / G.pieces, piece = lane - at * G.pieces;
  const int head0 = (wave - token * G.waves) * G.side * G.each + at;
  if (at >= G.side) return;
  const T* q = static_cast<const T*>(R.q) + token * R.ldq_t;
  T* out = static_cast<T*>(R.q_out) + token * R.ldo_t;
  const bool copy = piece >= G.turned;
  const int half = R.rotary / 2;
  // the lane's values: d, and of pairs half a rotation apart d + half
  const int d = copy ? R.rotary + 8 * (piece - G.turned) : 8 * piece;
  const bool two = !copy && !R.interleaved;
  uint32_t a[TURN_HEADS][W], b[TURN_HEADS][W];
#pragma unroll
  for (int n = 0; n < TURN_HEADS; ++n) {
    const int head = head0 + n * G.side;
    if (n >= G.each || head >= R.heads) break;
    load_words(q + head * R.ldq_h + d, R.q_vec, a[n]);
    if (two) load_words(q + head * R.ldq_h + d + half, R.q_vec, b[n]);
  }
  float c[8], s[8];
  if (two) {
    angles(R, P.pos, d, c, s);
  } else if (!copy) {
    float c4[4], s4[4];
    angles(R, P.pos, d / 2, c4, s4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = c4[e];
      s[e] = s4[e];
    }
  }
  const auto words = [](const float (&y)[8], uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(y[i]);
      else w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    }
  };
#pragma unroll
  for (int n = 0; n < TURN_HEADS; ++n) {
    const int head = head0 + n * G.side;
    if (n >= G.each || head >= R.heads) break;
    T* to = out + head * R.ldo_h + d;
    if (copy) {
      store_words(to, R.q_vec, a[n]);
      continue;
    }
    float x[8], o[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = word_value<T>(a[n], e);
    uint32_t w[W];
    if (R.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = turn_low(x[2 * e], x[2 * e + 1], c[e], s[e]);
        y[2 * e + 1] = turn_high(x[2 * e], x[2 * e + 1], c[e], s[e]);
      }
      words(y, w);
      store_words(to, R.q_vec, w);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] = word_value<T>(b[n], e);
      y[e] = turn_low(x[e], o[e], c[e], s[e]);
    }
    words(y, w);
    store_words(to, R.q_vec, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = turn_high(x[e], o[e], c[e], s[e]);
    words(y, w);
    store_words(to + half, R.q_vec, w);
  }
}

// As the write kernels, with K turned; workgroups from `rest` on take the queries.
template <int FMT, class T, bool NEIGHBOURS>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_append_groups_kernel(KvArgs K, KvRows A, KvTurn R, int slots, int rest) {
  const int at = blockIdx.x;
  if (at >= rest) return turn_queries<T>(K, R, (at - rest) * RW_WAVES + threadIdx.x / WAVE);
  const bool is_v = at >= rest / 2;
  const int of = is_v ? at - rest / 2 : at, head = of / slots;
  Group G;
  if (!find_group(K, K.q_start, K.T, of - head * slots, head, G) || G.t0 < 0) return;  // (no row before position 0 is read)
  if (!is_v) return write_turned_group<FMT, T, NEIGHBOURS>(K, A, R, G);
  const int r = threadIdx.x & 15;
  write_rows<FMT, T, true>(K, A, true, place_in(G, KvFormat<FMT>::bytes == 1 ? place_of(r) : r));
}

template <int FMT, class T, bool NEIGHBOURS>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_append_rows_kernel(KvArgs K, KvRows A, KvTurn R, int for_v, int rest, int side) {
  const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE, at = blockIdx.x;
  if (at >= rest) return turn_queries<T>(K, R, (at - rest) * RW_WAVES + wv);
  Place P;
  if (at < for_v) {
    row_place(K, K.q_start, K.T, at * RW_WAVES + wv, P);
    P.ok = P.ok && P.pos >= 0;
    write_v_row<FMT, T>(K, A, P);
  } else {
    const int lanes = turned_lanes(K.D), piece = lane & (lanes - 1), of = lane / lanes;
    row_place(K, K.q_start, K.T, ((at - for_v) * RW_WAVES + wv) * side + min(of, side - 1), P);
    P.ok = P.ok && P.pos >= 0 && of < side;
    TurnedPiece<T> t;
    const int page = P.ok ? page_entry(K, P) : -1;
    load_turned<T, NEIGHBOURS>(K, A, R, P, piece, t);
    write_turned<FMT, T, NEIGHBOURS>(K, R, token_in(K, P, page), lanes, piece, t);
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
  if (group_place(K, A.out_start, A.rows, blockIdx.x, blockIdx.y, blockIdx.z && KvFormat<FMT>::bytes == 1, P)) read_rows<FMT, T, true>(K, A, blockIdx.z, P);
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

// Workgroups of an append: of K and V, rows of their own (few new tokens a sequence) or in groups, and of the queries.
//
// Rows or groups, measured at 512 sequences of 8 heads of 128 with 32 query heads, us: one new token each bf16 9.5 and
// 16.7, int8 7.9 and 20.1; two 14.7 and 18.2, 12.7 and 20.8; four 29.7 and 25.8, 22.3 and 26.3; six 34 and 33, 33 and
// 32. Rows of K one or several a wave: one token 3.1 and 4.1, 225 of 4 heads into e4m3 4.8 and 4.7.
struct AppendGrid {
  bool rows;
  int slots;  // of groups, a head
  int side;   // rows of K side by side in a wave
  int64_t for_v, rest, for_q;  // (of rows: those of V, then K's)
};
AppendGrid append_grid(const KvArgs& K, const KvTurn& R, int fmt, int max_q) {
  AppendGrid g{};
  const int64_t rows = (int64_t)K.T * K.H;
  g.rows = max_q <= (fmt == SGMV_KV_E4M3 || fmt == SGMV_KV_I8 ? 4 : 2) && rows <= 0x1000000;
  const dim3 d = group_grid(K, K.T);
  g.side = rows <= 256 ? 1 : WAVE / turned_lanes(K.D);
  g.slots = (int)d.x;
  g.for_v = g.rows ? (rows + RW_WAVES - 1) / RW_WAVES : (int64_t)d.x * d.y;
  g.rest = g.for_v + (g.rows ? (rows + RW_WAVES * g.side - 1) / (RW_WAVES * g.side) : g.for_v);
  g.for_q = R.heads ? ((int64_t)K.T * turn_grid(R, K.T, K.D).waves + RW_WAVES - 1) / RW_WAVES : 0;
  return g;
}

template <int FMT, class T>
void launch_append(const KvArgs& K, const KvRows& A, const KvTurn& R, int max_q, hipStream_t stream) {
  const AppendGrid g = append_grid(K, R, FMT, max_q);
  const unsigned all = (unsigned)(g.rest + g.for_q);
  if (g.rows) {
    const auto kernel = R.interleaved ? kv_append_rows_kernel<FMT, T, true> : kv_append_rows_kernel<FMT, T, false>;
    kernel<<<all, RW_WAVES * WAVE, 0, stream>>>(K, A, R, (int)g.for_v, (int)g.rest, g.side);
  } else {
    const auto kernel = R.interleaved ? kv_append_groups_kernel<FMT, T, true> : kv_append_groups_kernel<FMT, T, false>;
    kernel<<<all, RW_WAVES * WAVE, 0, stream>>>(K, A, R, g.slots, (int)g.rest);
  }
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

// Waves of an append's launch.
int64_t kv_append_waves(const KvArgs& K, const KvTurn& R, int fmt, int max_q) {
  const AppendGrid g = append_grid(K, R, fmt, max_q);
  return (g.rest + g.for_q) * RW_WAVES;
}

hipError_t launch_kv_append(const KvArgs& K, const KvRows& A, const KvTurn& R, int fmt, int max_q, hipStream_t stream) {
  if (fmt == SGMV_KV_F32) launch_append<SGMV_KV_F32, float>(K, A, R, max_q, stream);
  else if (fmt == SGMV_KV_BF16) launch_append<SGMV_KV_BF16, uint16_t>(K, A, R, max_q, stream);
  else if (fmt == SGMV_KV_E4M3 && A.f32) launch_append<SGMV_KV_E4M3, float>(K, A, R, max_q, stream);
  else if (fmt == SGMV_KV_E4M3) launch_append<SGMV_KV_E4M3, uint16_t>(K, A, R, max_q, stream);
  else if (A.f32) launch_append<SGMV_KV_I8, float>(K, A, R, max_q, stream);
  else launch_append<SGMV_KV_I8, uint16_t>(K, A, R, max_q, stream);
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
