// Attention over the paged cache with keys and values loaded straight into matrix-core operands.
//
// For one (sequence, key/value head), a tile of 16 R rows (new token, query head of the group) and a
// range of tokens, each of the workgroup's waves takes every WAVES-th step of TOK tokens:
//   S^T = K Q^T   (tokens x rows),  p = exp2(c s - m),  O^T += V^T P^T,   one running (m, l) per row.
// In a 16x16 product lane (r = lane % 16, quad = lane / 16) gives row r of the left operand, column r of
// the right one and the inner indices 8 quad .. 8 quad + 7, and holds the result's rows 4 quad .. 4 quad
// + 3 of column r. Which token is a product's row is free: tile x gives row 4 q + i the token at place
// 4 x + i (V's order) of the piece that quad q loads of V, 16 bytes of one d. So a lane's probabilities
// are the right operand of the next product as they stand, every load of K and V is 16 bytes wide, and
// nothing goes through LDS but the waves' sums at the end. Scores, maxima, sums and outputs are fp32. With bf16
// rows the probabilities, times V's scales, are rounded to bf16 for that product: at most 2^-8 of sum p |v| / sum p,
// as the output's own rounding is 2^-8 of it, where fp32 products have a sixteenth of the rate. TOK is what makes those pieces whole:
// 64 tokens of 8-bit codes (quad q: group q), 32 of wider ones (quad q: half q % 2 of group q / 2).
//
// Bound: the bytes of K and V, read once per tile of rows. K and V of the next step are in flight while
// this one is computed, with two waves per SIMD at a head dimension of 128. Scales of 8-bit tokens are one
// load per lane, spread by row broadcasts: as 16-byte loads they took the registers that make the
// difference (64 sequences' drafts, int8: 238 us, 150 without their spills; 138 now). Measured (64 / 8 heads of 128):
// 256 sequences of 128..4096, bf16: 397 us, 5.6 TB/s of K and V (a large copy: 5.1); 16 of
// 8001..64003, e4m3: 233 us, 5.2 TB/s. One token over 1001, bf16: 8.9 us, the chain of loads from the
// sequence to its page to K, then 4 steps of 8 waves.
#pragma once

#include <utility>

#include "attn_operand.h"

namespace sgmv {

template <bool F32, int FMT> struct Direct {
  static constexpr int bytes = KvFormat<FMT>::bytes;
  static constexpr int C = 16 / bytes;                // values of d in one piece of K
  static constexpr int q_regs = F32 ? C : C / 2;      // registers of Q that go with one piece
  static constexpr int tokens = bytes == 1 ? 64 : 32; // of one step
  static constexpr int NT = tokens / 16;              // 16-token tiles of a step
  static constexpr int v_loads = bytes == 4 ? 2 : 1;  // pieces of V per 16 values of d

  // A piece of K (or of V) as operands: codes in bf16, or the values of fp32 products.
  struct Operand {
    u32x4_t h[F32 ? 1 : C / 8];
    float f[F32 ? C : 1];
  };
  static __device__ __forceinline__ Operand operand(u32x4_t w) {
    Operand a;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (bytes == 4) {
          a.f[i] = __uint_as_float(w[i]);
        } else {
          float g[4];
          codes4<FMT>(w[i], g);
#pragma unroll
          for (int j = 0; j < 4; ++j) a.f[4 * i + j] = g[j];
        }
      }
    } else if constexpr (bytes == 2) {
      a.h[0] = w;
    } else {
      a.h[0] = codes8_bf16<FMT>(u32x2_t{w.x, w.y});
      a.h[1] = codes8_bf16<FMT>(u32x2_t{w.z, w.w});
    }
    return a;
  }
  // s += K piece times Q piece
  static __device__ __forceinline__ f32x4_t qk(const Operand& k, const uint32_t (&q)[q_regs], f32x4_t s) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < C; ++i) s = mfma_16x16x4_f32(k.f[i], __uint_as_float(q[i]), s);
    } else {
#pragma unroll
      for (int i = 0; i < C / 8; ++i)
        s = mfma_16x16x32_bf16(as_bf16x8(k.h[i]), as_bf16x8(u32x4_t{q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]}), s);
    }
    return s;
  }
};

// The value of lane I of each 16 lanes, in all of them.
template <int I>
__device__ __forceinline__ float row_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x150 + I, 0xf, 0xf, true));
}

// f(0), .., f(15) with constants.
template <class F, int... I>
__device__ __forceinline__ void each_place(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <class F>
__device__ __forceinline__ void for_places(F f) {
  each_place(f, std::make_integer_sequence<int, 16>{});
}

// Waves per SIMD to allocate registers for.
constexpr int direct_occupancy(bool f32, int DP, int R) {
  if (f32) return DP <= 64 && R == 1 ? 2 : 1;
  if (DP <= 64 && R == 1) return 3;
  return DP <= 128 ? 2 : 1;
}

// The waves' sums.
template <int DP, int R, int WAVES> struct DirectShared {
  static constexpr int ROWS = 16 * R, LD = DP + 4;
  float m[WAVES][ROWS], l[WAVES][ROWS];
  alignas(16) float o[WAVES][ROWS * LD];
};

// One workgroup's piece. DP: head dimension, or (not EXACT) an upper bound of it
template <bool F32, int FMT, int DP, bool EXACT, int R, int WAVES>
__device__ __forceinline__ void attn_direct(const AttnArgs& A, int piece, DirectShared<DP, R, WAVES>& sh) {
  using X = Direct<F32, FMT>;
  constexpr int C = X::C, NT = X::NT, TOK = X::tokens, NG = TOK / 16, BYTES = X::bytes;
  constexpr bool SCALED = KvFormat<FMT>::scaled;
  constexpr int NCH = (DP / C + 3) / 4;  // pieces of K of one lane, per tile
  constexpr int NB = DP / 16;            // blocks of 16 values of d
  constexpr int VL = X::v_loads;
  constexpr int ROWS = 16 * R, LD = DP + 4;
  // wide fp32 rows: V in the registers that K had, not next to it (its products take longer than a load)
  constexpr bool LATE_V = BYTES == 4 && DP > 128;
  auto& s_m = sh.m;
  auto& s_l = sh.l;
  auto& s_o = sh.o;
  const KvArgs& K = A.kv;
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int r = lane & 15, quad = lane >> 4;
  const int D = EXACT ? DP : K.D;

  // this workgroup's piece: first ranges first, so that the ranges that shorter sequences lack come
  // last instead of leaving the same shader engines idle throughout
  const int kvh = piece % K.H;
  const int rest = piece / K.H;
  const int split = rest / A.slots[0], slot = rest - split * A.slots[0];
  int b, row0;
  if (A.one_tile) {
    b = slot;
    row0 = 0;
  } else {
    // row tiles of sequence b take the slots from (rows before b) / ROWS + b on
    b = wave_find(K.B, slot, [&](int i) {
      return (int)((int64_t)min(max(K.q_start[i], 0), K.T) * A.G / ROWS) + i;
    });
    b = __builtin_amdgcn_readfirstlane(b);
    row0 = (slot - ((int)((int64_t)min(max(K.q_start[b], 0), K.T) * A.G / ROWS) + b)) * ROWS;
  }
  const KvSeq s = kv_seq(K, b);
  const int rows = s.q_len * A.G;
  if (row0 < 0 || row0 >= rows || rows > A.direct_rows) return;
  const Span span = row_span(A, s, row0, ROWS);
  const int used = span_splits(A, span, 0);
  if (split >= used) return;
  const int t_begin = span.begin + split * A.chunk[0];
  const int t_end = split == used - 1 ? span.end : t_begin + A.chunk[0];

  const int first = s.kv_len - s.q_len;
  const int lo_pos = first + row0 / A.G;  // positions of the tile's first and last row
  const int hi_pos = first + (min(row0 + ROWS, rows) - 1) / A.G;
  const int ps = 1 << K.lps;
  const int32_t* table = K.table + (int64_t)b * K.ldp;

  // pages of this wave's next 64 / NG steps, lane NG i + g that of group g of step i, and of those
  // that follow
  constexpr int STEPS = WAVE / NG;
  auto load_pages = [&](int i0) {
    const int t = t_begin + TOK * (wv + WAVES * (i0 + lane / NG)) + 16 * (lane % NG);
    return t < t_end ? kv_page(K, table, t) : -1;
  };
  const int n_steps = max((t_end - t_begin + TOK - 1) / TOK, 0);
  const int mine = wv < n_steps ? (n_steps - wv + WAVES - 1) / WAVES : 0;
  int pages = load_pages(0), pages_next = load_pages(STEPS);

  // Q: rows r, 16 + r, .. of the tile; the pieces of d that this quad meets
  int pos[R];  // position of each row
  bool row_ok[R];
  uint32_t q[R][NCH][X::q_regs];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int row = row0 + 16 * t + r;
    row_ok[t] = row < rows;
    const int tok = (row_ok[t] ? row : 0) / A.G, head = kvh * A.G + (row_ok[t] ? row : 0) % A.G;
    pos[t] = first + tok;
    const int64_t at = (int64_t)(s.q0 + tok) * A.ldq_t + (int64_t)head * A.ldq_h;
    constexpr int NW = X::q_regs / 4;  // 16-byte pieces of Q that go with one of K
    constexpr int E = F32 ? 4 : 8;     // values in each
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int d = (4 * c + quad) * C + w * E;
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (row_ok[t] && d < D) {
          const char* p = static_cast<const char*>(A.q) + (at + d) * (F32 ? 4 : 2);
          if (A.q_vec) {
            v = load_u32x4(p);
          } else if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = reinterpret_cast<const uint16_t*>(p)[2 * j] |
                     (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * j + 1] << 16;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) q[t][c][4 * w + j] = v[j];
      }
  }

  f32x4_t o[R][NB];
  float m[R], l[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
#pragma unroll
    for (int n = 0; n < NB; ++n) o[t][n] = f32x4_t{};
    m[t] = -INFINITY;
    l[t] = 0.f;
  }

  // Groups that this lane loads from: of K as row r of a tile, of V as quad. Token of the lane's
  // row i of tile x: 16 * group + tok0 + step(x) + i.
  const int kg = BYTES == 1 ? r >> 2 : r >> 3, vg = BYTES == 1 ? quad : quad >> 1;
  const int k_tok = BYTES == 1 ? r & 3 : 4 * ((r >> 2) & 1) + (r & 3);
  const int v_half = BYTES == 1 ? 0 : quad & 1;
  auto tile_tok = [](int x) { return BYTES == 1 ? 8 * (x & 1) + 4 * (x >> 1) : 8 * x; };
  // [pages][H][page size] index of a group's first token
  auto group_at = [&](int p, int i, int g) {
    const int t = t_begin + TOK * (wv + WAVES * i) + 16 * g;
    return ((int64_t)max(p, 0) * K.H + kvh) * ps + (t & (ps - 1));
  };

  u32x4_t kr[NT][NCH], vr[NB][VL];
  // scales of the 16 tokens of this quad's group, lane r that of place r
  float ks = 0.f, vs = 0.f;
  (void)ks; (void)vs;
  const int place_tok = tile_tok(r >> 2) + (r & 3);
  bool missing;  // of the step whose K is loaded: some group is not there
  int vpage;     // and the page of this lane's group of V
  auto load_k = [&](int i) {
    const int idx = (i & (STEPS - 1)) * NG;
    const int p = __shfl(pages, idx + kg);
    vpage = __shfl(pages, idx + vg);
    missing = __any(p < 0);
    if constexpr (SCALED) ks = K.k_scale[group_at(vpage, i, vg) + place_tok];
    const char* base = static_cast<const char*>(K.k) + group_at(p, i, kg) * D * BYTES + k_tok * 16;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        int piece = 4 * c + quad;
        const bool whole = EXACT && DP / C % 4 == 0;
        if (!whole) piece = min(piece, D / C - 1);
        kr[x][c] = load_u32x4(base + piece * 256 + tile_tok(x) * 16);
        if (!whole && 4 * c + quad >= D / C) kr[x][c] = u32x4_t{0u, 0u, 0u, 0u};
      }
  };
  auto load_v = [&](int i) {
    const int64_t g = group_at(vpage, i, vg);
    if constexpr (SCALED) vs = K.v_scale[g + place_tok];
    const char* base = static_cast<const char*>(K.v) + (g * D + r * 16 + 8 * v_half) * BYTES;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < VL; ++e)
        if (EXACT || 16 * n < D) vr[n][e] = load_u32x4(base + n * 256 * BYTES + 16 * e);
  };

  int nan_first = mine, nan_last = -1;  // steps whose NaN, of codes or of scales, is written at the end
  bool nan_codes = false;  // codes among them
  (void)nan_first; (void)nan_last; (void)nan_codes;
  if constexpr (FMT == SGMV_KV_E4M3 && !EXACT) {  // past D
#pragma unroll
    for (int n = 0; n < NB; ++n) vr[n][0] = u32x4_t{0u, 0u, 0u, 0u};
  }
  if (mine > 0) {
    load_k(0);
    if (!LATE_V) load_v(0);
  }
  for (int i = 0; i < mine; ++i) {
    const int t0 = t_begin + TOK * (wv + WAVES * i);
    const bool gap = missing;
    const int page = vpage;  // of this lane's tokens

    f32x4_t sc[R][NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int t = 0; t < R; ++t) sc[t][x] = f32x4_t{};
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        if (EXACT || 4 * c * C < D) {
          const auto k = X::operand(kr[x][c]);
#pragma unroll
          for (int t = 0; t < R; ++t) sc[t][x] = X::qk(k, q[t][c], sc[t][x]);
        }
    }
    if constexpr (SCALED)
      for_places([&](auto at) {
        const float f = row_lane<at.value>(ks);
#pragma unroll
        for (int t = 0; t < R; ++t) sc[t][at.value / 4][at.value % 4] *= f;
      });
    if (LATE_V) load_v(i);
    auto load_next = [&] {
      if (((i + 1) & (STEPS - 1)) == 0) {
        pages = pages_next;
        pages_next = load_pages(i + 1 + STEPS);
      }
      load_k(i + 1);
    };
    if (!LATE_V && i + 1 < mine) load_next();

    // a step that some row sees only part of, or with tokens that are not there
    const bool edge = t0 + TOK - 1 > lo_pos || (A.window && t0 <= hi_pos - A.window) || gap;
    const int t_lane = t0 + 16 * vg + 4 * v_half;  // this lane's first token
    bool nan = false;
    (void)nan;
    if (edge) {
      // A V scale that is not finite meets only probabilities that are not 0, of rows that see its token. Rows that
      // see it with a probability too small for fp32 get its NaN at the end. (Whether the token is there is asked
      // then: here, that took three registers, and 5 us of 138 for 64 sequences' drafts, int8.)
      if constexpr (SCALED) nan = __any(!(fabsf(vs) < INFINITY));
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = t_lane + tile_tok(x) + j;
          const bool has = at < s.kv_len && page >= 0;
#pragma unroll
          for (int t = 0; t < R; ++t)
            if (!has || at > pos[t] || (A.window && at <= pos[t] - A.window)) sc[t][x][j] = -INFINITY;
        }
    }

    u32x4_t pb[R][NT / 2];  // probabilities in bf16, or in fp32
    float pf[R][NT][4];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float top = sc[t][0][0];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, sc[t][x][j]);
      top *= A.scale_log2;
      // a stale maximum is as good as long as nothing grows past 2^8
      if (__any(top > m[t] + 8.f)) {
        const float now = fmaxf(m[t], quad_max(top));
        const float f = m[t] == now ? 1.f : exp2f(m[t] - now);  // 0 from -inf on
        m[t] = now;
        l[t] *= f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[t][n][j] *= f;
      }
      const float base = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          pf[t][x][j] = __builtin_amdgcn_exp2f(fmaf(sc[t][x][j], A.scale_log2, -base));
          l[t] += pf[t][x][j];
        }
    }
    if constexpr (SCALED)
      for_places([&](auto at) {
        const float f = row_lane<at.value>(vs);
#pragma unroll
        for (int t = 0; t < R; ++t) {
          float& p = pf[t][at.value / 4][at.value % 4];
          p = edge && p == 0.f ? 0.f : p * f;
        }
      });
    if constexpr (!F32) {
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < 2; ++j) pb[t][x / 2][2 * (x & 1) + j] = pack_bf16x2(pf[t][x][2 * j], pf[t][x][2 * j + 1]);
    }

    if (edge) {
      uint32_t there = 0;  // this lane's places whose token exists
      const int n_there = page >= 0 ? min(max(s.kv_len - (t0 + 16 * vg), 0), 16) : 0;
      there = places_below(n_there) >> (8 * v_half);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < VL; ++e) {
          vr[n][e] = keep_elements<BYTES>(vr[n][e], there >> (4 * e));
          // An e4m3 code of NaN is left out as the V values below are, but its NaN waits until the end: next to
          // codes and operands, that loop took 66 registers more.
          if constexpr (FMT == SGMV_KV_E4M3) {
            nan_codes |= __any(nan_code_any(vr[n][e]) != 0u);
            vr[n][e] = drop_nonfinite<1>(vr[n][e]);
          }
        }
      if constexpr (SCALED) {
        nan |= nan_codes;
        nan_first = nan ? min(nan_first, i) : nan_first;
        nan_last = nan ? i : nan_last;
      }
      if constexpr (!SCALED) {
        // A V value that is not finite, in a step that some rows see only part of: in the product,
        // 0 * inf would spoil the rows that do not see it. It is left out of the product and added
        // to the rows that see it, token by token.
        bool odd = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < VL; ++e)
            if (EXACT || 16 * n < D) odd |= has_nonfinite<BYTES>(vr[n][e]);
        if (__any(odd)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < VL; ++e) vr[n][e] = drop_nonfinite<BYTES>(vr[n][e]);
#pragma unroll 1
          for (int x = 0; x < TOK; ++x) {
            const int at_t = t0 + x;
            const int p = kv_page(K, table, at_t);
            if (p < 0) continue;
            const int64_t at = ((((int64_t)p * K.H + kvh) * ps + ((at_t & (ps - 1)) & ~15)) * D) +
                               8 * ((x >> 2) & 1) + 4 * ((x >> 3) & 1) + (x & 3);
#pragma unroll 1
            for (int n = 0; n < D / 16; ++n) {
              float f[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int64_t e = at + (16 * n + 4 * quad + j) * 16;
                f[j] = F32 ? static_cast<const float*>(K.v)[e] : bf16_bits_to_f32(static_cast<const uint16_t*>(K.v)[e]);
              }
#pragma unroll
              for (int t = 0; t < R; ++t)
                if (at_t <= pos[t] && !(A.window && at_t <= pos[t] - A.window)) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (!(fabsf(f[j]) < INFINITY)) {
#pragma unroll
                      for (int k = 0; k < NB; ++k)
                        if (k == n) o[t][k][j] += f[j];
                    }
                }
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!EXACT && 16 * n >= D) continue;
#pragma unroll
      for (int e = 0; e < VL; ++e) {
        const auto v = X::operand(vr[n][e]);
#pragma unroll
        for (int t = 0; t < R; ++t) {
          if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < C; ++j)
              o[t][n] = mfma_16x16x4_f32(v.f[j], pf[t][BYTES == 1 ? j / 4 : e][j % 4], o[t][n]);
          } else {
#pragma unroll
            for (int h = 0; h < C / 8; ++h) o[t][n] = mfma_16x16x32_bf16(as_bf16x8(v.h[h]), as_bf16x8(pb[t][h]), o[t][n]);
          }
        }
      }
    }
    if (i + 1 < mine) {
      if (LATE_V) load_next();
      else load_v(i + 1);
    }
  }

  // The waves' sums. A wave that saw nothing has m = -inf, l = 0, o = 0 (or NaN where all it saw
  // was NaN, which has to stay).
#pragma unroll
  for (int t = 0; t < R; ++t) {
    l[t] = quad_sum(l[t]);
    if (quad == 0) {
      s_m[wv][16 * t + r] = m[t];
      s_l[wv][16 * t + r] = l[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < R; ++t) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, s_m[w][16 * t + r]);
    const float f = m[t] == -INFINITY ? 1.f : exp2f(m[t] - top);
#pragma unroll
    for (int n = 0; n < NB; ++n)
      if (EXACT || 16 * n < D)
        *reinterpret_cast<f32x4_t*>(&s_o[wv][(16 * t + r) * LD + 16 * n + 4 * quad]) =
            f32x4_t{o[t][n][0] * f, o[t][n][1] * f, o[t][n][2] * f, o[t][n][3] * f};
  }
  if constexpr (SCALED) {  // the NaN of codes and scales, to the rows that see them
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));  // (lane numbers of its own: shared ones cost the steps a register)
    const int r2 = thread & 15, quad2 = thread >> 4 & 3;
#pragma unroll 1
    for (int i = nan_first * NG; i < (nan_last + 1) * NG; ++i) {
      const int g0 = t_begin + TOK * (wv + WAVES * (i / NG)) + 16 * (i % NG), p = kv_page(K, table, g0);
      if (p < 0) continue;
      const int64_t group = ((int64_t)p * K.H + kvh) * ps + (g0 & (ps - 1));
      const uint32_t odd = places_of_nan(K.v_scale + group);
      uint32_t seen[R], some = 0;
#pragma unroll
      for (int t = 0; t < R; ++t) some |= odd & (seen[t] = places_seen(A, pos[t], g0));
      if (!nan_codes && !__any(some != 0u)) continue;
      const char* v = static_cast<const char*>(K.v) + group * D;
#pragma unroll 1
      for (int e = 0; e < D / 4; ++e) {
        const int d = 16 * (e >> 2) + 4 * quad2 + (e & 3);  // one that this lane has stored
#pragma unroll
        for (int t = 0; t < R; ++t) {
          bool nan = (seen[t] & odd) != 0u;
          if constexpr (FMT == SGMV_KV_E4M3) nan |= nan_among(load_u32x4(v + 16 * d), place_flags(seen[t]));
          if (nan) s_o[wv][(16 * t + r2) * LD + d] = NAN;
        }
      }
    }
  }
  __syncthreads();
  const int tile_rows = min(ROWS, rows - row0);
  const int per_row = D / 4;
  for (int e = threadIdx.x; e < tile_rows * per_row; e += WAVES * WAVE) {
    const int lr = e / per_row, d = 4 * (e - lr * per_row);
    f32x4_t sum_o = {0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      top = fmaxf(top, s_m[w][lr]);
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&s_o[w][lr * LD + d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum_o[j] += v[j];
    }
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float mw = s_m[w][lr];
      sum += mw == -INFINITY ? s_l[w][lr] : s_l[w][lr] * exp2f(mw - top);
    }
    const int tok = (row0 + lr) / A.G, head = kvh * A.G + (row0 + lr) % A.G;
    const int64_t at = (int64_t)(s.q0 + tok) * A.Hq + head;
    if (used > 1) {
      const int64_t place = split * A.part_rows[0] + part_row(A, 0, slot, kvh, lr, at);
      if (d == 0) {
        A.part_ml[0][2 * place] = top;
        A.part_ml[0][2 * place + 1] = sum;
      }
      *reinterpret_cast<f32x4_t*>(A.part_o[0] + place * D + d) = sum_o;
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (A.lse && d == 0) A.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
      store_out<F32>(A, (int64_t)(s.q0 + tok) * A.ldo_t + (int64_t)head * A.ldo_h + d, sum_o[0] * inv,
                     sum_o[1] * inv, sum_o[2] * inv, sum_o[3] * inv);
    }
  }
}

template <bool F32, int FMT, int DP, bool EXACT, int R, int WAVES>
__global__ __launch_bounds__(WAVES* WAVE, direct_occupancy(F32, DP, R)) void attn_direct_kernel(AttnArgs A) {
  __shared__ DirectShared<DP, R, WAVES> sh;
  attn_direct<F32, FMT, DP, EXACT, R, WAVES>(A, blockIdx.x, sh);
}

template <bool F32, int FMT, int DP, bool EXACT, int R, int WAVES>
hipError_t launch_direct(const AttnArgs& A, hipStream_t stream) {
  const dim3 g((unsigned)A.slots[0] * (unsigned)A.n_split[0] * (unsigned)A.kv.H);
  attn_direct_kernel<F32, FMT, DP, EXACT, R, WAVES><<<g, WAVES * WAVE, 0, stream>>>(A);
  return hipGetLastError();
}

template <bool F32, int FMT, int DP, bool EXACT, int R>
hipError_t launch_direct_waves(const AttnArgs& A, hipStream_t stream) {
  if constexpr (direct_eight_waves(DP, F32)) {
    if (A.direct_waves == 8) return launch_direct<F32, FMT, DP, EXACT, R, 8>(A, stream);
  }
  return launch_direct<F32, FMT, DP, EXACT, R, 4>(A, stream);
}

// Two tiles of rows per workgroup where their registers fit (direct_two_tiles).
template <int FMT, int R>
hipError_t launch_direct_dim(const AttnArgs& A, hipStream_t stream) {
  const int D = A.kv.D;
  if (D == 64) return launch_direct_waves<false, FMT, 64, true, R>(A, stream);
  if (D == 80) return launch_direct_waves<false, FMT, 80, true, R>(A, stream);
  if (D == 96) return launch_direct_waves<false, FMT, 96, true, R>(A, stream);
  if (D == 128) return launch_direct_waves<false, FMT, 128, true, R>(A, stream);
  if (D == 192) return launch_direct_waves<false, FMT, 192, true, R>(A, stream);
  if (D < 64) return launch_direct_waves<false, FMT, 64, false, R>(A, stream);
  if (D < 128) return launch_direct_waves<false, FMT, 128, false, R>(A, stream);
  if constexpr (R == 1) {
    if (D == 256) return launch_direct_waves<false, FMT, 256, true, 1>(A, stream);
    return launch_direct_waves<false, FMT, 256, false, 1>(A, stream);
  }
  return hipErrorInvalidValue;
}

template <int FMT>
hipError_t launch_direct_bf16(const AttnArgs& A, hipStream_t stream) {
  return A.direct_tile == 16 ? launch_direct_dim<FMT, 1>(A, stream)
                             : launch_direct_dim<FMT, 2>(A, stream);
}

}  // namespace sgmv
