// Attention of many rows (a prompt's chunk) over the paged cache: keys and values staged in LDS
// as bf16 and shared by the workgroup's waves.
//
// A workgroup takes WAVES * 32 rows (new token, query head of the group) of one (sequence, key/value
// head); each wave keeps 32 rows' queries and outputs in registers. Per tile of 64 tokens a wave has a
// phase of matrix products (O^T += V^T P^T of this tile, S^T = K Q^T of the next; between them the pieces
// that it loaded are converted and written to LDS, and the next ones' loads issued) and one of the softmax
// step. Scores and probabilities stay in registers as in attn_direct.h. Eight waves are two per SIMD, in
// two groups half a tile apart: a barrier ends each phase, so that one wave of a SIMD has the matrix cores
// while the other one computes exponentials. LDS holds the operands in the order the products read them: K
// as stored, V with its 16-byte halves of 8 tokens exchanged in every second 8 values of d, so that 16
// lanes read 16 different bank groups.
//
// Group 0 multiplies by V(i) and K(i + 1) in phase 2 i + 2, group 1 in phase 2 i + 3, and both then write
// their shares of K(i + 2) and V(i + 1): over K(i) and V(i - 1), last read in phase 2 i + 1, and in time for
// phase 2 i + 4, so two buffers of each are enough. The scales of tile i are read in phases 2 i + 1 and 2 i + 2
// of it; group 1 writes them.
//
// Bound: the matrix cores, at the clock that they leave themselves: the products alone, without loads,
// softmax and LDS reads, ran at 1420..1520 TFLOP/s on the largest shape here (a large matrix product of the
// library: 1250). 2048 tokens over 14001, e4m3, 32 / 8 heads of 128: 477..507 us (990..1050 TFLOP/s), matrix
// cores busy 48% of the cycles, a phase of products 1.5 thousand cycles where they need 1.0; eight prompts'
// chunks, bf16, 64 / 8 heads: 335..350 us (870..910): there the order of the tiles counts too, 2 us each, the last
// of the last sequence first. Handed to 256 compute units so, the 1192 of that shape end after 176 tiles, the
// longest first would after 153 (no order before 150). What did not pay: 64 rows per wave with the softmax
// between the products of one wave (registers: 954 us), e4m3 codes of V or of both in LDS, converted at
// each use (531 and 589 us beside 512), longer read-ahead, no or other wave priorities (533, 566).
#pragma once

#include "attn_direct.h"

namespace sgmv {

constexpr int TL_TOKENS = 64;

// All bits set where bit `at` of w is.
__device__ __forceinline__ uint32_t bit_mask(uint32_t w, int at) { return (uint32_t)((int32_t)(w << (31 - at)) >> 31); }

// Schedule of N products whose left operands come from LDS: four loads ahead.
template <int N>
__device__ __forceinline__ void read_ahead() {
  constexpr int MFMA = 0x008, DS_READ = 0x100;
  __builtin_amdgcn_sched_group_barrier(DS_READ, 4, 0);
#pragma unroll
  for (int i = 0; i < N / 2 - 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(MFMA, 2, 0);
    __builtin_amdgcn_sched_group_barrier(DS_READ, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(MFMA, 4, 0);
}

template <int FMT, int D> struct TiledShared {
  static constexpr int GROUP = D * 16;  // elements of a group
  alignas(16) uint16_t k[2][4 * GROUP], v[2][4 * GROUP];
  alignas(16) float ks[2][KvFormat<FMT>::scaled ? TL_TOKENS : 4], vs[2][KvFormat<FMT>::scaled ? TL_TOKENS : 4];
  int odd[4];  // [i % 4] = i: something that is not finite was left out of tile i
  int nan_first, nan_last;  // tiles from which e4m3 codes of NaN were left out
};

// One workgroup's piece.
template <int FMT, int D>
__device__ __forceinline__ void attn_tiled(const AttnArgs& A, int piece, TiledShared<FMT, D>& sh) {
  constexpr int WAVES = tiled_waves(D), THREADS = WAVES * WAVE, ROWS = WAVES * AT_ROWS;
  constexpr int BYTES = KvFormat<FMT>::bytes;
  constexpr bool SCALED = KvFormat<FMT>::scaled;
  constexpr int NK = D / 16, NB = (D + 31) / 32;
  constexpr int SCALE_WAVE = WAVES == 8 ? 4 : 0;  // the first of two waves that stage scales
  constexpr int GROUP = D * 16;                   // elements of a group
  constexpr int PIECES = GROUP * BYTES / 16;      // 16-byte pieces of a group as stored
  constexpr int NP = (4 * PIECES + THREADS - 1) / THREADS;
  constexpr bool BY_WAVE = PIECES % WAVE == 0;    // pieces of one group belong to whole waves
  auto& s_k = sh.k;
  auto& s_v = sh.v;
  auto& s_ks = sh.ks;
  auto& s_vs = sh.vs;
  auto& s_odd = sh.odd;

  const KvArgs& K = A.kv;
  const int tid = threadIdx.x, lane = tid & (WAVE - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int col = lane & 31, half = lane >> 5;

  // this workgroup's piece; the last tiles of a sequence look at the most tokens and start first
  const int kvh = piece % K.H;
  const int rest = A.slots[1] * A.n_split[1] - 1 - piece / K.H;
  const int split = rest % A.n_split[1], slot = rest / A.n_split[1];
  const auto first_slot = [&](int i) {
    return (int)((int64_t)min(max(K.q_start[i], 0), K.T) * A.G / ROWS) + i;
  };
  const int b = __builtin_amdgcn_readfirstlane(wave_find(K.B, slot, first_slot));
  const int tile0 = (slot - first_slot(b)) * ROWS;
  const KvSeq s = kv_seq(K, b);
  const int rows = s.q_len * A.G;
  if (tile0 < 0 || tile0 >= rows || rows <= A.direct_rows) return;
  const Span span = row_span(A, s, tile0, ROWS);
  const int used = span_splits(A, span, 1);
  if (split >= used) return;
  const int t_begin = span.begin + split * A.chunk[1];
  const int t_end = split == used - 1 ? span.end : t_begin + A.chunk[1];

  const int row0 = tile0 + wv * AT_ROWS, row = row0 + col;
  const bool row_ok = row < rows;
  const int tok = (row_ok ? row : 0) / A.G, head = kvh * A.G + (row_ok ? row : 0) % A.G;
  u32x4_t q[NK];
  {
    const int64_t at = (int64_t)(s.q0 + tok) * A.ldq_t + (int64_t)head * A.ldq_h;
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (row_ok) {
        const uint16_t* p = static_cast<const uint16_t*>(A.q) + at + 16 * c + 8 * half;
        if (A.q_vec) {
          v = load_u32x4(p);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = p[2 * j] | (uint32_t)p[2 * j + 1] << 16;
        }
      }
      q[c] = v;
    }
  }
  const int first = s.kv_len - s.q_len;
  const int pos = first + tok;
  const int lo_pos = first + min(row0, rows - 1) / A.G;
  const int hi_pos = first + (min(row0 + AT_ROWS, rows) - 1) / A.G;
  const int tile_lo = first + tile0 / A.G;  // of the whole workgroup
  const int tile_hi = first + (min(tile0 + ROWS, rows) - 1) / A.G;
  const int ps = 1 << K.lps;
  const int32_t* table = K.table + (int64_t)b * K.ldp;

  const int n_tiles = max((t_end - t_begin + TL_TOKENS - 1) / TL_TOKENS, 0);

  f32x16_t o[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i] = f32x16_t{};
  float m = -INFINITY, l = 0.f;

  // pages of the groups of 16 tiles, one per lane, and of the next 16; which exist (also of the 16 before)
  auto load_pages = [&](int i0) {
    const int t = t_begin + TL_TOKENS * i0 + 16 * lane;
    return t < t_end ? kv_page(K, table, t) : -1;
  };
  int pages = load_pages(0), pages_next = load_pages(16), block = 0;
  uint64_t have = __ballot(pages >= 0), have_before = 0;
  auto groups_of = [&](int i) { return (uint32_t)((i >> 4 == block ? have : have_before) >> ((4 * i) & 63)) & 15u; };

  // The pieces that this thread stages, in registers for K of a tile and V of the tile before. (Past the
  // last tile, of page 0, unused.)
  u32x4_t rk[NP], rv[NP];
  int64_t at_k[NP] = {}, at_v[NP];  // bytes before the groups that they are from
  const int64_t page_bytes = (int64_t)K.H * ps * D * BYTES, head_bytes = (int64_t)kvh * ps * D * BYTES;
  float rs = 0.f;
  (void)rs;
  auto group_of = [&](int n) { return (n * THREADS + (BY_WAVE ? wv * WAVE : tid)) / PIECES; };
  auto piece_of = [&](int n) { return BY_WAVE ? (n * THREADS + wv * WAVE) % PIECES + lane : (n * THREADS + tid) % PIECES; };
  auto load_tile = [&](int i) {  // K of tile i, V of tile i - 1
    const int t0 = t_begin + TL_TOKENS * i;
    if ((i & 15) == 0 && i > 0) {
      pages = pages_next;
      pages_next = load_pages(i + 16);
      have_before = have;
      have = __ballot(pages >= 0);
      block = i >> 4;
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int g = group_of(n), piece = piece_of(n);
      const int from = (4 * i + g) & 63;
      const int page = BY_WAVE ? __builtin_amdgcn_readlane(pages, from) : __shfl(pages, from);
      if (4 * PIECES % THREADS == 0 || g < 4) {
        const int off = piece * 16;
        int voff = off;
        if constexpr (!SCALED) {  // the exchange of halves
          const int d = piece >> 1;
          voff = d * 32 + ((piece ^ (d >> 3)) & 1) * 16;
        }
        at_v[n] = at_k[n];
        at_k[n] = max(page, 0) * page_bytes + head_bytes +
                  ((t0 + 16 * g) & (ps - 1)) * (D * BYTES);
        rk[n] = load_u32x4(static_cast<const char*>(K.k) + at_k[n] + off);
        rv[n] = load_u32x4(static_cast<const char*>(K.v) + at_v[n] + voff);
      }
    }
    if constexpr (SCALED) {
      if (wv >> 1 == SCALE_WAVE >> 1) {  // one wave the K scales, one the V scales of the tile of K
        const int p = max(__shfl(pages, (4 * i + (lane >> 4)) & 63), 0);
        const int64_t at = ((int64_t)p * K.H + kvh) * ps + ((t0 + lane) & (ps - 1));
        rs = (wv & 1 ? K.v_scale : K.k_scale)[at];
      }
    }
  };
  // whether some row of the workgroup sees only part of a tile
  auto some_see_part = [&](int i) {
    const int t0 = t_begin + TL_TOKENS * i;
    return t0 + TL_TOKENS - 1 > tile_lo || (A.window && t0 <= tile_hi - A.window) || groups_of(i) != 15u;
  };
  auto store_k = [&](int i) {
    const int buf = i & 1;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int g = group_of(n), piece = piece_of(n);
      if (4 * PIECES % THREADS == 0 || g < 4) {
        if constexpr (!SCALED) {
          *reinterpret_cast<u32x4_t*>(&s_k[buf][g * GROUP + piece * 8]) = rk[n];
        } else {
          // piece: token piece % 16, values 16 (piece / 16) .. + 15: two octets of d
          uint16_t* k = &s_k[buf][g * GROUP + (piece >> 4) * 256 + (piece & 15) * 8];
          *reinterpret_cast<u32x4_t*>(k) = codes8_bf16<FMT>(u32x2_t{rk[n].x, rk[n].y});
          *reinterpret_cast<u32x4_t*>(k + 128) = codes8_bf16<FMT>(u32x2_t{rk[n].z, rk[n].w});
        }
      }
    }
  };
  // A V scale that is not finite is left out as such a V value is (store_v).
  auto store_scales = [&](int i) {
    if constexpr (SCALED) {
      if (wv >> 1 == SCALE_WAVE >> 1) {
        if (wv & 1) {
          if (!(fabsf(rs) < INFINITY)) {
            s_odd[i & 3] = i;
            rs = 0.f;
          }
        } else {
          rs *= A.scale_log2;
        }
        (wv & 1 ? s_vs : s_ks)[i & 1][lane] = rs;
      }
    }
  };
  // V of tokens that are not there has to be finite, so that their probability 0 counts as such: e4m3 codes of
  // NaN become finite ones, and their tiles are noted for spoil(). (With a test of the codes alone in the way
  // of those that have none, 501 us for the largest shape above; with the change made to every code, 507.) Where
  // some rows of the workgroup see only part of the tile, bf16 values that are not finite are left out, for
  // 0 * inf would spoil the rows that do not see them, and the tile is marked for restore().
  int nan_first = n_tiles, nan_last = -1;  // (of this wave's pieces)
  (void)nan_first; (void)nan_last;
  auto store_v = [&](int i) {
    const int buf = i & 1;
    const bool some = !SCALED && some_see_part(i);
    if constexpr (FMT == SGMV_KV_E4M3) {
      uint32_t nan_codes = 0;
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (4 * PIECES % THREADS == 0 || group_of(n) < 4) nan_codes |= nan_code_any(rv[n]);
      if (__any(nan_codes != 0u)) {
        nan_first = min(nan_first, i);
        nan_last = i;
#pragma unroll
        for (int n = 0; n < NP; ++n) rv[n] = drop_nonfinite<1>(rv[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int g = group_of(n), piece = piece_of(n);
      if (4 * PIECES % THREADS == 0 || g < 4) {
        if constexpr (!SCALED) {
          if (some && has_nonfinite<2>(rv[n])) {
            s_odd[i & 3] = i;
            rv[n] = drop_nonfinite<2>(rv[n]);
          }
          *reinterpret_cast<u32x4_t*>(&s_v[buf][g * GROUP + piece * 8]) = rv[n];
        } else {
          // both halves of d = piece
          uint16_t* v = &s_v[buf][g * GROUP + piece * 16];
          const int x = (piece >> 3) & 1;
          *reinterpret_cast<u32x4_t*>(v + 8 * x) = codes8_bf16<FMT>(u32x2_t{rv[n].x, rv[n].y});
          *reinterpret_cast<u32x4_t*>(v + 8 * (1 - x)) = codes8_bf16<FMT>(u32x2_t{rv[n].z, rv[n].w});
        }
      }
    }
  };

  // whether some of this wave's rows see only part of a tile
  auto partly = [&](int i) {
    const int t0 = t_begin + TL_TOKENS * i;
    return t0 + TL_TOKENS - 1 > lo_pos || (A.window && t0 <= hi_pos - A.window) || groups_of(i) != 15u;
  };

  // tokens of tile i that this lane's row sees: bit reg_token(j, 0) of mask[u] for register j of product u
  auto visible = [&](int i, uint32_t (&mask)[2]) {
    const int t0 = t_begin + TL_TOKENS * i, n = pos - t0 + 1;
    const uint32_t groups = groups_of(i);
    uint64_t seen = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
    if (A.window) {
      const int gone = n - A.window;
      seen &= gone >= 64 ? 0ull : gone <= 0 ? ~0ull : ~((1ull << gone) - 1ull);
    }
    uint64_t there = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) there |= (groups >> g & 1 ? 0xffffull : 0ull) << (16 * g);
    seen = (seen & there) >> (4 * half);
    mask[0] = (uint32_t)seen;
    mask[1] = (uint32_t)(seen >> 32);
  };

  f32x16_t sc[2];
  u32x4_t pb[4];  // probabilities, per group
  // O^T += V^T P^T of tile i
  auto values = [&](int i) {
    const int buf = i & 1;
    // V operand of block n and group g: d = 32 n + col (D - 1 where there is no such d: its results are
    // not used), this half's 8 tokens
    const uint16_t* vb = &s_v[buf][col * 16 + ((half ^ (col >> 3)) & 1) * 8];
    const int last = min(32 * (NB - 1) + col, D - 1);
    const uint16_t* vl = &s_v[buf][last * 16 + ((half ^ (last >> 3)) & 1) * 8];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        o[n] = mfma_32x32_bf16(load_u32x4(D % 32 && n == NB - 1 ? vl + g * GROUP : vb + g * GROUP + n * 512), pb[g], o[n]);
    read_ahead<4 * NB>();
  };
  // What store_v (of 8-bit formats store_scales) has left out of tile i, added to the rows that see it, token by
  // token.
  auto restore = [&](int i) {
#pragma unroll 1
    for (int t = t_begin + TL_TOKENS * i, end = min(t + TL_TOKENS, s.kv_len); t < end; ++t) {
      const int p = kv_page(K, table, t);
      if (p < 0) continue;
      const bool seen = t <= pos && !(A.window && t <= pos - A.window);
      if constexpr (SCALED) {
        const float f = K.v_scale[((int64_t)p * K.H + kvh) * ps + (t & (ps - 1))];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[n][j] += seen && !(fabsf(f) < INFINITY) ? NAN : 0.f;
        continue;
      }
      const int place = 8 * ((t >> 2) & 1) + 4 * ((t >> 3) & 1) + (t & 3);
      const uint16_t* v = static_cast<const uint16_t*>(K.v) +
                          (((int64_t)p * K.H + kvh) * ps + (t & (ps - 1) & ~15)) * D + place + 64 * half;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (32 * n + reg_token(j, 0) >= D) continue;
          const float f = bf16_bits_to_f32(v[(32 * n + reg_token(j, 0)) * 16]);
          o[n][j] += seen && !(fabsf(f) < INFINITY) ? f : 0.f;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // S^T = K Q^T of tile i
  auto scores = [&](int i) {
    const uint16_t* kb = &s_k[i & 1][(lane >> 4 & 1) * GROUP + half * 128 + (lane & 15) * 8];
#pragma unroll
    for (int u = 0; u < 2; ++u) sc[u] = f32x16_t{};
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        sc[u] = mfma_32x32_bf16(load_u32x4(kb + u * 2 * GROUP + c * 256), q[c], sc[u]);
    read_ahead<2 * NK>();
  };
  auto softmax = [&](int i) {
    const int buf = i & 1;
    // exponents with the old maximum: wherever they stay below 8, it is as good as the new one
    float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4_t f = {A.scale_log2, A.scale_log2, A.scale_log2, A.scale_log2};
        if constexpr (SCALED) f = *reinterpret_cast<const f32x4_t*>(&s_ks[buf][32 * u + 8 * j + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][4 * j + e] = fmaf(sc[u][4 * j + e], f[e], -base);
      }
    if (partly(i)) {  // a row's own position is below kv_len
      uint32_t mask[2];
      visible(i, mask);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t on = bit_mask(mask[u], reg_token(j, 0));
          sc[u][j] = __uint_as_float((__float_as_uint(sc[u][j]) & on) | (0xff800000u & ~on));
        }
    }
    float top = sc[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, sc[u][j]);
    if (__any(top > (m == -INFINITY ? -INFINITY : 8.f))) {
      const float up = half_max(top), now = fmaxf(m, base + up);
      const float f = m == now ? 1.f : exp2f(m - now);  // 0 from -inf on
      const float step = now == -INFINITY ? 0.f : now - base;
      m = now;
      l *= f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[n][j] *= f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) sc[u][j] -= step;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float p[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        p[j] = __builtin_amdgcn_exp2f(sc[u][j]);
        l += p[j];
      }
      if constexpr (SCALED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4_t f = *reinterpret_cast<const f32x4_t*>(&s_vs[buf][32 * u + 8 * j + 4 * half]);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[4 * j + e] *= f[e];
        }
      }
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) pb[2 * u + g][j] = pack_bf16x2(p[8 * g + 2 * j], p[8 * g + 2 * j + 1]);
    }
  };

  const int group = WAVES == 8 ? wv >> 2 : 0;
  if (tid < 4) s_odd[tid] = -1;
  if (tid == 0) {
    sh.nan_first = n_tiles;
    sh.nan_last = -1;
  }
  if (n_tiles > 0) {
    load_tile(0);
    __syncthreads();  // s_odd
    store_k(0);
    store_scales(0);
    load_tile(1);
    store_k(1);
    store_scales(1);
    store_v(0);
    load_tile(2);
    __syncthreads();
    if (group) __syncthreads();
    scores(0);
    for (int i = 0; i < n_tiles; ++i) {
      __builtin_amdgcn_s_setprio(0);
      __syncthreads();
      if (i > 0 && __builtin_amdgcn_readfirstlane(s_odd[(i - 1) & 3]) == i - 1) restore(i - 1);
      softmax(i);
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int g = 0; g < 4; ++g) asm volatile("" : "+v"(pb[g]));
      __syncthreads();
      __builtin_amdgcn_s_setprio(1);
      values(i);
      store_k(i + 2);
      store_v(i + 1);
      scores(i + 1);  // of the last tile: of what was there, unused
      store_scales(i + 2);
      load_tile(i + 3);
    }
    if (__builtin_amdgcn_readfirstlane(s_odd[(n_tiles - 1) & 3]) == n_tiles - 1) restore(n_tiles - 1);
    __builtin_amdgcn_s_setprio(0);
    if (WAVES == 8 && !group) __syncthreads();  // as many barriers as the other group
    if constexpr (FMT == SGMV_KV_E4M3) {
      if (nan_last >= 0 && lane == 0) {
        atomicMin(&sh.nan_first, nan_first);
        atomicMax(&sh.nan_last, nan_last);
      }
      __syncthreads();
    }
  }
  if (!row_ok) return;

  // The NaN of the codes that store_v has changed, over what this lane has stored of a row that sees them.
  auto spoil = [&](auto store_nan) {
    if constexpr (FMT == SGMV_KV_E4M3) {
      if (n_tiles == 0) return;
      const int g_end = 4 * min(__builtin_amdgcn_readfirstlane(sh.nan_last) + 1, n_tiles);
#pragma unroll 1
      for (int g = 4 * __builtin_amdgcn_readfirstlane(sh.nan_first); g < g_end; ++g) {
        const int g0 = t_begin + 16 * g, p = kv_page(K, table, g0);
        if (p < 0) continue;
        const char* v = static_cast<const char*>(K.v) + p * page_bytes + head_bytes + (g0 & (ps - 1)) * D;
        const u32x4_t seen = place_flags(places_seen(A, pos, g0));
#pragma unroll 1
        for (int e = 0; e < D / 2; ++e) {
          const int d = 8 * (e >> 2) + 4 * half + (e & 3);
          if (nan_among(load_u32x4(v + 16 * d), seen)) store_nan(d);
        }
      }
    }
  };

  const float sum = half_sum(l);
  const int64_t at = (int64_t)(s.q0 + tok) * A.Hq + head;
  if (used > 1) {
    const int64_t place = split * A.part_rows[1] + part_row(A, 1, slot, kvh, row - tile0, at);
    if (half == 0) {
      A.part_ml[1][2 * place] = m;
      A.part_ml[1][2 * place + 1] = sum;
    }
    float* dst = A.part_o[1] + place * D;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * n + 8 * j < D)
          *reinterpret_cast<f32x4_t*>(dst + 32 * n + 8 * j + 4 * half) =
              f32x4_t{o[n][4 * j], o[n][4 * j + 1], o[n][4 * j + 2], o[n][4 * j + 3]};
    spoil([&](int d) { dst[d] = NAN; });
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (A.lse && half == 0)
    A.lse[at] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994531f;
  const int64_t oat = (int64_t)(s.q0 + tok) * A.ldo_t + (int64_t)head * A.ldo_h;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (32 * n + 8 * j < D)
        store_out<false>(A, oat + 32 * n + 8 * j + 4 * half, o[n][4 * j] * inv, o[n][4 * j + 1] * inv,
                       o[n][4 * j + 2] * inv, o[n][4 * j + 3] * inv);
  spoil([&](int d) { static_cast<uint16_t*>(A.out)[oat + d] = 0x7fc0; });
}

// Workgroups [0, tiled) take tiles of many rows, the others the sequences of few rows (as attn_direct.h
// does by itself): in one launch, these fill the compute units that finish their tiles early.
template <int FMT, int D>
__global__ __launch_bounds__(tiled_waves(D) * WAVE) void attn_tiled_kernel(AttnArgs A) {
  constexpr int WAVES = tiled_waves(D), R = tiled_direct_rows(D) / 16;
  __shared__ union Shared {
    TiledShared<FMT, D> tiled;
    DirectShared<D, R, WAVES> direct;
    __device__ Shared() {}
  } sh;
  const int tiled = A.slots[1] * A.n_split[1] * A.kv.H;
  if ((int)blockIdx.x < tiled) attn_tiled<FMT, D>(A, blockIdx.x, sh.tiled);
  else attn_direct<false, FMT, D, true, R, WAVES>(A, blockIdx.x - tiled, sh.direct);
}

template <int FMT, int D>
hipError_t launch_tiled(const AttnArgs& A, hipStream_t stream) {
  const dim3 g((unsigned)(A.slots[1] * A.n_split[1] + A.slots[0] * A.n_split[0]) * (unsigned)A.kv.H);
  attn_tiled_kernel<FMT, D><<<g, tiled_waves(D) * WAVE, 0, stream>>>(A);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_tiled_dim(const AttnArgs& A, hipStream_t stream) {
  switch (A.kv.D) {
    case 64: return launch_tiled<FMT, 64>(A, stream);
    case 80: return launch_tiled<FMT, 80>(A, stream);
    case 96: return launch_tiled<FMT, 96>(A, stream);
    case 128: return launch_tiled<FMT, 128>(A, stream);
    case 192: return launch_tiled<FMT, 192>(A, stream);
    case 256: return launch_tiled<FMT, 256>(A, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sgmv
