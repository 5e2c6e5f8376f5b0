// Attention of many rows (a prompt's chunk) over the paged cache: keys and values staged in LDS
// as bf16 and shared by the workgroup's waves.
//
// A workgroup takes WAVES * 32 rows (new token, query head of the group) of one (sequence, key/value
// head); each wave keeps 32 rows' queries and outputs in registers. Per 64 tokens: the next 64 are
// loaded into registers, S^T = K Q^T, the softmax step and O^T += V^T P^T run from LDS, then the
// loaded ones are converted (8-bit formats: once here instead of once per wave) and written to the other
// LDS buffer: one barrier per 64 tokens. Scores and probabilities stay in registers as in
// attn_direct.h. LDS holds the operands in the order the products read them: K as stored, V with its 16-byte
// halves of 8 tokens exchanged in every second 8 values of d, so that 16 lanes read 16 different bank groups.
#pragma once

#include "attn_operand.h"

namespace sgmv {

constexpr int TL_TOKENS = 64;

template <int FMT, int D>
__global__ __launch_bounds__(tiled_waves(D) * WAVE) void attn_tiled_kernel(AttnArgs A) {
  constexpr int WAVES = tiled_waves(D), THREADS = WAVES * WAVE, ROWS = WAVES * AT_ROWS;
  constexpr int BYTES = KvFormat<FMT>::bytes;
  constexpr bool SCALED = KvFormat<FMT>::scaled;
  constexpr int NK = D / 16, NB = D / 32;
  constexpr int GROUP = D * 16;                         // elements of a group
  constexpr int PIECES = GROUP * BYTES / 16;            // 16-byte pieces of a group as stored
  constexpr int NP = (4 * PIECES + THREADS - 1) / THREADS;
  __shared__ __align__(16) uint16_t s_k[2][4 * GROUP], s_v[2][4 * GROUP];
  __shared__ int s_odd[2];  // the last tile in each buffer with a V value that is not finite
  __shared__ __align__(16) float s_ks[2][SCALED ? TL_TOKENS : 4], s_vs[2][SCALED ? TL_TOKENS : 4];

  const KvArgs& K = A.kv;
  const int tid = threadIdx.x, lane = tid & (WAVE - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int col = lane & 31, half = lane >> 5;

  // this workgroup's piece; the last tiles of a sequence look at the most tokens and start first
  const int kvh = blockIdx.x % K.H;
  const int rest = (gridDim.x - 1 - blockIdx.x) / K.H;
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
  const bool any = row0 < rows;
  const int lo_pos = first + min(row0, rows - 1) / A.G;
  const int hi_pos = first + (min(row0 + AT_ROWS, rows) - 1) / A.G;
  const int ps = 1 << K.lps;
  const int32_t* table = K.table + (int64_t)b * K.ldp;

  f32x16_t o[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i] = f32x16_t{};
  float m = -INFINITY, l = 0.f;

  // pages of the groups of the next 16 tiles, one per lane
  int pages = -1;
  uint64_t have = 0;
  auto load_pages = [&](int i0) {
    const int t = t_begin + TL_TOKENS * i0 + 16 * lane;
    pages = t < t_end ? kv_page(K, table, t) : -1;
  };

  // the pieces that this thread stages: pieces of one group belong to whole waves
  u32x4_t rk[NP], rv[NP];
  float rs = 0.f;
  auto load_tile = [&](int i) {
    const int t0 = t_begin + TL_TOKENS * i;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int at = n * THREADS + wv * WAVE;
      const int g = at / PIECES;
      if (4 * PIECES % THREADS == 0 || g < 4) {
        const int p = max(__builtin_amdgcn_readlane(pages, (4 * i + g) & 63), 0);
        const int64_t block = (((int64_t)p * K.H + kvh) * ps + ((t0 + 16 * g) & (ps - 1))) * D * BYTES;
        const int off = (at % PIECES + lane) * 16;
        int voff = off;
        if constexpr (!SCALED) {  // the exchange of halves
          const int slot16 = at % PIECES + lane, d = slot16 >> 1;
          voff = d * 32 + ((slot16 ^ (d >> 3)) & 1) * 16;
        }
        rk[n] = load_u32x4(static_cast<const char*>(K.k) + block + off);
        rv[n] = load_u32x4(static_cast<const char*>(K.v) + block + voff);
      }
    }
    if constexpr (SCALED) {
      if (wv < 2) {  // wave 0 the K scales, wave 1 the V scales
        const int p = max(__shfl(pages, (4 * i + (lane >> 4)) & 63), 0);
        const int64_t at = ((int64_t)p * K.H + kvh) * ps + ((t0 + lane) & (ps - 1));
        rs = (wv ? K.v_scale : K.k_scale)[at];
      }
    }
  };
  // `i`: the tile that load_tile has loaded. V of tokens that are not there becomes 0, so that their
  // probability 0 counts as such; a V value that is not finite is noted.
  auto store_tile = [&](int buf, int i) {
    const int t0 = t_begin + TL_TOKENS * i;
    const uint32_t groups = (uint32_t)(have >> ((4 * i) & 63)) & 15u;
    const bool whole = groups == 15u && t0 + TL_TOKENS <= s.kv_len;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int at = n * THREADS + wv * WAVE;
      const int g = at / PIECES;
      if (4 * PIECES % THREADS == 0 || g < 4) {
        const int piece = at % PIECES + lane;
        const int there = groups >> g & 1 ? min(max(s.kv_len - t0 - 16 * g, 0), 16) : 0;  // tokens
        if constexpr (!SCALED) {
          u32x4_t v = rv[n];
          if (!whole) v = keep_elements<2>(v, places_below(there) >> (8 * ((piece ^ (piece >> 4)) & 1)));
          if (has_nonfinite<2>(v)) s_odd[buf] = i;
          *reinterpret_cast<u32x4_t*>(&s_k[buf][g * GROUP + piece * 8]) = rk[n];
          *reinterpret_cast<u32x4_t*>(&s_v[buf][g * GROUP + piece * 8]) = v;
        } else {
          if (!whole) rv[n] = keep_elements<1>(rv[n], places_below(there));
          // K piece: token piece % 16, values 16 (piece / 16) .. + 15: two octets of d
          uint16_t* k = &s_k[buf][g * GROUP + (piece >> 4) * 256 + (piece & 15) * 8];
          *reinterpret_cast<u32x4_t*>(k) = codes8_bf16<FMT>(u32x2_t{rk[n].x, rk[n].y});
          *reinterpret_cast<u32x4_t*>(k + 128) = codes8_bf16<FMT>(u32x2_t{rk[n].z, rk[n].w});
          // V piece: both halves of d = piece
          uint16_t* v = &s_v[buf][g * GROUP + piece * 16];
          const int x = (piece >> 3) & 1;
          *reinterpret_cast<u32x4_t*>(v + 8 * x) = codes8_bf16<FMT>(u32x2_t{rv[n].x, rv[n].y});
          *reinterpret_cast<u32x4_t*>(v + 8 * (1 - x)) = codes8_bf16<FMT>(u32x2_t{rv[n].z, rv[n].w});
        }
      }
    }
    if constexpr (SCALED) {
      if (wv < 2) (wv ? s_vs : s_ks)[buf][lane] = rs;
    }
  };

  const int n_tiles = max((t_end - t_begin + TL_TOKENS - 1) / TL_TOKENS, 0);
  if (tid < 2) s_odd[tid] = -1;
  __syncthreads();
  if (n_tiles > 0) {
    load_pages(0);
    have = __ballot(pages >= 0);
    load_tile(0);
    store_tile(0, 0);
  }
  __syncthreads();
  for (int i = 0; i < n_tiles; ++i) {
    const int buf = i & 1, t0 = t_begin + TL_TOKENS * i;
    const uint32_t groups = (uint32_t)(have >> ((4 * i) & 63)) & 15u;
    if (i + 1 < n_tiles) {
      if (((i + 1) & 15) == 0) {
        load_pages(i + 1);
        have = __ballot(pages >= 0);
      }
      load_tile(i + 1);
    }
    if (any && hi_pos >= t0 && !(A.window && t0 + TL_TOKENS - 1 <= lo_pos - A.window)) {
      f32x16_t sc[2] = {};
      const uint16_t* kb = &s_k[buf][(lane >> 4 & 1) * GROUP + half * 128 + (lane & 15) * 8];
#pragma unroll
      for (int c = 0; c < NK; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          sc[u] = mfma_32x32_bf16(load_u32x4(kb + u * 2 * GROUP + c * 256), q[c], sc[u]);
      if constexpr (SCALED) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4_t f = *reinterpret_cast<const f32x4_t*>(&s_ks[buf][32 * u + 8 * j + 4 * half]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[u][4 * j + e] *= f[e];
          }
      }
      const bool edge = t0 + TL_TOKENS - 1 > lo_pos || (A.window && t0 <= hi_pos - A.window) || groups != 15u;
      if (edge) {  // a row's own position is below kv_len
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = t0 + 32 * u + reg_token(j, half);
            if (!(groups >> (2 * u + (j >> 3)) & 1) || t > pos || (A.window && t <= pos - A.window))
              sc[u][j] = -INFINITY;
          }
      }
      float top = sc[0][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, sc[u][j]);
      top = half_max(top) * A.scale_log2;
      if (__any(top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float f = m == now ? 1.f : exp2f(m - now);
        m = now;
        l *= f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[n][j] *= f;
      }
      const float base = m == -INFINITY ? 0.f : m;
      u32x4_t pb[4];  // per group
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          p[j] = __builtin_amdgcn_exp2f(fmaf(sc[u][j], A.scale_log2, -base));
          l += p[j];
        }
        if constexpr (SCALED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4_t f = *reinterpret_cast<const f32x4_t*>(&s_vs[buf][32 * u + 8 * j + 4 * half]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[4 * j + e] = edge && p[4 * j + e] == 0.f ? 0.f : p[4 * j + e] * f[e];
          }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) pb[2 * u + g][j] = pack_bf16x2(p[8 * g + 2 * j], p[8 * g + 2 * j + 1]);
      }
      // V operand of block n and group g: d = 32 n + col, this half's 8 tokens
      const uint16_t* vb = &s_v[buf][col * 16 + ((half ^ (col >> 3)) & 1) * 8];
      if (SCALED || !edge || s_odd[buf] != i) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            o[n] = mfma_32x32_bf16(load_u32x4(vb + g * GROUP + n * 512), pb[g], o[n]);
      } else {  // see attn_direct.h
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const u32x4_t v = drop_nonfinite<2>(load_u32x4(vb + g * GROUP + n * 512));
            o[n] = mfma_32x32_bf16(v, pb[g], o[n]);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll 1
        for (int x = 0; x < TL_TOKENS; ++x) {
          const int t = t0 + x, place = 8 * ((x >> 2) & 1) + 4 * ((x >> 3) & 1) + (x & 3);
          if (!(groups >> (x >> 4) & 1) || t > pos || (A.window && t <= pos - A.window)) continue;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int d = 32 * n + reg_token(j, half);
              const float f = bf16_bits_to_f32(s_v[buf][(x >> 4) * GROUP + d * 16 + (place ^ (d & 8))]);
              if (!(fabsf(f) < INFINITY)) o[n][j] += f;
            }
        }
      }
    }
    if (i + 1 < n_tiles) store_tile(buf ^ 1, i + 1);
    __syncthreads();
  }
  if (!row_ok) return;

  const float sum = half_sum(l);
  const int64_t at = (int64_t)(s.q0 + tok) * A.Hq + head;
  if (used > 1) {
    const int64_t place = (int64_t)split * K.T * A.Hq + at;
    if (half == 0) {
      A.part_ml[2 * place] = m;
      A.part_ml[2 * place + 1] = sum;
    }
    float* dst = A.part_o + place * D;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4_t*>(dst + 32 * n + 8 * j + 4 * half) =
            f32x4_t{o[n][4 * j], o[n][4 * j + 1], o[n][4 * j + 2], o[n][4 * j + 3]};
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
      store_out<false>(A, oat + 32 * n + 8 * j + 4 * half, o[n][4 * j] * inv, o[n][4 * j + 1] * inv,
                       o[n][4 * j + 2] * inv, o[n][4 * j + 3] * inv);
}

}  // namespace sgmv
