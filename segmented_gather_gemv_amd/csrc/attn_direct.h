// Attention over the paged cache with keys and values loaded straight into matrix-core operands.
//
// For one (sequence, key/value head), a tile of 32 rows (new token, query head of the group) and a
// range of tokens, each of the workgroup's 4 waves takes every fourth 32 tokens:
//   S^T = K Q^T   (tokens x rows),  p = exp2(c s - m),  O^T += V^T P^T,   one running (m, l) per row.
// A lane holds one row's scores in its registers (of tokens 8 (i / 4) + 4 half + i % 4), its
// maximum needs one exchange with the other half, its sum none before the end, and its
// probabilities are the next product's operand as they stand (kv_common.h). Nothing goes through
// LDS but the four waves' sums at the end.
//
// Bound: the bytes of K and V, read once per tile of rows. 32x32 products on 8 rows waste three
// quarters of the matrix cores, which does not matter: at 13 bytes per clock and CU (8 TB/s over 256
// CUs) K and V of bf16 keep them 10% busy.
#pragma once

#include "attn.h"

namespace sgmv {

// Product of 32 rows of one operand with 32 of the other over one 16-byte chunk per lane and half.
// bf16 operands: chunk = 8 values (bf16 cache) or 16 (8-bit, converted); fp32: the k = 2 product.
template <bool F32, int FMT> struct Direct {
  static constexpr int bytes = KvFormat<FMT>::bytes;
  static constexpr int C = 16 / bytes;                 // values of d in one K chunk
  static constexpr int q_regs = F32 ? C : C / 2;       // registers of Q that go with one chunk
  static constexpr int v_loads = bytes == 4 ? 2 : 1;   // 16-byte (8-byte for 8-bit) loads per V group

  // S^T += chunk of K times Q
  static __device__ __forceinline__ f32x16_t qk(u32x4_t k, const uint32_t (&q)[q_regs], f32x16_t s) {
    if constexpr (F32) {
      float f[C];
      if constexpr (bytes == 4) {
        f[0] = __uint_as_float(k.x); f[1] = __uint_as_float(k.y);
        f[2] = __uint_as_float(k.z); f[3] = __uint_as_float(k.w);
      } else {
        const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float g[4];
          codes4<FMT>(w[i], g);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[4 * i + j] = g[j];
        }
      }
#pragma unroll
      for (int i = 0; i < C; ++i) s = mfma_32x32_f32(f[i], __uint_as_float(q[i]), s);
    } else if constexpr (bytes == 2) {
      s = mfma_32x32_bf16(k, u32x4_t{q[0], q[1], q[2], q[3]}, s);
    } else {
      s = mfma_32x32_bf16(codes8_bf16<FMT>(u32x2_t{k.x, k.y}), u32x4_t{q[0], q[1], q[2], q[3]}, s);
      s = mfma_32x32_bf16(codes8_bf16<FMT>(u32x2_t{k.z, k.w}), u32x4_t{q[4], q[5], q[6], q[7]}, s);
    }
    return s;
  }
};

// A V operand: 8 tokens of one d, as stored.
template <int BYTES> struct VRegs;
template <> struct VRegs<1> { u32x2_t w; };
template <> struct VRegs<2> { u32x4_t w; };
template <> struct VRegs<4> { u32x4_t w[2]; };

template <int BYTES>
__device__ __forceinline__ VRegs<BYTES> load_v(const char* p) {
  VRegs<BYTES> r;
  if constexpr (BYTES == 1) r.w = *reinterpret_cast<const u32x2_t*>(p);
  if constexpr (BYTES == 2) r.w = load_u32x4(p);
  if constexpr (BYTES == 4) {
    r.w[0] = load_u32x4(p);
    r.w[1] = load_u32x4(p + 16);
  }
  return r;
}

// Keep the tokens whose bit of `keep` (8 bits, one per stored element) is set, zero the others.
__device__ __forceinline__ uint32_t keep_pair(uint32_t w, uint32_t two) {
  return w & ((two & 1 ? 0x0000ffffu : 0u) | (two & 2 ? 0xffff0000u : 0u));
}
__device__ __forceinline__ void keep_tokens(VRegs<1>& r, uint32_t keep) {
  const uint32_t b = keep & 15, c = keep >> 4;
  auto bytes = [](uint32_t m) {
    return (m & 1 ? 0xffu : 0u) | (m & 2 ? 0xff00u : 0u) | (m & 4 ? 0xff0000u : 0u) | (m & 8 ? 0xff000000u : 0u);
  };
  r.w.x &= bytes(b);
  r.w.y &= bytes(c);
}
__device__ __forceinline__ void keep_tokens(VRegs<2>& r, uint32_t keep) {
  r.w.x = keep_pair(r.w.x, keep);
  r.w.y = keep_pair(r.w.y, keep >> 2);
  r.w.z = keep_pair(r.w.z, keep >> 4);
  r.w.w = keep_pair(r.w.w, keep >> 6);
}
__device__ __forceinline__ void keep_tokens(VRegs<4>& r, uint32_t keep) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(keep >> i & 1)) r.w[i / 4][i % 4] = 0u;
}

// The places (16 bits, in V's order) of a group's first n tokens.
__device__ __forceinline__ uint32_t places_below(int n) {
  const uint32_t t = (1u << n) - 1u;  // tokens 4-7 and 8-11 change places
  return (t & 0xf00fu) | (t & 0x00f0u) << 4 | (t & 0x0f00u) >> 4;
}

__device__ __forceinline__ bool has_nonfinite(const VRegs<2>& r) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    any |= (r.w[i] & 0x7f80u) == 0x7f80u || (r.w[i] & 0x7f800000u) == 0x7f800000u;
  return any;
}
__device__ __forceinline__ bool has_nonfinite(const VRegs<4>& r) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) any |= (r.w[i / 4][i % 4] & 0x7f800000u) == 0x7f800000u;
  return any;
}

__device__ __forceinline__ void drop_nonfinite(VRegs<2>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((r.w[i] & 0x7f80u) == 0x7f80u) r.w[i] &= 0xffff0000u;
    if ((r.w[i] & 0x7f800000u) == 0x7f800000u) r.w[i] &= 0x0000ffffu;
  }
}
__device__ __forceinline__ void drop_nonfinite(VRegs<4>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((r.w[i / 4][i % 4] & 0x7f800000u) == 0x7f800000u) r.w[i / 4][i % 4] = 0u;
}

// O^T += V^T P^T over one group of 16 tokens: p holds this lane's 8 probabilities
template <bool F32, int FMT>
__device__ __forceinline__ f32x16_t pv(const VRegs<KvFormat<FMT>::bytes>& v, const float* p, u32x4_t pb,
                                       f32x16_t o) {
  if constexpr (F32) {
    float f[8];
    if constexpr (KvFormat<FMT>::bytes == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v.w[i / 4][i % 4]);
    } else {
      float a[4], b[4];
      codes4<FMT>(v.w.x, a);
      codes4<FMT>(v.w.y, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o = mfma_32x32_f32(f[i], p[i], o);
    return o;
  } else if constexpr (KvFormat<FMT>::bytes == 2) {
    return mfma_32x32_bf16(v.w, pb, o);
  } else {
    return mfma_32x32_bf16(codes8_bf16<FMT>(v.w), pb, o);
  }
}

// DP: head dimension rounded up to 64, 128 or 256; EXACT: it is that
template <bool F32, int FMT, int DP, bool EXACT>
__global__ __launch_bounds__(256) void attn_direct_kernel(AttnArgs A) {
  using X = Direct<F32, FMT>;
  constexpr int WAVES = 4;
  constexpr int NCH = DP / (2 * X::C);  // K chunks of one lane (its half's)
  constexpr int NB = DP / 32;           // blocks of 32 values of d
  const KvArgs& K = A.kv;
  const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int col = lane & 31, half = lane >> 5;
  const int D = EXACT ? DP : K.D;

  // this workgroup's piece
  const int kvh = blockIdx.x % K.H;
  const int rest = blockIdx.x / K.H;
  const int split = rest % A.n_split[0], slot = rest / A.n_split[0];
  int b, row0;
  if (A.one_tile) {
    b = slot;
    row0 = 0;
  } else {
    // row tiles of sequence b take the slots from (rows before b) / 32 + b on
    b = wave_find(K.B, slot, [&](int i) {
      return (int)((int64_t)min(max(K.q_start[i], 0), K.T) * A.G / AT_ROWS) + i;
    });
    b = __builtin_amdgcn_readfirstlane(b);
    row0 = (slot - ((int)((int64_t)min(max(K.q_start[b], 0), K.T) * A.G / AT_ROWS) + b)) * AT_ROWS;
  }
  const KvSeq s = kv_seq(K, b);
  const int rows = s.q_len * A.G;
  if (row0 < 0 || row0 >= rows || rows > A.direct_rows) return;
  const Span span = row_span(A, s, row0, AT_ROWS);
  const int used = span_splits(A, span, 0);
  if (split >= used) return;
  const int t_begin = span.begin + split * A.chunk[0];
  const int t_end = split == used - 1 ? span.end : t_begin + A.chunk[0];

  // Q: this lane's row, the chunks of d that its half meets
  const int row = row0 + col;
  const bool row_ok = row < rows;
  const int tok = (row_ok ? row : 0) / A.G, head = kvh * A.G + (row_ok ? row : 0) % A.G;
  uint32_t q[NCH][X::q_regs];
  {
    const int64_t at = (int64_t)(s.q0 + tok) * A.ldq_t + (int64_t)head * A.ldq_h;
    constexpr int NW = X::q_regs / 4;  // 16-byte pieces per chunk
    constexpr int E = F32 ? 4 : 8;     // values of q per piece
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int d = (2 * c + half) * X::C + w * E;
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (row_ok && (EXACT || d < D)) {
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
        for (int j = 0; j < 4; ++j) q[c][4 * w + j] = v[j];
      }
  }

  const int first = s.kv_len - s.q_len;
  const int pos = first + tok;                      // this row's position
  const int lo_pos = first + row0 / A.G;            // the tile's first and last
  const int hi_pos = first + (min(row0 + AT_ROWS, rows) - 1) / A.G;
  const int ps = 1 << K.lps;
  const int32_t* table = K.table + (int64_t)b * K.ldp;

  f32x16_t o[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i] = f32x16_t{};
  float m = -INFINITY, l = 0.f;

  // pages of this wave's next 32 tiles: lane 2 i + g holds that of group g of tile i
  int pages = -1;
  auto load_pages = [&](int i0) {
    const int t = t_begin + 32 * (wv + WAVES * (i0 + (lane >> 1))) + 16 * (lane & 1);
    pages = t < t_end ? kv_page(K, table, t) : -1;
  };
  const int n_tiles = (t_end - t_begin + 31) / 32;
  const int mine = wv < n_tiles ? (n_tiles - wv + WAVES - 1) / WAVES : 0;

  u32x4_t kr[NCH];
  float ks[16], vs[16];
  (void)ks; (void)vs;
  // block of group g of tile i: first token's index in [pages][H][ps]
  auto group_at = [&](int i, int g) {
    const int p = __builtin_amdgcn_readlane(pages, (2 * i + g) & 63);
    const int t = t_begin + 32 * (wv + WAVES * i) + 16 * g;
    return ((int64_t)max(p, 0) * K.H + kvh) * ps + (t & (ps - 1));
  };
  auto load_k = [&](int i) {
    const int64_t g0 = group_at(i, 0), g1 = group_at(i, 1);
    const char* p = static_cast<const char*>(K.k) + (lane & 16 ? g1 : g0) * D * X::bytes + (lane & 15) * 16;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      int d = 2 * c + half;
      if (!EXACT) d = min(d, D / X::C - 1);
      kr[c] = load_u32x4(p + d * 256);
    }
    if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(K.k_scale + (j < 2 ? g0 : g1) + 8 * (j & 1) + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) ks[4 * j + e] = a[e];
      }
    }
  };

  if (mine > 0) {
    load_pages(0);
    load_k(0);
  }
  for (int i = 0; i < mine; ++i) {
    const int t0 = t_begin + 32 * (wv + WAVES * i);
    const int p0 = __builtin_amdgcn_readlane(pages, (2 * i) & 63);
    const int p1 = __builtin_amdgcn_readlane(pages, (2 * i + 1) & 63);
    const int64_t g0 = group_at(i, 0), g1 = group_at(i, 1);
    VRegs<X::bytes> vr[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      int d = 32 * n + col;
      if (!EXACT) d = min(d, D - 1);
#pragma unroll
      for (int g = 0; g < 2; ++g)
        vr[n][g] = load_v<X::bytes>(static_cast<const char*>(K.v) + ((g ? g1 : g0) * D + d * 16 + 8 * half) * X::bytes);
    }
    if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(K.v_scale + (j < 2 ? g0 : g1) + 8 * (j & 1) + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) vs[4 * j + e] = a[e];
      }
    }

    f32x16_t sc = {};
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (EXACT || 2 * c * X::C < D) sc = X::qk(kr[c], q[c], sc);
    if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
      for (int j = 0; j < 16; ++j) sc[j] *= ks[j];
    }
    if (i + 1 < mine) {
      if (((i + 1) & 31) == 0) load_pages(i + 1);
      load_k(i + 1);
    }

    // a tile that some row sees only part of, or with tokens that are not there
    const bool edge = t0 + 31 > lo_pos || (A.window && t0 <= hi_pos - A.window) || p0 < 0 || p1 < 0;
    uint32_t there = 0xffffu;  // this lane's tokens that exist
    if (edge) {
      there = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = t0 + reg_token(j, half);
        const bool has = t < s.kv_len && (j < 8 ? p0 : p1) >= 0;
        there |= has ? 1u << j : 0u;
        if (!has || t > pos || (A.window && t <= pos - A.window)) sc[j] = -INFINITY;
      }
    }

    float top = sc[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, sc[j]);
    top = half_max(top) * A.scale_log2;
    // a stale maximum is as good as long as nothing grows past 2^8
    if (__any(top > m + 8.f)) {
      const float now = fmaxf(m, top);
      const float f = m == now ? 1.f : exp2f(m - now);  // 0 from -inf on
      m = now;
      l *= f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[n][j] *= f;
    }
    const float base = m == -INFINITY ? 0.f : m;
    float p[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      p[j] = __builtin_amdgcn_exp2f(fmaf(sc[j], A.scale_log2, -base));
      l += p[j];
    }
    if constexpr (KvFormat<FMT>::scaled) {
#pragma unroll
      for (int j = 0; j < 16; ++j) p[j] = edge && p[j] == 0.f ? 0.f : p[j] * vs[j];
    }
    u32x4_t pb[2] = {};
    if constexpr (!F32) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) pb[g][j] = pack_bf16x2(p[8 * g + 2 * j], p[8 * g + 2 * j + 1]);
    }
    if (edge) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 2; ++g) keep_tokens(vr[n][g], there >> (8 * g) & 0xffu);
      if constexpr (!KvFormat<FMT>::scaled) {
        // A V value that is not finite, in a tile that some rows see only part of: in the product,
        // 0 * inf would spoil the rows that do not see it. It is left out of the product and added
        // to the rows that see it, token by token. (8-bit codes are finite; their scales meet only
        // probabilities that are not 0.)
        bool odd = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int g = 0; g < 2; ++g) odd |= has_nonfinite(vr[n][g]);
        if (__any(odd)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int g = 0; g < 2; ++g) drop_nonfinite(vr[n][g]);
#pragma unroll 1
          for (int x = 0; x < AT_TOKENS; ++x) {
            const int t = t0 + x;
            if ((x < 16 ? p0 : p1) < 0 || t > pos || (A.window && t <= pos - A.window)) continue;
            const int64_t at = (x < 16 ? g0 : g1) * D + 8 * ((x >> 2) & 1) + 4 * ((x >> 3) & 1) + (x & 3);
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int d = 32 * n + reg_token(j, half);
                if (!EXACT && d >= D) continue;
                const float f = F32 ? static_cast<const float*>(K.v)[at + d * 16]
                                    : bf16_bits_to_f32(static_cast<const uint16_t*>(K.v)[at + d * 16]);
                if (!(fabsf(f) < INFINITY)) o[n][j] += f;
              }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int g = 0; g < 2; ++g) o[n] = pv<F32, FMT>(vr[n][g], p + 8 * g, pb[g], o[n]);
  }

  // the four waves' sums: waves 2, 3 hand theirs to 0, 1, then 1 to 0
  __shared__ float s_m[WAVES][32], s_l[WAVES][32];
  __shared__ float s_o[2][NB * 16 * WAVE];
  l = half_sum(l);
  if (half == 0) {
    s_m[wv][col] = m;
    s_l[wv][col] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0][col], s_m[1][col]), fmaxf(s_m[2][col], s_m[3][col]));
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += s_m[w][col] == -INFINITY ? 0.f : s_l[w][col] * exp2f(s_m[w][col] - top);
  const float f = m == -INFINITY ? 0.f : exp2f(m - top);
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[n][j] *= f;
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (wv >= step && wv < 2 * step) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) s_o[wv - step][(n * 16 + j) * WAVE + lane] = o[n][j];
    }
    __syncthreads();
    if (wv < step) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[n][j] += s_o[wv][(n * 16 + j) * WAVE + lane];
    }
    __syncthreads();
  }
  if (wv != 0 || !row_ok) return;

  const int64_t at = (int64_t)(s.q0 + tok) * A.Hq + head;
  if (used > 1) {
    const int64_t place = (int64_t)split * K.T * A.Hq + at;
    if (half == 0) {
      A.part_ml[2 * place] = top;
      A.part_ml[2 * place + 1] = sum;
    }
    float* dst = A.part_o + place * D;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * n + 8 * j + 4 * half;
        if (EXACT || d < D)
          *reinterpret_cast<f32x4_t*>(dst + d) = f32x4_t{o[n][4 * j], o[n][4 * j + 1], o[n][4 * j + 2], o[n][4 * j + 3]};
      }
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (A.lse && half == 0)
    A.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
  const int64_t oat = (int64_t)(s.q0 + tok) * A.ldo_t + (int64_t)head * A.ldo_h;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * n + 8 * j + 4 * half;
      if (!EXACT && d >= D) continue;
      store_out<F32>(A, oat + d, o[n][4 * j] * inv, o[n][4 * j + 1] * inv, o[n][4 * j + 2] * inv, o[n][4 * j + 3] * inv);
    }
}

}  // namespace sgmv

