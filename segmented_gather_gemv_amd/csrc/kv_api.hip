// C-ABI of the paged cache, its attention and the draft check: argument validation, launch
// geometry and dispatch. Stateless; every call runs on the caller's stream. Declarations and
// contracts are in include/sgmv.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn.h"
#include "verify.h"

namespace sgmv {
hipError_t launch_kv_write(const KvArgs& K, const KvRows& R, int fmt, int max_q, hipStream_t stream);
hipError_t launch_kv_read(const KvArgs& K, const KvRows& R, int fmt, hipStream_t stream);
hipError_t launch_kv_append(const KvArgs& K, const KvRows& R, const KvTurn& turn, int fmt, int max_q, hipStream_t stream);
int64_t kv_append_waves(const KvArgs& K, const KvTurn& turn, int fmt, int max_q);
hipError_t launch_attn_direct_bf16(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_direct_e4m3(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_direct_i8(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_direct_f32(const AttnArgs& A, int fmt, hipStream_t stream);
hipError_t launch_attn_tiled_bf16(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_tiled_e4m3(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_tiled_i8(const AttnArgs& A, hipStream_t stream);
hipError_t launch_attn_combine(const AttnArgs& A, int kernel, hipStream_t stream);

namespace {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool scaled(int fmt) { return fmt == SGMV_KV_E4M3 || fmt == SGMV_KV_I8; }
inline int format_bytes(int fmt) { return fmt == SGMV_KV_F32 ? 4 : fmt == SGMV_KV_BF16 ? 2 : 1; }
inline bool row_type_ok(int dtype) { return dtype == SGMV_F32 || dtype == SGMV_BF16; }
// A cache that is not quantised holds rows of its own type only.
inline bool types_fit(int dtype, int fmt) {
  return scaled(fmt) || (fmt == SGMV_KV_F32) == (dtype == SGMV_F32);
}
constexpr int64_t MOST_ROWS = 0x7fffffff;
constexpr int64_t MOST_WAVES = 0xffffffffll / 64;  // of a launch: it takes fewer than 2^32 work items

sgmv_status shape_ok(int32_t pages, int32_t page_size, int32_t heads, int32_t head_dim, int32_t fmt) {
  if (pages < 1 || page_size < 1 || heads < 1 || head_dim < 1 || fmt < SGMV_KV_F32 || fmt > SGMV_KV_I8)
    return SGMV_EINVAL;
  if (page_size < SGMV_KV_GROUP || page_size > SGMV_KV_MAX_PAGE || (page_size & (page_size - 1)) ||
      head_dim % 16 || head_dim > SGMV_KV_MAX_HEAD_DIM || heads > SGMV_KV_MAX_HEADS)
    return SGMV_EUNSUPPORTED;
  return SGMV_OK;
}

sgmv_status cache_ok(const sgmv_kv_cache* c) {
  if (!c || !c->k || !c->v) return SGMV_EINVAL;
  const sgmv_status s = shape_ok(c->pages, c->page_size, c->heads, c->head_dim, c->format);
  if (s != SGMV_OK) return s;
  if (scaled(c->format) && (!c->k_scale || !c->v_scale)) return SGMV_EINVAL;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(c->k_scale, 16) ||
      !aligned_to(c->v_scale, 16))
    return SGMV_EINVAL;
  return SGMV_OK;
}

// Fills the arguments of a cache and a batch. `empty`: nothing to do.
sgmv_status fill(const sgmv_kv_batch* s, const sgmv_kv_cache* c, KvArgs& K, bool& empty) {
  const sgmv_status st = cache_ok(c);
  if (st != SGMV_OK) return st;
  if (!s || s->B < 0 || s->T < 0 || s->max_q < 0 || s->max_kv < 0 || s->table_pages < 0 ||
      s->ldp < s->table_pages)
    return SGMV_EINVAL;
  empty = s->B == 0;
  if (!empty && (!s->q_start || !s->kv_len || (s->table_pages > 0 && !s->page_table))) return SGMV_EINVAL;
  if (s->B > SGMV_KV_MAX_B) return SGMV_EUNSUPPORTED;
  K = KvArgs{c->k, c->v, c->k_scale, c->v_scale, s->q_start, s->kv_len, s->page_table, s->ldp,
             c->pages, __builtin_ctz((unsigned)c->page_size), s->table_pages, s->B, s->T, c->heads,
             c->head_dim};
  return SGMV_OK;
}

// Rows [n][heads][D] with a token and a head stride: rows must not overlap one another.
bool rows_ok(const void* p, int64_t n, int64_t ld_t, int64_t ld_h, int heads, int D) {
  return p && ld_h >= D && (n <= 1 || ld_t >= (int64_t)(heads - 1) * ld_h + D);
}

// Whether rows of k and v may be accessed 16 bytes at a time.
int rows_vec(const void* k, const void* v, int64_t kt, int64_t kh, int64_t vt, int64_t vh, int32_t dtype) {
  const int64_t n = dtype == SGMV_F32 ? 4 : 8;
  return aligned_to(k, 16) && aligned_to(v, 16) && kt % n == 0 && kh % n == 0 && vt % n == 0 && vh % n == 0;
}

sgmv_status launched(hipError_t e) { return e == hipSuccess ? SGMV_OK : SGMV_EHIP; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// n ranges of `tokens` tokens, chunk a multiple of `unit`.
void split_tokens(int64_t n, int64_t tokens, int unit, int32_t& n_split, int32_t& chunk) {
  n = std::min<int64_t>(std::max<int64_t>(n, 1), SGMV_KV_MAX_SPLITS);
  const int64_t c = ceil_div(ceil_div(std::max<int64_t>(tokens, 1), n), unit) * unit;
  chunk = (int32_t)std::min<int64_t>(c, 0x40000000);
  n_split = (int32_t)n;
}

// Ranges for the tiled kernel, whose workgroups fill a compute unit each: as many as fit beside each other,
// of at least two tiles (100 tokens over 4096, 8 heads: 17 us in 16 ranges, 91 us in 1). Not beyond, where
// tiles of different lengths leave units idle at the end: their parts cost more than that (4 chunks of
// 300..700 beside 28 single tokens, 200 tiles: 73 us in 1 range, 134 in 2).
int64_t tiled_splits(int64_t base, int64_t tokens) {
  return base > 0 ? std::min(256 / base, ceil_div(tokens, 128)) : 1;
}

// Ranges for the direct kernel. A split costs its parts and a launch that joins them, about as long as
// five steps of the waves: rows of no more than six steps are not split (one sequence of 1000 tokens,
// bf16: 9.1 us in 1 range, 10.3 in 4; of 4000: 19.6 in 1, 10.4 in 16). Longer ones are by two rules, also
// beside tiles of many rows (8 prompts of 512 and one token over 6000: 91 us split, 102 not):
//   fill  up to a workgroup of 8 waves (two of 4) per compute unit, down to one step of each wave;
//   even  sequences of different lengths leave compute units idle at the end: up to four workgroups of 8
//         waves (six of 4) per compute unit, of long ranges (16 sequences of 8001..64003, e4m3: 361 us in 1
//         range, 238 in 2, 231 in 8). From 1024 workgroups of 4 waves on a call is not split (256 of
//         128..4096, bf16: 397 us in 1, 418 in 3).
// fp32 steps, of 4 waves, take four times as long: up to 512 tokens are not split (4 x 20 rows over 400, 32 /
// 8 heads of 128: 18.4 us in 1 range, 27.5 in 2; over 300 in a window of 256, 14 / 2 heads of 80: 12.1 and
// 14.5; 4 single tokens over 500: 12.2 and, in 4, 11.1 and a second launch for the host), and fill stops
// at one workgroup per compute unit (4 x 8 over 1000, heads of 128: 24.2 us in 2 ranges, 29.0 in 4).
void split_direct(AttnArgs& A, int64_t base, int64_t tokens, int forced) {
  const int step = A.direct_waves * (A.kv.k_scale ? 64 : 32);
  int64_t n = forced;
  if (!n && base > 0) {
    const int64_t fill = std::min<int64_t>((A.direct_waves == 8 || A.f32 ? 256 : 512) / base, ceil_div(tokens, step));
    const int64_t even = std::min<int64_t>((A.direct_waves == 8 ? 1024 : 1536) / base, ceil_div(tokens, 2 * A.direct_waves * step));
    n = tokens <= (A.f32 ? 512 : 6 * step) ? 1 : std::max(fill, even);
  }
  split_tokens(n, tokens, step, A.n_split[0], A.chunk[0]);
}

// Geometry of an attention call; everything but the pointers of its rows and workspace.
sgmv_status plan(const sgmv_attention* a, const sgmv_kv_batch* s, const sgmv_kv_cache* c, AttnArgs& A,
                 bool& empty) {
  std::memset(&A, 0, sizeof(A));
  if (!a) return SGMV_EINVAL;
  const sgmv_status st = fill(s, c, A.kv, empty);
  if (st != SGMV_OK) return st;
  if (!row_type_ok(a->dtype) || !types_fit(a->dtype, c->format) || a->heads < 1 ||
      a->heads % c->heads || !std::isfinite(a->scale) || a->scale <= 0.f || a->window < 0 ||
      a->n_split < 0 || a->n_split > SGMV_KV_MAX_SPLITS)
    return SGMV_EINVAL;
  if (a->heads > SGMV_KV_MAX_HEADS) return SGMV_EUNSUPPORTED;
  A.Hq = a->heads;
  A.G = a->heads / c->heads;
  A.f32 = a->dtype == SGMV_F32;
  A.scale_log2 = a->scale * 1.44269504088896341f;
  if (!std::isfinite(A.scale_log2)) return SGMV_EINVAL;
  A.window = a->window;
  empty = empty || s->T == 0;
  if ((int64_t)s->T * A.Hq > MOST_ROWS) return SGMV_EUNSUPPORTED;
  // sequences of few rows are taken directly; so are all where the tiled kernel has no instance
  const int D = c->head_dim, few = tiled_direct_rows(D);
  const bool tiled = !A.f32 && tiled_dim(D) && (int64_t)s->max_q * A.G > few;
  A.direct_rows = tiled ? few : INT32_MAX;
  const int64_t most = tiled ? few : (int64_t)s->max_q * A.G;  // rows of such a sequence
  // two tiles of 16 rows share K and V; of fp32 rows, whose products take their time, only where that
  // leaves workgroups for every compute unit
  const bool pair = direct_two_tiles(D, A.f32) && (!A.f32 || ((int64_t)s->T * A.G / 32 + s->B) * c->heads >= 512);
  A.direct_tile = most > 16 && pair ? 32 : 16;
  A.one_tile = most <= A.direct_tile;
  int64_t direct = A.one_tile ? s->B : (int64_t)s->T * A.G / A.direct_tile + s->B;
  // B max_q rows: as a rule every sequence has max_q, and nothing is left for the direct kernel. What q_start
  // holds is not known here, so shorter sequences are the tiled kernel's then, instead of workgroups that
  // mostly find nothing (1 x 2048 over 14001, e4m3: 424 us, 427 with them; 1 x 256 over 4096: 43 and 44; 32
  // single tokens in a step of 32 x 64, over 4096: 124 and 106).
  if (tiled && s->T == (int64_t)s->B * s->max_q) {
    direct = 0;
    A.direct_rows = 0;
  }
  const int64_t tiles = tiled ? (int64_t)s->T * A.G / tiled_rows(D) + s->B : 0;
  int64_t tokens = s->max_kv;
  if (a->window) tokens = std::min(tokens, (int64_t)a->window + s->max_q + AT_TOKENS);
  A.direct_waves = tiled ? tiled_waves(D) : direct_eight_waves(D, A.f32) && direct * c->heads < 512 ? 8 : 4;
  split_direct(A, direct * c->heads, tokens, a->n_split);
  split_tokens(a->n_split ? a->n_split : tiled_splits(tiles * c->heads, tokens), tokens, 64, A.n_split[1], A.chunk[1]);
  if (!direct) A.n_split[0] = 1;
  if (!tiles) A.n_split[1] = 1;
  // workgroups of the attention launch, and of those that join parts (a wave for a row)
  const int64_t joined = std::max(A.n_split[0] > 1 ? direct * A.direct_tile : 0, A.n_split[1] > 1 ? tiles * tiled_rows(D) : 0);
  if ((direct * A.n_split[0] + tiles * A.n_split[1]) * c->heads * (tiled ? tiled_waves(D) : A.direct_waves) > MOST_WAVES ||
      joined * c->heads > MOST_WAVES)
    return SGMV_EUNSUPPORTED;
  A.slots[0] = (int32_t)direct;
  A.slots[1] = (int32_t)tiles;
  return SGMV_OK;
}

// Places the parts of both kernels in the workspace; returns its bytes.
size_t place_parts(AttnArgs& A, void* workspace) {
  float* at = static_cast<float*>(workspace);
  size_t floats = 0;
  for (int kernel = 0; kernel < 2; ++kernel) {
    if (A.n_split[kernel] <= 1) continue;
    const int tile = kernel ? tiled_rows(A.kv.D) : A.direct_tile;
    const int64_t rows = (int64_t)A.kv.T * A.Hq, slots = (int64_t)A.slots[kernel] * tile * A.kv.H;
    A.part_rows[kernel] = std::min(rows, slots);
    A.part_tile[kernel] = slots < rows ? tile : 0;
    const size_t n = (size_t)A.n_split[kernel] * A.part_rows[kernel];
    A.part_o[kernel] = at ? at + floats : nullptr;  // 16-byte aligned: D is a multiple of 16, and so is the rest
    A.part_ml[kernel] = at ? A.part_o[kernel] + n * A.kv.D : nullptr;
    floats += n * (A.kv.D + 2);
    if (kernel == 0) floats = (floats + 3) & ~(size_t)3;
  }
  return floats * sizeof(float);
}

}  // namespace
}  // namespace sgmv

using namespace sgmv;

extern "C" {

sgmv_status sgmv_kv_init(int32_t pages, int32_t page_size, int32_t heads, int32_t head_dim,
                         int32_t format, sgmv_kv_cache* cache, size_t* data_bytes,
                         size_t* scale_bytes) {
  if (!cache || !data_bytes || !scale_bytes) return SGMV_EINVAL;
  const sgmv_status s = shape_ok(pages, page_size, heads, head_dim, format);
  if (s != SGMV_OK) return s;
  *cache = sgmv_kv_cache{nullptr, nullptr, nullptr, nullptr, pages, page_size, heads, head_dim, format};
  const size_t rows = (size_t)pages * page_size * heads;
  *data_bytes = rows * head_dim * format_bytes(format);
  *scale_bytes = scaled(format) ? rows * sizeof(float) : 0;
  return SGMV_OK;
}

sgmv_status sgmv_kv_write(const void* k, int64_t ldk_token, int64_t ldk_head, const void* v,
                          int64_t ldv_token, int64_t ldv_head, int32_t dtype,
                          const sgmv_kv_batch* batch, const sgmv_kv_cache* cache, void* stream) {
  KvArgs K;
  bool empty;
  const sgmv_status s = fill(batch, cache, K, empty);
  if (s != SGMV_OK) return s;
  if (!row_type_ok(dtype) || !types_fit(dtype, cache->format)) return SGMV_EINVAL;
  if (empty || batch->T == 0) return SGMV_OK;
  if (!rows_ok(k, K.T, ldk_token, ldk_head, K.H, K.D) || !rows_ok(v, K.T, ldv_token, ldv_head, K.H, K.D))
    return SGMV_EINVAL;
  const KvRows R{const_cast<void*>(k), const_cast<void*>(v), ldk_token, ldk_head, ldv_token, ldv_head,
                 nullptr, 0, dtype == SGMV_F32,
                 rows_vec(k, v, ldk_token, ldk_head, ldv_token, ldv_head, dtype)};
  return launched(launch_kv_write(K, R, cache->format, batch->max_q, static_cast<hipStream_t>(stream)));
}

sgmv_status sgmv_kv_append(const sgmv_kv_rotation* turn, const void* k, int64_t ldk_token, int64_t ldk_head,
                           const void* v, int64_t ldv_token, int64_t ldv_head, int32_t dtype,
                           const sgmv_kv_batch* batch, const sgmv_kv_cache* cache, void* stream) {
  KvArgs K;
  bool empty;
  const sgmv_status s = fill(batch, cache, K, empty);
  if (s != SGMV_OK) return s;
  if (!turn || !row_type_ok(dtype) || !types_fit(dtype, cache->format) || turn->rotary < 1 || turn->rotary > K.D ||
      turn->positions < 1 || turn->ld < turn->rotary || turn->heads < 0 || (turn->interleaved != 0 && turn->interleaved != 1))
    return SGMV_EINVAL;
  if (turn->rotary % 16 || turn->heads > SGMV_KV_MAX_HEADS) return SGMV_EUNSUPPORTED;
  if (empty || batch->T == 0) return SGMV_OK;
  if (!turn->cos_sin || !aligned_to(turn->cos_sin, 4) || !rows_ok(k, K.T, ldk_token, ldk_head, K.H, K.D) ||
      !rows_ok(v, K.T, ldv_token, ldv_head, K.H, K.D))
    return SGMV_EINVAL;
  if (turn->heads > 0 && (!rows_ok(turn->q, K.T, turn->ldq_token, turn->ldq_head, turn->heads, K.D) ||
                          !rows_ok(turn->q_out, K.T, turn->ldo_token, turn->ldo_head, turn->heads, K.D)))
    return SGMV_EINVAL;
  if (turn->heads > 0 && (turn->q_out == k || turn->q_out == v)) return SGMV_EINVAL;
  if (turn->heads > 0 && turn->q == turn->q_out && ((K.T > 1 && turn->ldq_token != turn->ldo_token) ||
                                                    (turn->heads > 1 && turn->ldq_head != turn->ldo_head)))
    return SGMV_EINVAL;
  const KvRows R{const_cast<void*>(k), const_cast<void*>(v), ldk_token, ldk_head, ldv_token, ldv_head,
                 nullptr, 0, dtype == SGMV_F32,
                 rows_vec(k, v, ldk_token, ldk_head, ldv_token, ldv_head, dtype)};
  const KvTurn t{turn->cos_sin, turn->ld, turn->positions, turn->rotary, turn->interleaved,
                 turn->q, turn->q_out, turn->ldq_token, turn->ldq_head, turn->ldo_token, turn->ldo_head, turn->heads,
                 rows_vec(turn->q, turn->q_out, turn->ldq_token, turn->ldq_head, turn->ldo_token, turn->ldo_head, dtype)};
  if (kv_append_waves(K, t, cache->format, batch->max_q) > MOST_WAVES) return SGMV_EUNSUPPORTED;
  return launched(launch_kv_append(K, R, t, cache->format, batch->max_q, static_cast<hipStream_t>(stream)));
}

sgmv_status sgmv_kv_read(const sgmv_kv_batch* batch, const sgmv_kv_cache* cache,
                         const int32_t* out_start, int32_t rows, void* k, int64_t ldk_token,
                         int64_t ldk_head, void* v, int64_t ldv_token, int64_t ldv_head,
                         int32_t dtype, void* stream) {
  KvArgs K;
  bool empty;
  const sgmv_status s = fill(batch, cache, K, empty);
  if (s != SGMV_OK) return s;
  if (!row_type_ok(dtype) || !types_fit(dtype, cache->format) || rows < 0) return SGMV_EINVAL;
  if (empty || rows == 0) return SGMV_OK;
  if (!out_start || !rows_ok(k, rows, ldk_token, ldk_head, K.H, K.D) ||
      !rows_ok(v, rows, ldv_token, ldv_head, K.H, K.D))
    return SGMV_EINVAL;
  const KvRows R{k, v, ldk_token, ldk_head, ldv_token, ldv_head, out_start, rows, dtype == SGMV_F32,
                 rows_vec(k, v, ldk_token, ldk_head, ldv_token, ldv_head, dtype)};
  return launched(launch_kv_read(K, R, cache->format, static_cast<hipStream_t>(stream)));
}

sgmv_status sgmv_kv_attention_workspace(const sgmv_attention* attn, const sgmv_kv_batch* batch,
                                        const sgmv_kv_cache* cache, size_t* bytes) {
  if (!bytes) return SGMV_EINVAL;
  AttnArgs A;
  bool empty = true;
  const sgmv_status s = plan(attn, batch, cache, A, empty);
  if (s != SGMV_OK) return s;
  *bytes = empty ? 0 : place_parts(A, nullptr);
  return SGMV_OK;
}

sgmv_status sgmv_kv_attention(const sgmv_attention* attn, const sgmv_kv_batch* batch,
                              const sgmv_kv_cache* cache, void* workspace, size_t workspace_bytes,
                              void* stream) {
  AttnArgs A;
  bool empty = true;
  const sgmv_status s = plan(attn, batch, cache, A, empty);
  if (s != SGMV_OK) return s;
  if (empty) return SGMV_OK;
  const int D = A.kv.D;
  if (!rows_ok(attn->q, A.kv.T, attn->ldq_token, attn->ldq_head, A.Hq, D) ||
      !rows_ok(attn->out, A.kv.T, attn->ldo_token, attn->ldo_head, A.Hq, D))
    return SGMV_EINVAL;
  A.q = attn->q;
  A.out = attn->out;
  A.lse = attn->lse;
  A.ldq_t = attn->ldq_token;
  A.ldq_h = attn->ldq_head;
  A.ldo_t = attn->ldo_token;
  A.ldo_h = attn->ldo_head;
  const int e = A.f32 ? 4 : 2;
  A.q_vec = aligned_to(A.q, 16) && A.ldq_t * e % 16 == 0 && A.ldq_h * e % 16 == 0;
  A.o_vec = aligned_to(A.out, 4 * e) && A.ldo_t % 4 == 0 && A.ldo_h % 4 == 0;
  if (const size_t need = place_parts(A, workspace)) {
    if (!workspace || !aligned_to(workspace, 16)) return SGMV_EINVAL;
    if (workspace_bytes < need) return SGMV_ECAPACITY;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t err = hipSuccess;
  if (A.slots[1])
    err = (cache->format == SGMV_KV_BF16   ? launch_attn_tiled_bf16
           : cache->format == SGMV_KV_E4M3 ? launch_attn_tiled_e4m3
                                           : launch_attn_tiled_i8)(A, st);
  else if (A.f32)
    err = launch_attn_direct_f32(A, cache->format, st);
  else
    err = (cache->format == SGMV_KV_BF16   ? launch_attn_direct_bf16
           : cache->format == SGMV_KV_E4M3 ? launch_attn_direct_e4m3
                                           : launch_attn_direct_i8)(A, st);
  for (int kernel = 0; kernel < 2 && err == hipSuccess; ++kernel)
    if (A.n_split[kernel] > 1) err = launch_attn_combine(A, kernel, st);
  return launched(err);
}

size_t sgmv_verify_drafts_workspace(int32_t B, int32_t vocab) {
  if (B < 1 || vocab < 1) return 0;
  return (size_t)B * (size_t)ceil_div(vocab, VF_PART) * 2 * sizeof(double);
}

sgmv_status sgmv_verify_drafts(const void* target, int64_t ldt, const void* draft, int64_t ldd,
                               int32_t vocab, int32_t dtype, const int32_t* draft_ids,
                               const int32_t* draft_start, int32_t B, int32_t N,
                               int32_t max_drafts, const float* accept_u, const float* sample_u,
                               int32_t* tokens, int64_t ldo, int32_t* accepted, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (B < 0 || N < 0 || vocab < 1 || max_drafts < 0 || !row_type_ok(dtype)) return SGMV_EINVAL;
  if (B == 0) return SGMV_OK;
  if (!target || !draft_start || !sample_u || !tokens || !accepted || ldt < vocab ||
      (draft && ldd < vocab) || ldo < (int64_t)max_drafts + 1)
    return SGMV_EINVAL;
  if (N > 0 && max_drafts > 0 && (!draft_ids || !accept_u)) return SGMV_EINVAL;
  if (B >= SGMV_KV_MAX_B || vocab > SGMV_MAX_VOCAB) return SGMV_EUNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 16)) return SGMV_EINVAL;
  if (workspace_bytes < sgmv_verify_drafts_workspace(B, vocab)) return SGMV_ECAPACITY;
  const int e = dtype == SGMV_F32 ? 4 : 2;
  const bool vec = aligned_to(target, 4 * e) && ldt % 4 == 0 &&
                   (!draft || (aligned_to(draft, 4 * e) && ldd % 4 == 0));
  const VerifyArgs A{target, draft, ldt, ldd, draft_ids, draft_start, accept_u, sample_u, tokens, ldo,
                     accepted, static_cast<double*>(workspace), B, vocab, N, max_drafts,
                     dtype == SGMV_BF16, (int32_t)ceil_div(vocab, VF_PART), vec};
  return launched(launch_verify(A, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
