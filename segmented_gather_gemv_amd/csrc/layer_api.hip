// C-ABI of the norm and of the base product: argument validation and launch geometry. Stateless; every call runs on
// the caller's stream. Declarations and contracts are in include/sgmv.h.
#include <algorithm>
#include <cmath>

#include "base.h"
#include "norm.h"

namespace sgmv {

namespace {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool row_type_ok(int dtype) { return dtype == SGMV_F32 || dtype == SGMV_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline sgmv_status launched(hipError_t e) { return e == hipSuccess ? SGMV_OK : SGMV_EHIP; }
constexpr int64_t MOST_WAVES = 0xffffffffll / 64;  // of a launch: it takes fewer than 2^32 work items

// Rows [T][heads][W] with a token and a head stride: rows must not overlap one another, tokens or heads outermost.
bool rows_ok(const void* p, const sgmv_norm* n, int64_t ld_t, int64_t ld_h) {
  const int64_t T = n->T, H = n->heads, W = n->width;
  const auto nested = [W](int64_t inner, int64_t ld_in, int64_t outer, int64_t ld_out) {
    return (inner == 1 || ld_in >= W) && (outer == 1 || (__int128)ld_out >= (inner == 1 ? 0 : (__int128)(inner - 1) * ld_in) + W);
  };
  return p && (nested(H, ld_h, T, ld_t) || nested(T, ld_t, H, ld_h));
}

// Whether outputs may stand where they do. Rows are read whole before they are written, each by the threads that write
// it: an output may be x or the residual row for row, and nothing else may be in two places of a call.
bool places_ok(const sgmv_norm* n) {
  const auto row_for_row = [n](const void* out, int64_t out_t, int64_t out_h, const void* in, int64_t in_t, int64_t in_h) {
    return !out || out != in || ((n->T == 1 || out_t == in_t) && (n->heads == 1 || out_h == in_h));
  };
  const void* const outs[] = {n->residual_out, n->out, n->codes, n->scale};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    for (int k = 0; k < i; ++k)
      if (outs[i] == outs[k]) return false;
    if (outs[i] == n->weight || (i >= 2 && (outs[i] == n->x || outs[i] == n->residual))) return false;
  }
  return row_for_row(n->out, n->ldo_token, n->ldo_head, n->x, n->ldx_token, n->ldx_head) &&
         row_for_row(n->out, n->ldo_token, n->ldo_head, n->residual, n->ldr_token, n->ldr_head) &&
         row_for_row(n->residual_out, n->lds_token, n->lds_head, n->x, n->ldx_token, n->ldx_head) &&
         row_for_row(n->residual_out, n->lds_token, n->lds_head, n->residual, n->ldr_token, n->ldr_head);
}

// The sizes of a weight's parts.
struct BaseShape {
  int64_t tiles, blocks, groups, s, scale_rows, per_group;
};

BaseShape base_shape(const sgmv_base& b) {
  BaseShape h;
  h.tiles = ceil_div(b.N, BASE_N);
  h.blocks = ceil_div(b.K, BASE_K);
  h.groups = ceil_div(b.K, b.group);
  h.s = b.group < BASE_K ? BASE_K / b.group : 1;
  h.scale_rows = b.group < BASE_K ? h.blocks : h.groups;
  h.per_group = b.group < BASE_K ? 1 : b.group / BASE_K;
  return h;
}

sgmv_status base_shape_ok(int32_t N, int32_t K, int32_t group, int32_t format, int32_t dtype, int32_t has_zero) {
  if (N < 1 || K < 1 || group < 1 || (format != SGMV_BASE_I4 && format != SGMV_BASE_E2M1) || !row_type_ok(dtype) ||
      (has_zero != 0 && has_zero != 1))
    return SGMV_EINVAL;
  if (format == SGMV_BASE_E2M1 && (has_zero || group != 32)) return SGMV_EINVAL;
  if ((group != 32 && group != 64 && group % BASE_K) || N > SGMV_BASE_MAX_SIZE || K > SGMV_BASE_MAX_SIZE)
    return SGMV_EUNSUPPORTED;
  return SGMV_OK;
}

sgmv_status base_ok(const sgmv_base* b) {
  if (!b || !b->codes || !b->scale) return SGMV_EINVAL;
  const sgmv_status s = base_shape_ok(b->N, b->K, b->group, b->format, b->dtype, b->has_zero);
  if (s != SGMV_OK) return s;
  if ((b->has_zero != 0) != (b->zero != nullptr)) return SGMV_EINVAL;
  if (!aligned_to(b->codes, 16) || !aligned_to(b->scale, 16) || !aligned_to(b->zero, 16)) return SGMV_EINVAL;
  return SGMV_OK;
}

// How a product is computed.
struct BasePlan {
  bool tiled;
  int32_t splits, split_blocks;
  size_t rows, parts;  // floats of workspace
};

// The tiled kernel converts each code for 64 rows, not 16 or 32, but has its rows prepared in a launch of its own and
// takes few workgroups: for bf16 rows, from 160 full tiles or 1e10 products on, for fp32 ones from 128 or 5e9. Measured
// (in tiles by the ranges below, direct; us): bf16, I4: 850 rows, 3008 x 1408: 24 and 20, 600 rows, 4096 x 1024: 19 and
// 16, 1000 rows: 20 and 23, 256 rows, 4096 x 4096: 27 and 18, 128 rows, 8192 x 8192: 36 and 30, 150 rows, 8192 x 8000: 43
// and 43, 256 rows, 8192 x 8192: 52 and 55, 64 rows, 28672 x 8192: 53 and 62, x 5000 (which the rule leaves direct): 38
// and 40; fp32: 800 rows, 2527 x 313: 21 and 16, 400 rows, 4096 x 1024: 32 and 22, 170 rows, 4096 x 4096: 40 and 30, 200
// rows, 1088 x 12096: 57 and 30, 1000 rows, 4096 x 1024: 41 and 43, 128 rows, 8192 x 8192: 65 and 71, 340 rows, 4096 x
// 4096: 57 and 53.
//
// Tiles fill the card from 256 on; of fewer, K is split into up to 8 ranges of 8 steps and more (256 rows, 8192 x 8192:
// 82 us in 1, 54 in 2, 51 in 4, 60 in 8; 1024 over 4096 x 4096, 256 tiles: 49 us in 1, 53 in 2); of fp32 rows into up to
// 16 of 12 steps (202 rows, 732 x 15403: 72 us in 8, 53 in 16; 100 rows, 4096 x 4096: 33 in 8, 37 in 16).
BasePlan base_plan(int32_t T, const sgmv_base& b, int32_t n_split) {
  const BaseShape h = base_shape(b);
  BasePlan p{};
  p.splits = 1;
  const bool f32 = b.dtype == SGMV_F32;
  const double area = (double)T * b.N, full = (double)TILE_T * TILE_N;
  if (!n_split && (f32 ? T <= 16 || (area < 128 * full && area * b.K < 5e9) : T <= 32 || (area < 160 * full && area * b.K < 1e10)))
    return p;
  p.tiled = true;
  const int64_t bands = ceil_div(T, TILE_T), tiles = bands * ceil_div(b.N, TILE_N), steps = h.blocks * (f32 ? 3 : 1);
  if (n_split) p.splits = n_split;
  else if (tiles < 256) {
    const int64_t most = std::max(std::min<int64_t>(8, steps / 8), f32 ? std::min<int64_t>(SGMV_BASE_MAX_SPLITS, steps / 12) : 1);
    p.splits = (int32_t)std::max<int64_t>(1, std::min(512 / tiles, most));
  }
  p.split_blocks = (int32_t)ceil_div(h.blocks, p.splits);
  p.splits = (int32_t)ceil_div(h.blocks, p.split_blocks);
  p.rows = (size_t)bands * TILE_T * h.blocks * (f32 ? 3 : 1) * (BASE_K / 2 + (b.format == SGMV_BASE_I4 ? h.s : 0));
  if (p.splits > 1) p.parts = (size_t)p.splits * tiles * TILE_T * TILE_N;
  return p;
}

inline int scale_size(int format, int dtype) { return format == SGMV_BASE_E2M1 ? 1 : dtype == SGMV_F32 ? 4 : 2; }

}  // namespace
}  // namespace sgmv

using namespace sgmv;

extern "C" {

sgmv_status sgmv_rms_norm(const sgmv_norm* n, void* stream) {
  if (!n || n->T < 0 || n->heads < 1 || n->width < 1 || !row_type_ok(n->dtype) || !std::isfinite(n->eps) || n->eps <= 0.f)
    return SGMV_EINVAL;
  if (n->codes && n->format != SGMV_KV_E4M3 && n->format != SGMV_KV_I8) return SGMV_EINVAL;
  if (n->width > SGMV_MAX_NORM_WIDTH) return SGMV_EUNSUPPORTED;
  if (n->T == 0) return SGMV_OK;
  if (!n->weight || !rows_ok(n->x, n, n->ldx_token, n->ldx_head) || (n->codes != nullptr) != (n->scale != nullptr) ||
      (!n->out && !n->codes) || (n->residual_out && !n->residual))
    return SGMV_EINVAL;
  if ((n->residual && !rows_ok(n->residual, n, n->ldr_token, n->ldr_head)) ||
      (n->residual_out && !rows_ok(n->residual_out, n, n->lds_token, n->lds_head)) ||
      (n->out && !rows_ok(n->out, n, n->ldo_token, n->ldo_head)) ||
      (n->codes && !rows_ok(n->codes, n, n->ldc_token, n->ldc_head)) || !places_ok(n))
    return SGMV_EINVAL;
  const int E = n->dtype == SGMV_F32 ? 4 : 8;
  const NormArgs A{n->x, n->residual, n->weight, n->residual_out, n->out, n->codes, n->scale,
                   n->ldx_token, n->ldx_head, n->ldr_token, n->ldr_head, n->lds_token, n->lds_head,
                   n->ldo_token, n->ldo_head, n->ldc_token, n->ldc_head, (int64_t)n->T * n->heads, n->heads, n->width,
                   n->eps};
  const NormShape s = norm_shape(A.rows, (int)ceil_div(n->width, E));
  if (ceil_div(A.rows * s.group, 64) + 16 > MOST_WAVES) return SGMV_EUNSUPPORTED;
  return launched(launch_norm(A, n->dtype, n->format, static_cast<hipStream_t>(stream)));
}

sgmv_status sgmv_base_init(int32_t N, int32_t K, int32_t group, int32_t format, int32_t dtype, int32_t has_zero,
                           sgmv_base* base, size_t* code_bytes, size_t* scale_bytes, size_t* zero_bytes) {
  if (!base || !code_bytes || !scale_bytes || !zero_bytes) return SGMV_EINVAL;
  const sgmv_status st = base_shape_ok(N, K, group, format, dtype, has_zero);
  if (st != SGMV_OK) return st;
  *base = sgmv_base{nullptr, nullptr, nullptr, N, K, group, format, dtype, has_zero};
  const BaseShape h = base_shape(*base);
  const size_t scales = (size_t)h.tiles * h.scale_rows * BASE_N * h.s;
  *code_bytes = (size_t)h.tiles * h.blocks * BASE_N * BASE_K / 2;
  *scale_bytes = scales * scale_size(format, dtype);
  *zero_bytes = has_zero ? scales : 0;
  return SGMV_OK;
}

sgmv_status sgmv_base_pack(const uint8_t* codes, int64_t ldc, const void* scale, const uint8_t* zero,
                           const sgmv_base* b, void* stream) {
  const sgmv_status st = base_ok(b);
  if (st != SGMV_OK) return st;
  if (!codes || ldc < (b->K + 1) / 2 || !scale || (zero != nullptr) != (b->has_zero != 0)) return SGMV_EINVAL;
  const BaseShape h = base_shape(*b);
  if (h.tiles * h.blocks * 4 > MOST_WAVES || h.tiles * h.scale_rows * BASE_N * h.s / 64 + 4 > MOST_WAVES) return SGMV_EUNSUPPORTED;
  const BasePackArgs A{codes, ldc, scale, zero, b->codes, b->scale, b->zero, b->N, b->K, (int32_t)h.groups,
                       (int32_t)h.blocks, (int32_t)h.scale_rows, (int32_t)h.s, b->format == SGMV_BASE_E2M1,
                       scale_size(b->format, b->dtype)};
  return launched(launch_base_pack(A, static_cast<hipStream_t>(stream)));
}

sgmv_status sgmv_base_product_workspace(int32_t T, const sgmv_base* b, int32_t n_split, size_t* bytes) {
  if (!bytes || T < 0 || n_split < 0 || n_split > SGMV_BASE_MAX_SPLITS) return SGMV_EINVAL;
  const sgmv_status st = base_ok(b);
  if (st != SGMV_OK) return st;
  const BasePlan p = base_plan(T, *b, n_split);
  *bytes = (p.rows + p.parts) * sizeof(float);
  return SGMV_OK;
}

sgmv_status sgmv_base_product(const void* x, int64_t ldx, int32_t T, const sgmv_base* b, void* y, int64_t ldy,
                              int32_t n_split, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const sgmv_status st = sgmv_base_product_workspace(T, b, n_split, &need);
  if (st != SGMV_OK) return st;
  if (T == 0) return SGMV_OK;
  if (!x || !y || x == y || (T > 1 && (ldx < b->K || ldy < b->N))) return SGMV_EINVAL;
  if (need) {
    if (!workspace || !aligned_to(workspace, 16)) return SGMV_EINVAL;
    if (workspace_bytes < need) return SGMV_ECAPACITY;
  }
  const BaseShape h = base_shape(*b);
  const BasePlan p = base_plan(T, *b, n_split);
  const int f32 = b->dtype == SGMV_F32;
  const BaseArgs A{b->codes, b->scale, b->zero, x, y, ldx, ldy, T, b->N, b->K, (int32_t)h.blocks, (int32_t)h.scale_rows,
                   (int32_t)h.per_group, static_cast<char*>(workspace), aligned_to(y, 16) && (T == 1 || ldy % 8 == 0), p.splits, p.split_blocks,
                   static_cast<float*>(workspace) + p.rows};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (p.tiled) {
    const int64_t bands = ceil_div(T, TILE_T);
    if ((bands * ceil_div(b->N, TILE_N) + 8) * 4 * std::max(p.splits, TILE_T / 16) > MOST_WAVES ||
        bands * h.blocks * 4 > MOST_WAVES)
      return SGMV_EUNSUPPORTED;
    return launched(launch_base_tiled(A, b->format, b->dtype, (int)h.s, s));
  }
  if (ceil_div(T, 16) * h.tiles * 16 > MOST_WAVES) return SGMV_EUNSUPPORTED;
  return launched(f32                           ? launch_base_direct_f32(A, b->format, (int)h.s, s)
                  : b->format == SGMV_BASE_E2M1 ? launch_base_direct_e2m1(A, s)
                  : b->zero                     ? launch_base_direct_i4z(A, (int)h.s, s)
                                                : launch_base_direct_i4(A, (int)h.s, s));
}

}  // extern "C"
