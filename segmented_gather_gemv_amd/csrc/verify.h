// Arguments of the draft check (verify.hip).
#pragma once

#include "common.h"

namespace sgmv {

constexpr int VF_PART = 1024;  // entries of a row that one wave sums

struct VerifyArgs {
  const void* target;
  const void* draft;  // null: point masses
  int64_t ldt, ldd;
  const int32_t* ids;
  const int32_t* start;
  const float* accept_u;
  const float* sample_u;
  int32_t* tokens;
  int64_t ldo;
  int32_t* accepted;
  double* sums;  // [B][parts][2]: of what is left of the row, of the row itself
  int32_t B, V, N, max_drafts, bf16, parts;
  int32_t vec;  // rows may be read four entries at a time
};

hipError_t launch_verify(const VerifyArgs& A, hipStream_t stream);

}  // namespace sgmv
