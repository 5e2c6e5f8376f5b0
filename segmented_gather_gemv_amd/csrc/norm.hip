// Root-mean-square norm of rows, with the addition of a residual before it and 8-bit codes beside its output:
//   h = x + r,  g = h w,  out = g / sqrt(sum h^2 / W + eps),  scale = max |g| / sqrt(..) / F,  code = round(g F / max |g|).
// h and g are fp32, each rounded once (the sum of two bf16 values is exact unless they are 2^16 apart); the sum of
// squares is fp32. The codes need no root: it cancels, so that they are those of g's exact quotient (quantise.h).
//
// A row is held in registers by the threads that share it, 16 bytes of x and r a piece, from one read of memory; its
// sum and its maximum go over the group in one step (codes of a second pass would read the row
// again). Bound: the rows' bytes; of few rows, a launch, the loads and that step. Measured (with residual;
// a large copy: 5.14 TB/s): 8192 rows of 8192 with int8 codes 109 us (604 MB, 5.5 TB/s), 256 rows of 4096 with e4m3
// codes 5.2, one row of 8192 3.8; 7021 rows of 80, fp32 3.5; 6057 rows of 1716 with int8 codes 17.5 (52 MB, 3.0 TB/s).
#include "norm.h"
#include "quantise.h"

namespace sgmv {

namespace {

constexpr int NONE = -1;  // no codes

// 16, 8, 4 and 2 bytes, wherever they start.
typedef u32x4_t any16_t __attribute__((aligned(1)));
typedef u32x2_t any8_t __attribute__((aligned(1)));
typedef uint32_t any4_t __attribute__((aligned(1)));
typedef uint16_t any2_t __attribute__((aligned(1)));

// 16 bytes of a row, n of its values inside it. Rows start anywhere (a load of 16 bytes takes no longer off its
// alignment); of a piece that the row ends in, 8, 4 and 2 bytes as its length has them, at once and in their places.
template <class T>
__device__ __forceinline__ u32x4_t load_piece(const T* p, int n) {
  constexpr int E = 16 / sizeof(T), HALF = E / 2;
  if (n >= E) return *reinterpret_cast<const any16_t*>(p);
  u32x2_t front = {0u, 0u}, back = {0u, 0u};
  if (n & HALF) front = *reinterpret_cast<const any8_t*>(p);
  if constexpr (sizeof(T) == 4) {
    if (n & 1) back[0] = *reinterpret_cast<const any4_t*>(p + (n & 2));
  } else {
    uint32_t pair = 0u, one = 0u;
    if (n & 2) pair = *reinterpret_cast<const any4_t*>(p + (n & 4));
    if (n & 1) one = p[n & 6];
    back = n & 2 ? u32x2_t{pair, one} : u32x2_t{one, 0u};
  }
  return n & HALF ? u32x4_t{front[0], front[1], back[0], back[1]} : u32x4_t{back[0], back[1], 0u, 0u};
}

template <class T, int E>
__device__ __forceinline__ void store_piece(T* p, int n, const float (&y)[E]) {
  constexpr int HALF = E / 2;
  u32x4_t v;
  if constexpr (sizeof(T) == 4) v = u32x4_t{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
  else v = u32x4_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
  if (n >= E) {
    *reinterpret_cast<any16_t*>(p) = v;
    return;
  }
  if (n & HALF) *reinterpret_cast<any8_t*>(p) = u32x2_t{v[0], v[1]};
  const u32x2_t back = n & HALF ? u32x2_t{v[2], v[3]} : u32x2_t{v[0], v[1]};
  if constexpr (sizeof(T) == 4) {
    if (n & 1) *reinterpret_cast<any4_t*>(p + (n & 2)) = back[0];
  } else {
    if (n & 2) *reinterpret_cast<any4_t*>(p + (n & 4)) = back[0];
    if (n & 1) p[n & 6] = (T)(n & 2 ? back[1] : back[0]);
  }
}

// Codes of a piece.
template <int E>
__device__ __forceinline__ void store_codes(char* p, int n, const uint32_t (&c)[E / 4]) {
  if (n >= E) {
    if constexpr (E == 8) *reinterpret_cast<any8_t*>(p) = u32x2_t{c[0], c[1]};
    else *reinterpret_cast<any4_t*>(p) = c[0];
    return;
  }
  uint32_t back = c[0];
  if constexpr (E == 8) {
    if (n & 4) {
      *reinterpret_cast<any4_t*>(p) = c[0];
      back = c[1];
    }
  }
  if (n & 2) *reinterpret_cast<any2_t*>(p + (n & 4)) = (uint16_t)back;
  if (n & 1) p[n & 6] = (char)(n & 2 ? back >> 16 : back);
}

// Value e of a piece.
template <class T>
__device__ __forceinline__ float piece_value(u32x4_t v, int e) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(v[e]);
  return __uint_as_float(e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16);
}

// Sum of s and maximum of t over the lanes of a group within a wave.
template <int LANES, class S>
__device__ __forceinline__ void reduce_lanes(S& s, uint32_t& t) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    s += __shfl_xor(s, o);
    t = max(t, (uint32_t)__shfl_xor((int)t, o));
  }
}

template <class T, int FMT, int GROUP, int PER>
__global__ __launch_bounds__(GROUP > 256 ? GROUP : 256) void norm_kernel(NormArgs A) {
  constexpr int E = 16 / sizeof(T), THREADS = GROUP > 256 ? GROUP : 256, WAVES = GROUP / WAVE;
  const int i = threadIdx.x % GROUP;
  const int64_t row = (int64_t)blockIdx.x * (THREADS / GROUP) + threadIdx.x / GROUP;
  if (row >= A.rows) return;  // (whole groups; those of several waves have a workgroup each)
  int64_t t = row;
  int head = 0;
  if (A.H > 1) {
    t = row / A.H;
    head = (int)(row - t * A.H);
  }
  const T* x = static_cast<const T*>(A.x) + t * A.ldx_t + head * A.ldx_h;
  const T* w = static_cast<const T*>(A.weight);
  const auto left = [&](int p) { return A.W - p * E; };  // values of the row from piece p on

  u32x4_t xw[PER], rw[PER], ww[PER];
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    const int p = i + n * GROUP;
    xw[n] = left(p) > 0 ? load_piece<T>(x + p * E, left(p)) : u32x4_t{0u, 0u, 0u, 0u};
  }
  if (A.residual) {
    const T* r = static_cast<const T*>(A.residual) + t * A.ldr_t + head * A.ldr_h;
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int p = i + n * GROUP;
      rw[n] = left(p) > 0 ? load_piece<T>(r + p * E, left(p)) : u32x4_t{0u, 0u, 0u, 0u};
    }
  }
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    const int p = i + n * GROUP;
    ww[n] = left(p) > 0 ? load_piece<T>(w + p * E, left(p)) : u32x4_t{0u, 0u, 0u, 0u};
  }

  float h[PER][E];
#pragma unroll
  for (int n = 0; n < PER; ++n)
#pragma unroll
    for (int e = 0; e < E; ++e) h[n][e] = piece_value<T>(xw[n], e);
  if (A.residual) {
    T* s = static_cast<T*>(A.residual_out) + t * A.lds_t + head * A.lds_h;
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int p = i + n * GROUP;
#pragma unroll
      for (int e = 0; e < E; ++e) h[n][e] += piece_value<T>(rw[n], e);
      if (A.residual_out && left(p) > 0) store_piece<T, E>(s + p * E, left(p), h[n]);
    }
  }
  const auto g = [&](int n, int e) { return h[n][e] * piece_value<T>(ww[n], e); };

  float sum = 0.f;
  uint32_t top = 0u;  // bits of the maximum of |g|
#pragma unroll
  for (int n = 0; n < PER; ++n)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum = fmaf(h[n][e], h[n][e], sum);
      if constexpr (FMT != NONE) top = max(top, __float_as_uint(g(n, e)) & 0x7fffffffu);
    }
  reduce_lanes<GROUP < WAVE ? GROUP : WAVE>(sum, top);
  __shared__ float s_sum[WAVES ? WAVES : 1];
  __shared__ uint32_t s_top[WAVES ? WAVES : 1];
  __shared__ double s_far[WAVES ? WAVES : 1];
  const int wv = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
  if constexpr (WAVES > 1) {
    if (lane == 0) {
      s_sum[wv] = sum;
      s_top[wv] = top;
    }
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      sum += s_sum[k];
      top = max(top, s_top[k]);
    }
  }
  float root = 1.f / sqrtf(sum / (float)A.W + A.eps), down = 1.f;
  // Squares that fp32 does not hold, or a sum next to which those that it has lost may count: again in fp64, with
  // values of the largest rows scaled so that the root does not leave fp32 either.
  if (!(sum < 1e37f) || sum < 1e-24f) {
    double far = 0.0;
#pragma unroll
    for (int n = 0; n < PER; ++n)
#pragma unroll
      for (int e = 0; e < E; ++e) far += (double)h[n][e] * (double)h[n][e];
    uint32_t unused = 0u;
    reduce_lanes<GROUP < WAVE ? GROUP : WAVE>(far, unused);
    if constexpr (WAVES > 1) {
      if (lane == 0) s_far[wv] = far;
      __syncthreads();
      far = 0.0;
#pragma unroll
      for (int k = 0; k < WAVES; ++k) far += s_far[k];
    }
    down = sum < 1e-24f ? 1.f : 0x1p-64f;
    root = (float)(1.0 / sqrt(far / A.W + (double)A.eps) / (double)down);
  }

  if (A.out) {
    T* out = static_cast<T*>(A.out) + t * A.ldo_t + head * A.ldo_h;
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int p = i + n * GROUP;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = g(n, e) * down * root;
      if (left(p) > 0) store_piece<T, E>(out + p * E, left(p), y);
    }
  }
  if constexpr (FMT != NONE) {
    const RowScale S = row_scale<FMT>(top);
    constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
    // (NaN where a value is not finite, as the scale of such a row of the cache)
    if (i == 0) A.scale[row] = top >= 0x7f800000u ? S.scale : S.amax * down * root / F;
    char* codes = static_cast<char*>(A.codes) + t * A.ldc_t + head * A.ldc_h;
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int p = i + n * GROUP;
      uint32_t c[E / 4];
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        const float q[4] = {g(n, 4 * k), g(n, 4 * k + 1), g(n, 4 * k + 2), g(n, 4 * k + 3)};
        c[k] = quantise4<FMT, float>(q, S);
      }
      if (left(p) > 0) store_codes<E>(codes + p * E, left(p), c);
    }
  }
}

template <class T, int FMT, int GROUP, int PER>
hipError_t launch(const NormArgs& A, hipStream_t stream) {
  constexpr int THREADS = GROUP > 256 ? GROUP : 256, ROWS = THREADS / GROUP;
  norm_kernel<T, FMT, GROUP, PER><<<(unsigned)((A.rows + ROWS - 1) / ROWS), THREADS, 0, stream>>>(A);
  return hipGetLastError();
}

template <class T, int FMT>
hipError_t launch_shape(const NormArgs& A, hipStream_t stream) {
  const NormShape s = norm_shape(A.rows, (A.W + 16 / (int)sizeof(T) - 1) / (16 / (int)sizeof(T)));
  if (s.group == 16) return s.per == 1 ? launch<T, FMT, 16, 1>(A, stream) : launch<T, FMT, 16, 2>(A, stream);
  if (s.group == 64) {
    if (s.per == 1) return launch<T, FMT, 64, 1>(A, stream);
    return s.per == 2 ? launch<T, FMT, 64, 2>(A, stream) : launch<T, FMT, 64, 4>(A, stream);
  }
  if (s.group == 256) {
    if (s.per == 1) return launch<T, FMT, 256, 1>(A, stream);
    return s.per == 2 ? launch<T, FMT, 256, 2>(A, stream) : launch<T, FMT, 256, 4>(A, stream);
  }
  if (s.group == 512) return launch<T, FMT, 512, 4>(A, stream);
  if (s.per == 1) return launch<T, FMT, 1024, 1>(A, stream);
  if (s.per == 2) return launch<T, FMT, 1024, 2>(A, stream);
  if (s.per == 4) return launch<T, FMT, 1024, 4>(A, stream);
  if constexpr (sizeof(T) == 4) {
    if (s.per == 8) return launch<T, FMT, 1024, 8>(A, stream);
  }
  return hipErrorInvalidValue;
}

template <class T>
hipError_t launch_format(const NormArgs& A, int format, hipStream_t stream) {
  if (!A.codes) return launch_shape<T, NONE>(A, stream);
  return format == SGMV_KV_E4M3 ? launch_shape<T, SGMV_KV_E4M3>(A, stream) : launch_shape<T, SGMV_KV_I8>(A, stream);
}

}  // namespace

// As few threads as hold the row in up to four pieces each, so that their loads are in flight together; of few rows,
// which do not fill the card, as many as it has pieces for. Measured with codes, us: 129 to 256 pieces in 256 threads
// and in 64 with four each: 740 rows of 1833 6.0 and 7.8, 2324 of 1834 12.7 and 12.5, 6057 of 1716 18.2 and 17.5; 1025 to
// 2048 pieces in 512 threads with four each and in 1024: 1500 rows of 16384 47 and 52, 600 of 12000 13.7 and 12.9.
NormShape norm_shape(int64_t rows, int pieces) {
  if (pieces <= 16) return {16, 1};
  if (pieces <= 32) return {16, 2};
  if (pieces <= 64) return {64, 1};
  const bool few = rows < 512;
  if (few && pieces > 256) return {1024, pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : pieces <= 4096 ? 4 : 8};
  if (few) return {256, 1};
  if (pieces <= 128) return {64, 2};
  if (pieces <= 256) return rows < 2048 ? NormShape{256, 1} : NormShape{64, 4};
  if (pieces <= 512) return {256, 2};
  if (pieces <= 1024) return {256, 4};
  if (pieces <= 2048) return rows < 1024 ? NormShape{1024, 2} : NormShape{512, 4};
  return {1024, pieces <= 4096 ? 4 : 8};
}

hipError_t launch_norm(const NormArgs& A, int dtype, int format, hipStream_t stream) {
  return dtype == SGMV_F32 ? launch_format<float>(A, format, stream) : launch_format<uint16_t>(A, format, stream);
}

}  // namespace sgmv
