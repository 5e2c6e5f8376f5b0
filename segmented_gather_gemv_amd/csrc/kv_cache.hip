// Writing new tokens into the paged key/value cache, quantised on the way, and reading tokens back.
//
// A row is one (token, head): D values. For the 8-bit formats, with F = 448 (e4m3) or 127 (int8):
//   amax = max |x|,  scale = amax / F,  code = round(x * F / amax) to the format, ties to even;
//   a row of zeros has scale 0 and codes 0; a row with a non-finite value has scale NaN and codes
//   0, so that it reads back as NaN whatever the format can hold.
// bf16 rows: x * F is exact in fp32 and one correctly rounded division follows; a quotient of so
// few bits lies on a border of the format or far from it, so the code is the definition's. fp32
// rows: the quotient is formed in fp64 and rounded to odd before the last rounding, for the same
// result. Either way the arithmetic hides behind the rows' bytes.
//
// One wave per group of 16 tokens (of one sequence) and head: lane l takes the values d = 2 l + ...
// of one token after another, so loads of a row are contiguous; the codes go through LDS into
// the group's layout, and the stores are contiguous pieces of it. A group whose 16 places are not all written keeps the
// bytes of the others: every store is of one element run that belongs to a written token.
#include "kv_common.h"

namespace sgmv {

namespace {

constexpr int RW_WAVES = 4;

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(uint16_t* p, float v) {
  *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
}

// fp32 nearest to d, rounded to odd: a later rounding to fewer bits then equals a single one.
__device__ __forceinline__ float to_odd(double d) {
  const float f = __double2float_rz(d);
  return (double)f == d ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

template <int FMT>
__device__ __forceinline__ uint32_t encode(float q) {
  if constexpr (FMT == SGMV_KV_E4M3) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xffu;
  } else {
    return (uint32_t)(int)rintf(q) & 0xffu;
  }
}

template <int FMT, class T>
__device__ __forceinline__ uint32_t quantise(float x, float amax) {
  constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
  if constexpr (sizeof(T) == 4) {
    return encode<FMT>(to_odd((double)x * (double)F / (double)amax));
  } else {
    // amax near fp32's largest would overflow x * F: both scaled by a power of two
    const float s = amax > 1e30f ? 0x1p-32f : 1.f;
    return encode<FMT>(x * s * F / (amax * s));
  }
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// (sequence, first token of the group) of slot `w`: the groups of sequence b take the slots from
// first(b) = (tokens before b) / 16 + 2 b on; a sequence of n tokens touches at most
// (n + 14) / 16 + 1 groups of its own.
template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_write_kernel(KvArgs K, KvRows A) {
  const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE;
  const int slot = blockIdx.x * RW_WAVES + wv, head = blockIdx.y;
  const int b = wave_find(K.B, slot, [&](int i) { return min(max(K.q_start[i], 0), K.T) / 16 + 2 * i; });
  const KvSeq s = kv_seq(K, b);
  const int first = s.kv_len - s.q_len;  // position of the first new token; may be negative
  const int g0 = (first >> 4) + (slot - (s.q0 / 16 + 2 * b));
  const int t_lo = max(max(16 * g0, first), 0), t_hi = min(16 * g0 + 16, s.kv_len);
  if (t_lo >= t_hi) return;
  const int page = kv_page(K, K.table + (int64_t)b * K.ldp, t_lo);
  if (page < 0) return;
  const int ps = 1 << K.lps, D = K.D;
  const int64_t row = ((int64_t)page * K.H + head) * ps;  // first token of the (page, head) block
  const int64_t group = (row + ((16 * g0) & (ps - 1))) * D;
  constexpr int C = 16 / KvFormat<FMT>::bytes;
  for (int t = t_lo; t < t_hi; ++t) {
    const int64_t src = s.q0 + (t - first);
    const int r = t & 15, place = 8 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);
    const T* kr = static_cast<const T*>(A.k) + src * A.ldk_t + head * A.ldk_h;
    const T* vr = static_cast<const T*>(A.v) + src * A.ldv_t + head * A.ldv_h;
    if constexpr (!KvFormat<FMT>::scaled) {
      T* kc = static_cast<T*>(const_cast<void*>(K.k)) + group;
      T* vc = static_cast<T*>(const_cast<void*>(K.v)) + group;
      for (int d = lane; d < D; d += WAVE) {
        kc[(d / C) * (16 * C) + r * C + d % C] = kr[d];
        vc[d * 16 + place] = vr[d];
      }
    } else {
      uint8_t* kc = static_cast<uint8_t*>(const_cast<void*>(K.k)) + group;
      uint8_t* vc = static_cast<uint8_t*>(const_cast<void*>(K.v)) + group;
      constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
      float xk[4], xv[4], ak = 0.f, av = 0.f, bad_k = 0.f, bad_v = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = lane + WAVE * i;
        xk[i] = d < D ? load_elem(kr + d) : 0.f;
        xv[i] = d < D ? load_elem(vr + d) : 0.f;
        ak = fmaxf(ak, fabsf(xk[i]));
        av = fmaxf(av, fabsf(xv[i]));
        bad_k += xk[i] * 0.f;  // NaN where x is not finite
        bad_v += xv[i] * 0.f;
      }
      ak = wave_max(ak);
      av = wave_max(av);
      const bool ok_k = !__any(bad_k != 0.f), ok_v = !__any(bad_v != 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = lane + WAVE * i;
        if (d < D) {
          kc[(d / C) * (16 * C) + r * C + d % C] =
              ok_k && ak > 0.f ? (uint8_t)quantise<FMT, T>(xk[i], ak) : 0;
          vc[d * 16 + place] = ok_v && av > 0.f ? (uint8_t)quantise<FMT, T>(xv[i], av) : 0;
        }
      }
      if (lane == 0) {
        const float nan = __uint_as_float(0x7fc00000u);
        const_cast<float*>(K.k_scale)[row + (t & (ps - 1))] = ok_k ? ak / F : nan;
        const_cast<float*>(K.v_scale)[row + (t & (ps - 1))] = ok_v ? av / F : nan;
      }
    }
  }
}

template <int FMT>
__device__ __forceinline__ float load_code(const void* p, int64_t i) {
  if constexpr (FMT == SGMV_KV_F32) {
    return static_cast<const float*>(p)[i];
  } else if constexpr (FMT == SGMV_KV_BF16) {
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  } else {
    float f[4];
    codes4<FMT>((uint32_t)static_cast<const uint8_t*>(p)[i], f);
    return f[0];
  }
}

template <int FMT, class T>
__global__ __launch_bounds__(RW_WAVES* WAVE) void kv_read_kernel(KvArgs K, KvRows A) {
  const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE;
  const int slot = blockIdx.x * RW_WAVES + wv, head = blockIdx.y;
  const int b = wave_find(K.B, slot, [&](int i) { return min(max(A.out_start[i], 0), A.rows) / 16 + 2 * i; });
  const int r0 = min(max(A.out_start[b], 0), A.rows), r1 = min(max(A.out_start[b + 1], 0), A.rows);
  const int n = max(r1 - r0, 0), kv_len = kv_seq(K, b).kv_len;
  const int first = kv_len - n;
  const int g0 = (first >> 4) + (slot - (r0 / 16 + 2 * b));
  const int t_lo = max(16 * g0, first), t_hi = min(16 * g0 + 16, kv_len);
  if (t_lo >= t_hi) return;
  const int page = kv_page(K, K.table + (int64_t)b * K.ldp, t_lo);
  const int ps = 1 << K.lps, D = K.D;
  const int64_t row = ((int64_t)max(page, 0) * K.H + head) * ps;
  const int64_t group = (row + ((16 * g0) & (ps - 1))) * D;
  constexpr int C = 16 / KvFormat<FMT>::bytes;
  for (int t = t_lo; t < t_hi; ++t) {
    const int64_t dst = r0 + (t - first);
    const int r = t & 15, place = 8 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);
    T* kr = static_cast<T*>(A.k) + dst * A.ldk_t + head * A.ldk_h;
    T* vr = static_cast<T*>(A.v) + dst * A.ldv_t + head * A.ldv_h;
    float ks = 1.f, vs = 1.f;
    if constexpr (KvFormat<FMT>::scaled) {
      if (page >= 0) {
        ks = K.k_scale[row + (t & (ps - 1))];
        vs = K.v_scale[row + (t & (ps - 1))];
      }
    }
    for (int d = lane; d < D; d += WAVE) {
      float x = 0.f, y = 0.f;
      if (page >= 0) {
        x = load_code<FMT>(K.k, group + (d / C) * (16 * C) + r * C + d % C);
        y = load_code<FMT>(K.v, group + d * 16 + place);
        if constexpr (KvFormat<FMT>::scaled) {
          x *= ks;
          y *= vs;
        }
      }
      store_elem(kr + d, x);
      store_elem(vr + d, y);
    }
  }
}

}  // namespace

// Slots of 16-token groups for `tokens` rows of B sequences (see kv_write_kernel).
static dim3 row_grid(const KvArgs& K, int64_t tokens) {
  const int64_t slots = tokens / 16 + 2 * (int64_t)K.B;
  return dim3((unsigned)((slots + RW_WAVES - 1) / RW_WAVES), (unsigned)K.H);
}

#define KV_ROWS(KERNEL_, N_)                                                                   \
  do {                                                                                         \
    const dim3 g = row_grid(K, N_), b(RW_WAVES * WAVE);                                        \
    if (fmt == SGMV_KV_F32) KERNEL_<SGMV_KV_F32, float><<<g, b, 0, stream>>>(K, R);            \
    else if (fmt == SGMV_KV_BF16) KERNEL_<SGMV_KV_BF16, uint16_t><<<g, b, 0, stream>>>(K, R);  \
    else if (fmt == SGMV_KV_E4M3 && R.f32) KERNEL_<SGMV_KV_E4M3, float><<<g, b, 0, stream>>>(K, R); \
    else if (fmt == SGMV_KV_E4M3) KERNEL_<SGMV_KV_E4M3, uint16_t><<<g, b, 0, stream>>>(K, R);  \
    else if (R.f32) KERNEL_<SGMV_KV_I8, float><<<g, b, 0, stream>>>(K, R);                     \
    else KERNEL_<SGMV_KV_I8, uint16_t><<<g, b, 0, stream>>>(K, R);                             \
  } while (0)

hipError_t launch_kv_write(const KvArgs& K, const KvRows& R, int fmt, hipStream_t stream) {
  KV_ROWS(kv_write_kernel, K.T);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs& K, const KvRows& R, int fmt, hipStream_t stream) {
  KV_ROWS(kv_read_kernel, R.rows);
  return hipGetLastError();
}

#undef KV_ROWS

}  // namespace sgmv
