// Checking drafted tokens against the target's probabilities, with the random numbers given.
//
// Sequence b has drafts d_1..d_n, target rows p_1..p_{n+1}, draft rows q_1..q_n (or point masses at
// the drafts), uniforms a_1..a_n and r. Draft i is taken while a_i q_i(d_i) < p_i(d_i): for a
// uniform a that is the probability min(1, p / q). After the first draft that is not, i, the token
// is drawn from max(p_i - q_i, 0), which makes the pair's distribution p_i; where all are taken, from
// p_{n+1}. A row is drawn from by its running sum: the lowest j whose sum passes r times the total.
//
// Sums are in fp64: with 2^17 entries a running sum in fp32 is off by more than an entry's own
// weight. Bound by reading the one or two rows that are drawn from, so a row is cut into parts of VF_PART
// entries, one wave each: the first launch sums them (every wave looks at its sequence's drafts itself, a
// few loads), the second, one wave per sequence without a barrier, finds the part that r falls into and
// the entry in it (256 sequences over 131072 entries: 35 + 5 us, 5.4 TB/s; bf16 rows, 8 bytes a load, 34 us in all;
// the draw by a workgroup with barriers took 12 us). One launch in which the last wave of a sequence does the second part would need a
// cleared counter, which is a launch too.
#include "verify.h"

namespace sgmv {

namespace {

constexpr int VF_WAVES = 4;               // of a workgroup of the first launch
constexpr int VF_ONE_WAVES = 16;          // of a workgroup that does a row alone
constexpr int VF_ONE_PARTS = 32;          // of such a row
constexpr int VF_EACH = VF_PART / WAVE;   // entries of one lane

__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// What is not a weight (negative, NaN, infinite) counts as none.
__device__ __forceinline__ float clean(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
__device__ __forceinline__ double rest(double p, double q) { return p > q ? p - q : 0.; }

__device__ __forceinline__ double wave_scan(double v) {  // inclusive
  const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
  for (int o = 1; o < WAVE; o <<= 1) {
    const double u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The row that sequence b is drawn from: target row p, draft row q (or none), entry left out (or -1).
template <class T> struct Row {
  const T* p;
  const T* q;
  int hole;
};

struct Drafts {
  int first, n;
};

__device__ __forceinline__ Drafts drafts(const VerifyArgs& A, int b) {
  const int first = min(max(A.start[b], 0), A.N);
  return {first, max(min(min(max(A.start[b + 1], 0), A.N) - first, A.max_drafts), 0)};
}

template <class T>
__device__ __forceinline__ Row<T> drawn_row(const VerifyArgs& A, int b, Drafts d, int taken) {
  const bool out = taken < d.n;
  return {static_cast<const T*>(A.target) + (int64_t)(d.first + b + taken) * A.ldt,
          out && A.draft ? static_cast<const T*>(A.draft) + (int64_t)(d.first + taken) * A.ldd : nullptr,
          out && !A.draft ? A.ids[d.first + taken] : -1};
}

// Entries [j, j + 4) of a row, j a multiple of 4; 0 past the end.
template <class T, bool VEC>
__device__ __forceinline__ void four(const T* row, int j, int V, float (&f)[4]) {
  if (VEC && j + 4 <= V) {
    if constexpr (sizeof(T) == 4) {
      const u32x4_t v = load_u32x4(row + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = clean(__uint_as_float(v[i]));
    } else {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + j);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = clean(__uint_as_float(v[i] << 16));
        f[2 * i + 1] = clean(__uint_as_float(v[i] & 0xffff0000u));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = j + i < V ? clean(prob(row + j + i)) : 0.f;
  }
}

// How many of sequence b's drafts are taken, in every lane.
template <class T>
__device__ __forceinline__ int count_taken(const VerifyArgs& A, int b, Drafts d) {
  const int lane = threadIdx.x & (WAVE - 1);
  const T* target = static_cast<const T*>(A.target) + (int64_t)(d.first + b) * A.ldt;
  const T* draft = static_cast<const T*>(A.draft) + (A.draft ? (int64_t)d.first * A.ldd : 0);
  for (int i0 = 0; i0 < d.n; i0 += WAVE) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < d.n) {
      const int id = A.ids[d.first + i];
      ok = false;
      if ((uint32_t)id < (uint32_t)A.V) {
        const double p = clean(prob(target + (int64_t)i * A.ldt + id));
        const double q = A.draft ? clean(prob(draft + (int64_t)i * A.ldd + id)) : 1.0;
        ok = (double)A.accept_u[d.first + i] * q < p;  // exact: 24 bits times 24
      }
    }
    const uint64_t bad = __ballot(!ok);
    if (bad) return i0 + __ffsll((unsigned long long)bad) - 1;
  }
  return d.n;
}

// Everything of sequence b's outputs but the drawn token: one wave.
__device__ __forceinline__ void store_taken(const VerifyArgs& A, int b, Drafts d, int taken) {
  const int lane = threadIdx.x & (WAVE - 1);
  int32_t* out = A.tokens + (int64_t)b * A.ldo;
  for (int i = lane; i <= A.max_drafts; i += WAVE)
    if (i != taken) out[i] = i < taken ? A.ids[d.first + i] : -1;
  if (lane == 0) A.accepted[b] = taken;
}

// Sums of one part of the row (what lies past its end counts as 0): of what is left of p, and, BOTH, of p
// itself; in every lane.
template <class T, bool VEC, bool BOTH>
__device__ __forceinline__ void sum_part(const VerifyArgs& A, const Row<T>& row, int part, double& sum, double& all) {
  const int lane = threadIdx.x & (WAVE - 1);
  sum = all = 0.;
#pragma unroll
  for (int i = 0; i < VF_EACH / 4; ++i) {
    const int j = part * VF_PART + 4 * (i * WAVE + lane);
    float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
    four<T, VEC>(row.p, j, A.V, p);
    if (row.q) four<T, VEC>(row.q, j, A.V, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BOTH) all += p[e];
      sum += j + e == row.hole ? 0. : rest(p[e], q[e]);
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    sum += __shfl_xor(sum, o);
    if constexpr (BOTH) all += __shfl_xor(all, o);
  }
}

// The token that u falls on in a row whose parts have these sums (pairs as sum_part has them): one wave.
template <class T, bool VEC>
__device__ __forceinline__ int draw(const VerifyArgs& A, const Row<T>& row, const double* sums, double u) {
  const int lane = threadIdx.x & (WAVE - 1);
  // the part that u falls into; over p itself where nothing is left of it
  const int per = (A.parts + WAVE - 1) / WAVE;
  const int c0 = min(lane * per, A.parts), c1 = min(c0 + per, A.parts);
  double left = 0., all = 0.;
  for (int c = c0; c < c1; ++c) {
    left += sums[2 * c];
    all += sums[2 * c + 1];
  }
  const int pass = __any(left > 0.) ? 0 : 1;
  const double weight = pass ? all : left;
  double upto = wave_scan(weight);
  double before = __shfl_up(upto, 1);
  if (lane == 0) before = 0.;
  const double at = u * __shfl(upto, WAVE - 1);
  // The lowest lane with a weight whose sum passes; the last one with a weight if rounding leaves none. (The
  // lanes' sums are formed in different orders: that of a lane without a weight can pass where the sum of the
  // lane before it, or any lane's, does not.)
  const uint64_t some = __ballot(weight > 0.), here = __ballot(weight > 0. && at < upto);
  int token = -1;
  if (some && u >= 0. && u < 1.) {
    const int owner = here ? __ffsll((unsigned long long)here) - 1 : WAVE - 1 - __clzll((long long)some);
    double base = before;
    int part = c0;
    if (lane == owner) {
      double sum = before;
      for (int c = c0; c < c1; ++c) {
        const double x = sums[2 * c + pass];
        if (!(x > 0.)) continue;
        part = c;
        base = sum;
        sum += x;
        if (sum > at) break;
      }
    }
    part = __shfl(part, owner);
    base = __shfl(base, owner);

    const int j0 = part * VF_PART + lane * VF_EACH;
    double w[VF_EACH], mine = 0.;
#pragma unroll
    for (int i = 0; i < VF_EACH / 4; ++i) {
      float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
      four<T, VEC>(row.p, j0 + 4 * i, A.V, p);
      if (row.q && !pass) four<T, VEC>(row.q, j0 + 4 * i, A.V, q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[4 * i + e] = !pass && j0 + 4 * i + e == row.hole ? 0. : rest(p[e], q[e]);
        mine += w[4 * i + e];
      }
    }
    upto = wave_scan(mine);
    before = __shfl_up(upto, 1);
    double sum = base + (lane ? before : 0.);
    // the lowest entry that passes; the last one with a weight if rounding leaves none (the part's sum was
    // formed in another order)
    int found = -1, weighted = -1;
#pragma unroll
    for (int i = 0; i < VF_EACH; ++i) {
      sum += w[i];
      if (w[i] > 0.) {
        weighted = j0 + i;
        if (found < 0 && sum > at) found = j0 + i;
      }
    }
    const uint64_t f = __ballot(found >= 0), l = __ballot(weighted >= 0);
    if (f) token = __shfl(found, __ffsll((unsigned long long)f) - 1);
    else if (l) token = __shfl(weighted, WAVE - 1 - __clzll((long long)l));
  }
  return token;
}

template <class T, bool VEC>
__global__ __launch_bounds__(VF_WAVES* WAVE) void verify_sum_kernel(VerifyArgs A) {
  const int lane = threadIdx.x & (WAVE - 1), b = blockIdx.y;
  const int part = blockIdx.x * VF_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  if (part >= A.parts) return;
  const Drafts d = drafts(A, b);
  const int taken = count_taken<T>(A, b, d);
  if (part == 0) store_taken(A, b, d, taken);
  double sum, all;
  sum_part<T, VEC, true>(A, drawn_row<T>(A, b, d, taken), part, sum, all);
  if (lane < 2) A.sums[((int64_t)b * A.parts + part) * 2 + lane] = lane ? all : sum;
}

template <class T, bool VEC>
__global__ __launch_bounds__(WAVE) void verify_draw_kernel(VerifyArgs A) {
  const int b = blockIdx.x, taken = A.accepted[b];
  const int token = draw<T, VEC>(A, drawn_row<T>(A, b, drafts(A, b), taken), A.sums + (int64_t)b * A.parts * 2,
                                 (double)A.sample_u[b]);
  if (threadIdx.x == 0) A.tokens[(int64_t)b * A.ldo + taken] = token;
}

// Both in one launch, one workgroup per sequence, for rows of few parts: the fp64 sums of two parts per wave
// take a compute unit about as long as the second launch (fp32 rows, 4 drafts; replayed: 64 sequences of
// 32000 entries 10.9 us, 10.5 in two launches; 256 of them 17.2 and 19.3, one 8.5 and 8.6), and the host launches
// once (12 us a call, 14.5). The sums of p itself are formed only where nothing is left of it.
template <class T, bool VEC>
__global__ __launch_bounds__(VF_ONE_WAVES* WAVE) void verify_one_kernel(VerifyArgs A) {
  __shared__ double s_sums[2 * VF_ONE_PARTS];
  const int b = blockIdx.x, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), lane = threadIdx.x & (WAVE - 1);
  const Drafts d = drafts(A, b);
  const double u = A.sample_u[b];
  const int taken = count_taken<T>(A, b, d);
  if (wv == 0) store_taken(A, b, d, taken);
  const Row<T> row = drawn_row<T>(A, b, d, taken);
  double sum, none;
  for (int part = wv; part < A.parts; part += VF_ONE_WAVES) {
    sum_part<T, VEC, false>(A, row, part, sum, none);
    if (lane < 2) s_sums[2 * part + lane] = lane ? 0. : sum;
  }
  __syncthreads();
  if (!__any(lane < A.parts && s_sums[2 * min(lane, VF_ONE_PARTS - 1)] > 0.)) {  // the same in every wave
    for (int part = wv; part < A.parts; part += VF_ONE_WAVES) {
      sum_part<T, VEC, false>(A, Row<T>{row.p, nullptr, -1}, part, sum, none);
      if (lane == 0) s_sums[2 * part + 1] = sum;
    }
    __syncthreads();
  }
  if (wv) return;
  const int token = draw<T, VEC>(A, row, s_sums, u);
  if (threadIdx.x == 0) A.tokens[(int64_t)b * A.ldo + taken] = token;
}

template <class T, bool VEC>
void launch(const VerifyArgs& A, hipStream_t stream) {
  if (A.parts <= VF_ONE_PARTS) {
    verify_one_kernel<T, VEC><<<dim3((unsigned)A.B), VF_ONE_WAVES * WAVE, 0, stream>>>(A);
    return;
  }
  const dim3 g((unsigned)((A.parts + VF_WAVES - 1) / VF_WAVES), (unsigned)A.B);
  verify_sum_kernel<T, VEC><<<g, VF_WAVES * WAVE, 0, stream>>>(A);
  verify_draw_kernel<T, VEC><<<dim3((unsigned)A.B), WAVE, 0, stream>>>(A);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& A, hipStream_t stream) {
  if (A.bf16) A.vec ? launch<uint16_t, true>(A, stream) : launch<uint16_t, false>(A, stream);
  else A.vec ? launch<float, true>(A, stream) : launch<float, false>(A, stream);
  return hipGetLastError();
}

}  // namespace sgmv
