// Checking drafted tokens against the target's probabilities, with the random numbers given.
//
// Sequence b has drafts d_1..d_n, target rows p_1..p_{n+1}, draft rows q_1..q_n (or point masses at
// the drafts), uniforms a_1..a_n and r. Draft i is taken while a_i q_i(d_i) < p_i(d_i): for a
// uniform a that is the probability min(1, p / q). After the first draft that is not, i, the token
// is drawn from max(p_i - q_i, 0), which makes the pair's distribution p_i; where all are taken, from
// p_{n+1}. A row is drawn from by its running sum: the lowest j whose sum passes r times the total.
//
// Sums are in fp64: with 2^17 entries a running sum in fp32 is off by more than an entry's own
// weight. Bound by reading the one or two rows that are drawn from.
#include "verify.h"

namespace sgmv {

namespace {

constexpr int VF_THREADS = 1024;

template <class T> __device__ __forceinline__ float prob(const T* p);
template <> __device__ __forceinline__ float prob(const float* p) { return *p; }
template <> __device__ __forceinline__ float prob(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// What is not a weight (negative, NaN, infinite) counts as none.
__device__ __forceinline__ double weight(double w) { return w > 0. && w < 1e300 ? w : 0.; }
__device__ __forceinline__ float clean(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }

__device__ __forceinline__ double wave_scan(double v) {  // inclusive
  const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
  for (int o = 1; o < WAVE; o <<= 1) {
    const double u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

template <class T>
__global__ __launch_bounds__(VF_THREADS) void verify_kernel(VerifyArgs A) {
  __shared__ double s_sum[VF_THREADS / WAVE];
  __shared__ int s_at;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & (WAVE - 1), wv = tid / WAVE;
  const int d0 = min(max(A.start[b], 0), A.N);
  const int n = max(min(min(max(A.start[b + 1], 0), A.N) - d0, A.max_drafts), 0);
  const T* target = static_cast<const T*>(A.target) + (int64_t)(d0 + b) * A.ldt;
  const T* draft = static_cast<const T*>(A.draft) + (A.draft ? (int64_t)d0 * A.ldd : 0);
  int taken = n;
  for (int i0 = 0; i0 < n && taken == n; i0 += WAVE) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < n) {
      const int id = A.ids[d0 + i];
      ok = false;
      if ((uint32_t)id < (uint32_t)A.V) {
        const double p = clean(prob(target + (int64_t)i * A.ldt + id));
        const double q = A.draft ? clean(prob(draft + (int64_t)i * A.ldd + id)) : 1.0;
        ok = (double)A.accept_u[d0 + i] * q < p;
      }
    }
    const uint64_t bad = __ballot(!ok);
    if (bad) taken = i0 + __ffsll((unsigned long long)bad) - 1;
  }
  int32_t* out = A.tokens + (int64_t)b * A.ldo;
  for (int i = tid; i <= A.max_drafts; i += VF_THREADS)
    if (i != taken) out[i] = i < taken ? A.ids[d0 + i] : -1;
  if (tid == 0) A.accepted[b] = taken;

  const T* p = target + (int64_t)taken * A.ldt;
  const T* q = taken < n && A.draft ? draft + (int64_t)taken * A.ldd : nullptr;
  const int hole = taken < n && !A.draft ? A.ids[d0 + taken] : -1;
  const int per = (A.V + VF_THREADS - 1) / VF_THREADS;
  const int j0 = min(tid * per, A.V), j1 = min(j0 + per, A.V);
  if (tid == 0) s_at = -1;
  for (int pass = 0; pass < 2; ++pass) {  // the second where the rest is all zero: p itself
    auto w = [&](int j) {
      const float a = clean(prob(p + j));
      if (pass) return (double)a;
      return weight(j == hole ? 0. : (double)a - (q ? (double)clean(prob(q + j)) : 0.));
    };
    double mine = 0.;
    for (int j = j0; j < j1; ++j) mine += w(j);
    const double upto = wave_scan(mine);
    __syncthreads();
    if (lane == WAVE - 1) s_sum[wv] = upto;
    __syncthreads();
    double before = 0., total = 0.;
    for (int i = 0; i < VF_THREADS / WAVE; ++i) {
      if (i < wv) before += s_sum[i];
      total += s_sum[i];
    }
    if (!(total > 0.)) continue;
    const double at = (double)A.sample_u[b] * total;
    // the same sums on both sides of a border, so that the intervals leave no gap
    const double left = __shfl_up(upto, 1);
    const double lo = lane ? before + left : before, hi = before + upto;
    if (mine > 0. && lo <= at && at < hi) {
      double c = lo;
      int found = -1;
      for (int j = j0; j < j1; ++j) {
        const double x = w(j);
        c += x;
        if (x > 0.) found = j;
        if (c > at) break;
      }
      atomicMax(&s_at, found);
    }
    break;
  }
  __syncthreads();
  if (tid == 0) out[taken] = s_at;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& A, hipStream_t stream) {
  if (A.bf16) verify_kernel<uint16_t><<<dim3(A.B), dim3(VF_THREADS), 0, stream>>>(A);
  else verify_kernel<float><<<dim3(A.B), dim3(VF_THREADS), 0, stream>>>(A);
  return hipGetLastError();
}

}  // namespace sgmv
