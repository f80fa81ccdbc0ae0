// Global gradient norm over many tensors, and the clip coefficient.
#include "adamw.h"

namespace muon {
namespace {

// Sum over the workgroup, in a fixed order; every thread has the result.
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = wave_sum_f64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ double load_partial(const double* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void add_square(double& s, float x) {
  const double d = x;
  s = __builtin_fma(d, d, s);
}

// Squares of the V = 16 bytes' worth of elements in one load.
template <bool BF16>
__device__ __forceinline__ void add_vector(double (&s)[2], uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      add_square(s[0], __uint_as_float(w[k] << 16));
      add_square(s[1], __uint_as_float(w[k] & 0xffff0000u));
    } else {
      add_square(s[k & 1], __uint_as_float(w[k]));
    }
  }
}

// This thread's share of a run: 16-byte vectors threadIdx.x + k * threads,
// four in flight, then the elements behind the last whole vector.
template <bool BF16>
__device__ __forceinline__ double run_sum(const void* g, int64_t begin, int64_t count) {
  constexpr int V = BF16 ? 8 : 4, U = 4;
  const char* base = static_cast<const char*>(g) + begin * (BF16 ? 2 : 4);
  const MUON_GLOBAL uint4* q = reinterpret_cast<const MUON_GLOBAL uint4*>(gmem(base));
  const int64_t nv = count / V;
  double s[2] = {0.0, 0.0};
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * kNormThreads < nv; i += U * kNormThreads) {
    uint4 u[U];
#pragma unroll
    for (int k = 0; k < U; ++k) u[k] = q[i + k * kNormThreads];
#pragma unroll
    for (int k = 0; k < U; ++k) add_vector<BF16>(s, u[k]);
  }
  for (; i < nv; i += kNormThreads) add_vector<BF16>(s, q[i]);
  const int64_t e = nv * V + threadIdx.x;
  if (e < count) add_square(s[0], load_elem(base, e, BF16 ? DT_BF16 : DT_F32));
  return s[0] + s[1];
}

__global__ __launch_bounds__(kNormThreads) void k_grad_norm(NormArgs a) {
  __shared__ double red[4];
  __shared__ bool last;
  for (uint32_t r = a.first_run[blockIdx.x]; r < a.first_run[blockIdx.x + 1]; ++r) {
    const NormRun run = a.runs[r];
    const NormTensor& t = a.tensors[run.tensor];
    const double part = t.dt == DT_BF16 ? run_sum<true>(t.g, run.begin, run.count)
                                        : run_sum<false>(t.g, run.begin, run.count);
    const double sum = block_sum(part, red);
    if (threadIdx.x == 0) __hip_atomic_store(&a.partial[r], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // The last workgroup to store its sums adds them all up.  The sums are
  // stored and loaded at agent scope, past the XCD's own L2, and each is
  // complete before its workgroup counts itself; so the counter needs no
  // release, which would write back the whole L2.
  if (threadIdx.x == 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last = ticket_last(a.tickets, ticket_take(a.tickets));
  }
  __syncthreads();
  if (!last) return;
  double sum = 0.0;
  for (uint32_t r = threadIdx.x; r < a.nruns; r += kNormThreads) sum += load_partial(&a.partial[r]);
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    a.out[0] = static_cast<float>(norm);
    a.out[1] = norm <= a.max_norm ? 1.0f : static_cast<float>(a.max_norm / norm);
  }
  if (a.tensor_norms)
    for (uint32_t t = threadIdx.x; t < a.ntensors; t += kNormThreads) {
      double own = 0.0;
      for (uint32_t r = a.tensors[t].run0; r < a.tensors[t + 1].run0; ++r) own += load_partial(&a.partial[r]);
      a.tensor_norms[t] = static_cast<float>(sqrt(own));
    }
}

}  // namespace

hipError_t launch_grad_norm(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_norm, dim3(a.nwg), dim3(kNormThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
