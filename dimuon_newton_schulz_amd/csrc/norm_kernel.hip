// Global gradient norm over many tensors, and the clip coefficient.
#include "adamw.h"

namespace muon {
namespace {

// Sum over the workgroup, in a fixed order; thread 0 has the result.
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

__global__ __launch_bounds__(kNormThreads) void k_grad_norm(NormArgs a) {
  __shared__ double red[4];
  __shared__ bool last;
  for (uint32_t r = a.first_run[blockIdx.x]; r < a.first_run[blockIdx.x + 1]; ++r) {
    const NormRun run = a.runs[r];
    const NormTensor& t = a.tensors[run.tensor];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < run.count; i += kNormThreads) {
      const double x = load_elem(t.g, run.begin + i, t.dt);
      sum = __builtin_fma(x, x, sum);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) __hip_atomic_store(&a.partial[r], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // The last workgroup to store its sums adds them all up.
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  double sum = 0.0;
  for (uint32_t r = threadIdx.x; r < a.nruns; r += kNormThreads) sum += load_partial(&a.partial[r]);
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    a.out[0] = static_cast<float>(norm);
    a.out[1] = norm <= a.max_norm ? 1.0f : static_cast<float>(a.max_norm / norm);
    *a.ticket = 0;
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
