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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Squares of the elements of one 16-byte load.
template <bool BF16>
__device__ __forceinline__ void add_vector(double (&s)[2], u32x4 u) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      add_square(s[0], __uint_as_float(u[k] << 16));
      add_square(s[1], __uint_as_float(u[k] & 0xffff0000u));
    } else {
      add_square(s[k & 1], __uint_as_float(u[k]));
    }
  }
}

// This thread's share of a leaf: 16-byte vectors threadIdx.x + k * threads,
// eight in flight, then the elements behind the last whole vector.
template <bool BF16, bool STREAM>
__device__ __forceinline__ double leaf_sum(const void* g, int count) {
  constexpr int V = BF16 ? 8 : 4, U = kNormLeafBytes / (16 * kNormThreads);
  const MUON_GLOBAL u32x4* q = reinterpret_cast<const MUON_GLOBAL u32x4*>(gmem(static_cast<const char*>(g)));
  const int nv = count / V;
  double s[2] = {0.0, 0.0};
  if (nv == U * kNormThreads) {
    u32x4 u[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if constexpr (STREAM) u[k] = __builtin_nontemporal_load(q + threadIdx.x + k * kNormThreads);
      else u[k] = q[threadIdx.x + k * kNormThreads];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) add_vector<BF16>(s, u[k]);
  } else {
    for (int i = threadIdx.x; i < nv; i += kNormThreads) add_vector<BF16>(s, q[i]);
    const int e = nv * V + threadIdx.x;
    if (e < count) add_square(s[0], load_elem(g, e, BF16 ? DT_BF16 : DT_F32));
  }
  return s[0] + s[1];
}

// Reads every element once, and squares and adds it in binary64 (which no
// float32 value overflows; a conversion and a product-sum an element, hidden
// behind the reads).
//   369M bf16: 116 us, 6.4 TB/s (a kernel that only reads reaches 7.4 to 7.7)
//   4M float32 in 128 tensors: 7.5 us, of which 2 for the tree's two levels
//     (three sets of gradients in turn; 6.2 where two sets stay in the caches,
//     as in the comparisons below)
// Against 2048 workgroups with long stretches and one that adds up all sums:
// 140 and 11.8 us.  Leaves of 16 KB took 126 and 7.3 us, of 64 KB 135 and 7.0
// (both before STREAM and with 64 children a node), against 130 and 7.0.
//
// STREAM: the gradients do not fit the 256 MB Infinity Cache, and are read
// past it (non-temporal).  369M bf16: 130 us without, 118 us with; 4M float32,
// which fit: 7.0 us without, 7.2 to 8 with (64 children a node).
template <bool STREAM>
__global__ __launch_bounds__(kNormThreads) void k_grad_norm(NormArgs a) {
  __shared__ double red[4];
  const NormLeaf leaf = a.leaves[blockIdx.x];
  const int count = static_cast<int>(leaf.count);
  double sum = block_sum(leaf.dt == DT_BF16 ? leaf_sum<true, STREAM>(leaf.g, count)
                                             : leaf_sum<false, STREAM>(leaf.g, count),
                         red);
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  uint32_t slot = leaf.slot, parent = leaf.parent, tensor = leaf.tensor;
  for (;;) {
    if (lane == 0 && tensor != kNone && a.tensor_norms) a.tensor_norms[tensor] = static_cast<float>(sqrt(sum));
    if (parent == kNone) break;
    // Sums are stored and loaded at agent scope, past the XCD's own L2, and
    // each is complete before its owner counts itself; so the counter needs no
    // release, which would write back the whole L2.
    const NormNode node = a.nodes[parent];
    uint32_t before = 0;
    if (lane == 0) {
      __hip_atomic_store(&a.sums[slot], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      before = __hip_atomic_fetch_add(&a.arrived[parent].count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    before = __builtin_amdgcn_readfirstlane(before);
    if (before != node.children - 1) return;
    asm volatile("" ::: "memory");
    if (lane == 0) __hip_atomic_store(&a.arrived[parent].count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    double own[kNormChildren / 64];
#pragma unroll
    for (int k = 0; k < kNormChildren / 64; ++k) {
      const int c = lane + 64 * k;
      own[k] = c < static_cast<int>(node.children) ? load_partial(&a.sums[node.first + c]) : 0.0;
    }
    sum = own[0];
#pragma unroll
    for (int k = 1; k < kNormChildren / 64; ++k) sum += own[k];
    sum = wave_sum_f64(sum);
    slot = node.slot;
    parent = node.parent;
    tensor = node.tensor;
  }
  if (lane == 0) {
    const double norm = sqrt(sum);
    a.out[0] = static_cast<float>(norm);
    a.out[1] = norm <= a.max_norm ? 1.0f : static_cast<float>(a.max_norm / norm);
  }
}

}  // namespace

hipError_t launch_grad_norm(const NormArgs& a, hipStream_t s) {
  if (a.stream)
    hipLaunchKernelGGL(k_grad_norm<true>, dim3(a.nleaves), dim3(kNormThreads), 0, s, a);
  else
    hipLaunchKernelGGL(k_grad_norm<false>, dim3(a.nleaves), dim3(kNormThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
