// Tokens sorted by expert and back, with weights, and the gradient.
//
// A token's choice j is slot t * top + j.  The sort is stable: an expert's
// rows lie in the order of their slots, so results repeat bit for bit and no
// atomic decides a place.
#include <algorithm>

#include "expert.h"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
// Bucket of a slot: its expert, or `experts` for a number outside 0..experts-1.
template <typename I>
__device__ __forceinline__ int bucket(const I* ids, int64_t i, int experts) {
  const I id = gmem(ids)[i];
  return (id >= 0 && id < experts) ? static_cast<int>(id) : experts;
}

// counts[b][e]: slots of workgroup b with bucket e.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_expert_count(const I* ids, int slots, int per, int experts,
                                                              int32_t* counts) {
  __shared__ int hist[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * per, hi = min(slots, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&hist[bucket(ids, i, experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += kSortThreads)
    counts[static_cast<int64_t>(blockIdx.x) * (experts + 1) + e] = hist[e];
}

// Places of workgroup b's slots.  base[e] starts as the place of its first
// slot of bucket e: all slots of lower buckets, and bucket e's in the
// workgroups before.  Then 1024 slots at a time, in order: a wave finds the
// lanes with its bucket by one ballot per bit; the sixteen waves' counts are
// added up in wave order.
// ALONE: one workgroup, which counts by itself.
template <typename I, bool ALONE>
__global__ __launch_bounds__(kSortThreads) void k_expert_place(const I* ids, int slots, int per, int bits, Routes r,
                                                              const int32_t* counts) {
  constexpr int NW = kSortThreads / 64;
  __shared__ int total[kMaxExperts + 1], base[kMaxExperts + 1], wave_sum[NW];
  extern __shared__ uint16_t wave_count[];   // NW x (experts + 1), within the 1024 slots
  const int ne = r.experts + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * per, hi = min(slots, lo + per);
  for (int e = tid; e < ne; e += kSortThreads) total[e] = base[e] = 0;
  __syncthreads();
  if constexpr (ALONE) {
    for (int i = tid; i < slots; i += kSortThreads) atomicAdd(&total[bucket(ids, i, r.experts)], 1);
  } else {
    for (int e = lane; e < ne; e += 64) {
      int all = 0, before = 0;
      for (int b = wave; b < static_cast<int>(gridDim.x); b += NW) {
        const int c = gmem(counts)[static_cast<int64_t>(b) * ne + e];
        all += c;
        if (b < static_cast<int>(blockIdx.x)) before += c;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  // Exclusive sums of total (one bucket a thread, and the last one).
  {
    const int v = tid < ne ? total[tid] : 0;
    int sum = v;
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int below = 0;
    for (int w = 0; w < wave; ++w) below += wave_sum[w];
    const int first = below + sum - v;
    if (tid < ne) {
      base[tid] += first;
      if (blockIdx.x == 0) r.offsets[tid] = first;
    }
    if (ne > kSortThreads && tid == kSortThreads - 1) {
      base[kSortThreads] += first + v;
      if (blockIdx.x == 0) r.offsets[kSortThreads] = first + v;
    }
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += kSortThreads) {
    for (int e = tid; e < NW * ne; e += kSortThreads) wave_count[e] = 0;
    __syncthreads();
    const int i = i0 + tid;
    const bool in = i < hi;
    const int b = in ? bucket(ids, i, r.experts) : -1;
    uint64_t same = __ballot(in);
    for (int k = 0; k < bits; ++k) {
      const bool bit = (b >> k) & 1;
      const uint64_t v = __ballot(bit);
      same &= bit ? v : ~v;
    }
    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
    if (in && rank == 0) wave_count[wave * ne + b] = static_cast<uint16_t>(__popcll(same));
    __syncthreads();
    for (int e = tid; e < ne; e += kSortThreads) {
      int at = 0;
      for (int w = 0; w < NW; ++w) {
        const int c = wave_count[w * ne + e];
        wave_count[w * ne + e] = static_cast<uint16_t>(at);
        at += c;
      }
      total[e] = at;
    }
    __syncthreads();
    if (in) {
      const int at = base[b] + wave_count[wave * ne + b] + rank;
      const bool routed = b < r.experts;
      r.order[at] = routed ? i : -1;
      r.place[i] = routed ? at : -1;
    }
    __syncthreads();
    for (int e = tid; e < ne; e += kSortThreads) base[e] += total[e];
  }
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A run of V elements as floats: V = 16 bytes' worth, or one element (rows
// that do not lie on 16-byte borders).
template <typename T, bool VEC>
struct Run {
  static constexpr int V = VEC ? 16 / sizeof(T) : 1;
  float v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
      set(*reinterpret_cast<const MUON_GLOBAL u32x4*>(gmem(p)));
    } else if constexpr (sizeof(T) == 4) {
      v[0] = gmem(reinterpret_cast<const float*>(p))[0];
    } else {
      v[0] = bf16_to_f32(gmem(reinterpret_cast<const uint16_t*>(p))[0]);
    }
  }
  __device__ __forceinline__ void set(u32x4 u) {
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          v[e] = __uint_as_float(u[e]);
        } else {
          v[2 * e] = __uint_as_float(u[e] << 16);
          v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) u[e] = __float_as_uint(v[e]);
        else u[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      }
      *reinterpret_cast<MUON_GLOBAL u32x4*>(gmem(p)) = u;
    } else if constexpr (sizeof(T) == 4) {
      gmem(reinterpret_cast<float*>(p))[0] = v[0];
    } else {
      gmem(reinterpret_cast<uint16_t*>(p))[0] = f32_to_bf16(v[0]);
    }
  }
};

constexpr int kMoveThreads = 256;

// A row index of place[], or -1: out of range counts as unrouted.
__device__ __forceinline__ int place_of(const MoveArgs& a, int64_t slot) {
  const int p = gmem(a.place)[slot];
  return (p >= 0 && p < a.slots) ? p : -1;
}

// xs[place[t][j]] = x[t]: a thread reads one run of a token and writes it to
// every row of the token.
template <typename T, bool VEC>
__global__ __launch_bounds__(kMoveThreads) void k_expert_gather(MoveArgs a, int runs) {
  using R = Run<T, VEC>;
  const int64_t n = static_cast<int64_t>(a.tokens) * runs, step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < n; i += step) {
    const int64_t t = i / runs;
    const int col = static_cast<int>(i % runs) * R::V;
    R x;
    x.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
    for (int j = 0; j < a.top; ++j) {
      const int p = place_of(a, t * a.top + j);
      if (p >= 0) x.store(static_cast<T*>(a.rows_out) + p * a.rows_out_ld + col);
    }
  }
}

// y[t] = residual[t] + sum over j of w[t][j] ys[place[t][j]], j ascending, in
// float32, rounded once.
template <typename T, bool VEC>
__global__ __launch_bounds__(kMoveThreads) void k_expert_combine(MoveArgs a, int runs) {
  using R = Run<T, VEC>;
  const int64_t n = static_cast<int64_t>(a.tokens) * runs, step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < n; i += step) {
    const int64_t t = i / runs;
    const int col = static_cast<int>(i % runs) * R::V;
    R y;
    if (a.tok) {
      y.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
    } else {
#pragma unroll
      for (int e = 0; e < R::V; ++e) y.v[e] = 0.0f;
    }
    for (int j = 0; j < a.top; ++j) {
      const int64_t slot = t * a.top + j;
      const int p = place_of(a, slot);
      if (p < 0) continue;
      const float w = a.weights ? load_elem(a.weights, slot, a.w_dt) : 1.0f;
      R x;
      x.load(static_cast<const T*>(a.rows) + p * a.rows_ld + col);
#pragma unroll
      for (int e = 0; e < R::V; ++e) y.v[e] = __builtin_fmaf(w, x.v[e], y.v[e]);
    }
    y.store(static_cast<T*>(a.tok_out) + t * a.tok_out_ld + col);
  }
}

// dys[place[t][j]] = w[t][j] dy[t];  dw[t][j] = <dy[t], ys[place[t][j]]>: a
// workgroup per token and choice.
template <typename T, bool VEC>
__global__ __launch_bounds__(kMoveThreads) void k_expert_combine_grad(MoveArgs a, int runs) {
  using R = Run<T, VEC>;
  __shared__ float red[kMoveThreads / 64];
  for (int64_t slot = blockIdx.x; slot < a.slots; slot += gridDim.x) {
    const int64_t t = slot / a.top;
    const int p = place_of(a, slot);
    float dot = 0.0f;
    if (p >= 0) {
      const float w = load_elem(a.weights, slot, a.w_dt);
      for (int c = threadIdx.x; c < runs; c += kMoveThreads) {
        const int col = c * R::V;
        R g, x;
        g.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
        x.load(static_cast<const T*>(a.rows) + p * a.rows_ld + col);
#pragma unroll
        for (int e = 0; e < R::V; ++e) {
          dot = __builtin_fmaf(g.v[e], x.v[e], dot);
          g.v[e] *= w;
        }
        g.store(static_cast<T*>(a.rows_out) + p * a.rows_out_ld + col);
      }
    }
    dot = wave_tree_sum(dot);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) store_elem(a.dweights, slot, a.w_dt, (red[0] + red[1]) + (red[2] + red[3]));
    __syncthreads();
  }
}

template <typename T>
int runs_of(const MoveArgs& a, bool vec) {
  return vec ? a.width / static_cast<int>(16 / sizeof(T)) : a.width;
}

// Workgroups for n threads' work; longer work is walked in strides.
constexpr int64_t kMaxBlocks = int64_t{1} << 22;
int64_t blocks_of(const MoveArgs& a, int runs) {
  return std::min(kMaxBlocks, (static_cast<int64_t>(a.tokens) * runs + kMoveThreads - 1) / kMoveThreads);
}

}  // namespace

hipError_t launch_expert_sort(const void* ids, int id_bytes, const Routes& r, int32_t* counts, hipStream_t s) {
  int64_t per, blocks;
  sort_shape(r.slots, per, blocks);
  int bits = 1;
  while ((1 << bits) <= r.experts) ++bits;
  const size_t lds = sizeof(uint16_t) * (kSortThreads / 64) * (r.experts + 1);
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(kSortThreads);
#define MUON_SORT(I)                                                                                                  \
  if (blocks > 1) {                                                                                                   \
    hipLaunchKernelGGL(k_expert_count<I>, grid, threads, 0, s, static_cast<const I*>(ids), r.slots, (int)per,         \
                       r.experts, counts);                                                                            \
    hipError_t e = hipGetLastError();                                                                                 \
    if (e != hipSuccess) return e;                                                                                    \
    hipLaunchKernelGGL((k_expert_place<I, false>), grid, threads, lds, s, static_cast<const I*>(ids), r.slots,        \
                       (int)per, bits, r, counts);                                                                    \
  } else {                                                                                                            \
    hipLaunchKernelGGL((k_expert_place<I, true>), grid, threads, lds, s, static_cast<const I*>(ids), r.slots,         \
                       (int)per, bits, r, counts);                                                                    \
  }
  if (id_bytes == 8) {
    MUON_SORT(int64_t)
  } else {
    MUON_SORT(int32_t)
  }
#undef MUON_SORT
  return hipGetLastError();
}

#define MUON_MOVE(KERNEL, BLOCKS)                                                                                      \
  do {                                                                                                                 \
    if (dt == DT_BF16) {                                                                                               \
      const int runs = runs_of<uint16_t>(a, vec);                                                                      \
      const dim3 grid(static_cast<uint32_t>(BLOCKS));                                                                  \
      if (vec) hipLaunchKernelGGL((KERNEL<uint16_t, true>), grid, dim3(kMoveThreads), 0, s, a, runs);                  \
      else hipLaunchKernelGGL((KERNEL<uint16_t, false>), grid, dim3(kMoveThreads), 0, s, a, runs);                     \
    } else {                                                                                                           \
      const int runs = runs_of<float>(a, vec);                                                                         \
      const dim3 grid(static_cast<uint32_t>(BLOCKS));                                                                  \
      if (vec) hipLaunchKernelGGL((KERNEL<float, true>), grid, dim3(kMoveThreads), 0, s, a, runs);                     \
      else hipLaunchKernelGGL((KERNEL<float, false>), grid, dim3(kMoveThreads), 0, s, a, runs);                        \
    }                                                                                                                  \
    return hipGetLastError();                                                                                          \
  } while (0)

hipError_t launch_expert_gather(const MoveArgs& a, int dt, bool vec, hipStream_t s) {
  MUON_MOVE(k_expert_gather, blocks_of(a, runs));
}
hipError_t launch_expert_combine(const MoveArgs& a, int dt, bool vec, hipStream_t s) {
  MUON_MOVE(k_expert_combine, blocks_of(a, runs));
}
hipError_t launch_expert_combine_grad(const MoveArgs& a, int dt, bool vec, hipStream_t s) {
  MUON_MOVE(k_expert_combine_grad, std::min<int64_t>(kMaxBlocks, a.slots));
}
#undef MUON_MOVE

}  // namespace muon
