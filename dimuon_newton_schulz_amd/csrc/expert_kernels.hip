// Tokens sorted by expert and back, with weights, and the gradient.
//
// A token's choice j is slot t * top + j.  The sort is stable: an expert's
// rows lie in the order of their slots, so results repeat bit for bit and no
// atomic decides a place.
//
// Sort: bound by latency (a launch and a few barriers: 48 slots 3.7 us, 98304
// slots of 64 experts 12 us in two launches).  Rows: bound by memory; 16384
// tokens of six choices, 2048 bf16: gather 91 us (5.2 TB/s), combine with
// weights and residual 88 to 97 (5.5 to 6.1), its gradient 174 (5.0); a copy
// reaches 5.1 on the same card, writes alone 6.8.
#include <algorithm>
#include <type_traits>

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

// Many workgroups: counts[b][e] becomes the number of slots of bucket e in the
// workgroups before b, and the row behind the last one their number in all.
// A workgroup per bucket.
__global__ __launch_bounds__(kSortThreads) void k_expert_scan(int32_t* counts, int blocks, int ne) {
  __shared__ int wave_sum[kSortThreads / 64];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0;
  for (int b0 = 0; b0 <= blocks; b0 += kSortThreads) {
    const int b = b0 + tid;
    const int c = b < blocks ? counts[static_cast<int64_t>(b) * ne + e] : 0;
    int sum = c;
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int below = before, all = 0;
    for (int w = 0; w < kSortThreads / 64; ++w) {
      if (w < wave) below += wave_sum[w];
      all += wave_sum[w];
    }
    if (b <= blocks) counts[static_cast<int64_t>(b) * ne + e] = below + sum - c;
    before += all;
    __syncthreads();
  }
}

// Places of workgroup b's slots.  Wave w has a run of consecutive slots of its
// own, taken 64 at a time: the lanes with one bucket are found by a ballot per
// bit, and the wave's own counters (LDS, no barrier) say how many came before.
// Then the waves' counts, the workgroups' (counts[], k_expert_count) and the
// buckets' are added up, and every slot's place is its bucket's start + the
// counts before + its number within the wave.
constexpr int kSortWaves = kSortThreads / 64;
enum SortOthers { SORT_ALONE, SORT_SUMMED, SORT_SCANNED };   // no other workgroup; counts[]; k_expert_scan's

template <typename I, SortOthers OTHERS>
__global__ __launch_bounds__(kSortThreads) void k_expert_place(const I* ids, int slots, int per, int bits, Routes r,
                                                              const int32_t* counts) {
  constexpr int MOST = kSortAlone / kSortThreads;   // turns of 64 slots of a wave
  __shared__ int base[kMaxExperts + 1], totals[kMaxExperts + 1], wave_sum[kSortWaves];
  extern __shared__ uint16_t wave_count[];   // waves x (experts + 1); a wave has at most 64 * MOST slots
  const int ne = r.experts + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * per, hi = min(slots, lo + per);
  const int turns = (hi - lo + kSortThreads - 1) / kSortThreads, from = lo + wave * turns * 64;
  uint16_t* mine = wave_count + wave * ne;
  for (int e = lane; e < ne; e += 64) mine[e] = 0;
  for (int e = tid; e < ne; e += kSortThreads) base[e] = totals[e] = 0;
  int bucket_of[MOST], before[MOST];   // of the lane's slots
#pragma unroll
  for (int t = 0; t < MOST; ++t) {
    const int i = from + t * 64 + lane;
    bucket_of[t] = t < turns && i < hi ? bucket(ids, i, r.experts) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MOST; ++t) {
    if (t >= turns) break;
    const int b = bucket_of[t];
    uint64_t same = __ballot(b >= 0);
    for (int k = 0; k < bits; ++k) {
      const bool bit = (b >> k) & 1;
      const uint64_t v = __ballot(bit);
      same &= bit ? v : ~v;
    }
    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
    const int seen = b >= 0 ? mine[b] : 0;
    before[t] = seen + rank;
    // (The wave's reads of its counters come before the update, which one
    // lane of each bucket makes, and that before the next turn's reads.)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (b >= 0 && rank == 0) mine[b] = static_cast<uint16_t>(seen + __popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (OTHERS == SORT_SUMMED) {
    for (int e = lane; e < ne; e += 64) {
      int all = 0, sum = 0;
#pragma unroll 4
      for (int b = wave; b < static_cast<int>(gridDim.x); b += kSortWaves) {
        const int c = gmem(counts)[static_cast<int64_t>(b) * ne + e];
        all += c;
        sum += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
      if (all) atomicAdd(&totals[e], all);
      if (sum) atomicAdd(&base[e], sum);
    }
  } else if constexpr (OTHERS == SORT_SCANNED) {
    for (int e = tid; e < ne; e += kSortThreads) {
      base[e] = gmem(counts)[static_cast<int64_t>(blockIdx.x) * ne + e];
      totals[e] = gmem(counts)[static_cast<int64_t>(gridDim.x) * ne + e];
    }
  }
  __syncthreads();
  // Thread e < ne: the waves' counts become what came before them; the
  // bucket's slots in all.
  int total = 0;
  for (int e = tid; e < ne; e += kSortThreads) {
    int at = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = wave_count[w * ne + e];
      wave_count[w * ne + e] = static_cast<uint16_t>(at);
      at += c;
    }
    if (e == tid) total = OTHERS == SORT_ALONE ? at : totals[e];
  }
  // Exclusive sums over the buckets (one a thread; bucket 1024, of the
  // unrouted slots, starts where the last thread's ends).
  int sum = total;
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  int below = 0;
  for (int w = 0; w < wave; ++w) below += wave_sum[w];
  const int first = below + sum - total;
  auto start = [&](int e, int at) {
    base[e] += at;
    if (blockIdx.x == 0) r.offsets[e] = at;
  };
  if (tid < ne) start(tid, first);
  if (ne > kSortThreads && tid == kSortThreads - 1) start(kSortThreads, first + total);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MOST; ++t) {
    const int b = bucket_of[t];
    if (b < 0) continue;
    const int i = from + t * 64 + lane, at = base[b] + mine[b] + before[t];
    const bool routed = b < r.experts;
    r.order[at] = routed ? i : -1;
    r.place[i] = routed ? at : -1;
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
  using Raw = typename std::conditional<VEC, u32x4, T>::type;   // as loaded
  float v[V];
  // Rows that are read once, past the caches' lines in use.
  static __device__ __forceinline__ Raw read_once(const T* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const MUON_GLOBAL Raw*>(gmem(p)));
  }
  static __device__ __forceinline__ Raw read(const T* p) {
    return *reinterpret_cast<const MUON_GLOBAL Raw*>(gmem(p));
  }
  __device__ __forceinline__ void load(const T* p) { set(read(p)); }
  __device__ __forceinline__ void set(Raw u) {
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
    } else if constexpr (sizeof(T) == 4) {
      v[0] = u;
    } else {
      v[0] = bf16_to_f32(u);
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

// Choices of a token that are handled at once, their rows' loads in flight together.
constexpr int kAtOnce = 8;

// Places (and weights) of the choices j0 .. j0 + N - 1 of the token whose slots
// start at `slot0`; -1 where there is none.
template <int N>
__device__ __forceinline__ void places_of(const MoveArgs& a, int64_t slot0, int j0, int (&p)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) p[j] = j0 + j < a.top ? place_of(a, slot0 + j0 + j) : -1;
}
template <int N>
__device__ __forceinline__ void weights_of(const MoveArgs& a, int64_t slot0, int j0, float (&w)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    w[j] = j0 + j < a.top && a.weights ? load_elem(a.weights, slot0 + j0 + j, a.w_dt) : 1.0f;
}

// xs[place[t][j]] = x[t]: a thread reads one run of a token and writes it to
// every row of the token (rows in their own order, each reading its token,
// take 40% longer: the training batch's 403 MB 130 instead of 91 us).
template <typename T, bool VEC>
__global__ __launch_bounds__(kMoveThreads) void k_expert_gather(MoveArgs a, int runs) {
  using R = Run<T, VEC>;
  const int64_t n = static_cast<int64_t>(a.tokens) * runs, step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < n; i += step) {
    const int64_t t = i / runs;
    const int col = static_cast<int>(i - t * runs) * R::V;
    R x;
    x.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
    for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
      int p[kAtOnce];
      places_of(a, t * a.top, j0, p);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (p[j] >= 0) x.store(static_cast<T*>(a.rows_out) + p[j] * a.rows_out_ld + col);
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
    const int col = static_cast<int>(i - t * runs) * R::V;
    R y;
    if (a.tok) {
      y.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
    } else {
#pragma unroll
      for (int e = 0; e < R::V; ++e) y.v[e] = 0.0f;
    }
    for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
      int p[kAtOnce];
      float w[kAtOnce];
      typename R::Raw x[kAtOnce];
      places_of(a, t * a.top, j0, p);
      weights_of(a, t * a.top, j0, w);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (p[j] >= 0) x[j] = R::read_once(static_cast<const T*>(a.rows) + p[j] * a.rows_ld + col);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (p[j] < 0) continue;
        R v;
        v.set(x[j]);
#pragma unroll
        for (int e = 0; e < R::V; ++e) y.v[e] = __builtin_fmaf(w[j], v.v[e], y.v[e]);
      }
    }
    y.store(static_cast<T*>(a.tok_out) + t * a.tok_out_ld + col);
  }
}

// dys[place[t][j]] = w[t][j] dy[t];  dw[t][j] = <dy[t], ys[place[t][j]]>: WPT
// waves per token (four for wide rows, one for narrow ones) and N of its
// choices (all together where tokens are many; one, where that many waves
// would not fill the GPU).
template <typename T, bool VEC, int WPT, int N>
__global__ __launch_bounds__(kMoveThreads) void k_expert_combine_grad(MoveArgs a, int runs) {
  using R = Run<T, VEC>;
  constexpr int TPW = kMoveThreads / 64 / WPT, LANES = 64 * WPT;   // tokens of a workgroup, threads of a token
  __shared__ float red[N][kMoveThreads / 64];
  const int wave = threadIdx.x >> 6, thread = threadIdx.x % LANES, j0 = blockIdx.y * N;
  const int64_t groups = (static_cast<int64_t>(a.tokens) + TPW - 1) / TPW;
  for (int64_t b = blockIdx.x; b < groups; b += gridDim.x) {
    const int64_t t = b * TPW + wave / WPT;
    const bool in = t < a.tokens;
    float dot[N];
#pragma unroll
    for (int j = 0; j < N; ++j) dot[j] = 0.0f;
    if (in) {
      int p[N];
      float w[N];
      places_of(a, t * a.top, j0, p);
      weights_of(a, t * a.top, j0, w);
      for (int c = thread; c < runs; c += LANES) {
        const int col = c * R::V;
        R g;
        typename R::Raw x[N];
        g.load(static_cast<const T*>(a.tok) + t * a.tok_ld + col);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (p[j] >= 0) x[j] = R::read(static_cast<const T*>(a.rows) + p[j] * a.rows_ld + col);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (p[j] < 0) continue;
          R v;
          v.set(x[j]);
#pragma unroll
          for (int e = 0; e < R::V; ++e) {
            dot[j] = __builtin_fmaf(g.v[e], v.v[e], dot[j]);
            v.v[e] = g.v[e] * w[j];
          }
          v.store(static_cast<T*>(a.rows_out) + p[j] * a.rows_out_ld + col);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      dot[j] = wave_tree_sum(dot[j]);
      if (WPT > 1 && (threadIdx.x & 63) == 0) red[j][wave] = dot[j];
    }
    if constexpr (WPT > 1) __syncthreads();
    if (thread < N && in && j0 + thread < a.top) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float v = dot[j];
        if constexpr (WPT > 1) {
          v = red[j][wave / WPT * WPT];
#pragma unroll
          for (int w = 1; w < WPT; ++w) v += red[j][wave / WPT * WPT + w];
        }
        s = j == thread ? v : s;
      }
      store_elem(a.dweights, t * a.top + j0 + thread, a.w_dt, s);
    }
    if constexpr (WPT > 1) __syncthreads();
  }
}

template <typename T>
int runs_of(const MoveArgs& a, bool vec) {
  return vec ? a.width / static_cast<int>(16 / sizeof(T)) : a.width;
}

// Workgroups for n threads' work; longer work is walked in strides.
constexpr int64_t kMaxBlocks = int64_t{1} << 22;
int64_t blocks_of(int64_t rows, int runs) {
  return std::min(kMaxBlocks, (rows * runs + kMoveThreads - 1) / kMoveThreads);
}

}  // namespace

hipError_t launch_expert_sort(const void* ids, int id_bytes, const Routes& r, int32_t* counts, hipStream_t s) {
  int64_t per, blocks;
  sort_shape(r.slots, per, blocks);
  int bits = 1;
  while ((1 << bits) <= r.experts) ++bits;
  const size_t lds = sizeof(uint16_t) * (kSortThreads / 64) * (r.experts + 1);
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(kSortThreads);
  const int n = static_cast<int>(per);
#define MUON_SORT(I)                                                                                                  \
  do {                                                                                                                \
    const I* p = static_cast<const I*>(ids);                                                                          \
    if (blocks > 1)                                                                                                   \
      hipLaunchKernelGGL(k_expert_count<I>, grid, threads, 0, s, p, r.slots, n, r.experts, counts);                   \
    if (blocks > kSortSummed)                                                                                         \
      hipLaunchKernelGGL(k_expert_scan, dim3(r.experts + 1), threads, 0, s, counts, (int)blocks, r.experts + 1);      \
    if (blocks == 1)                                                                                                  \
      hipLaunchKernelGGL((k_expert_place<I, SORT_ALONE>), grid, threads, lds, s, p, r.slots, n, bits, r, counts);     \
    else if (blocks <= kSortSummed)                                                                                   \
      hipLaunchKernelGGL((k_expert_place<I, SORT_SUMMED>), grid, threads, lds, s, p, r.slots, n, bits, r, counts);    \
    else                                                                                                              \
      hipLaunchKernelGGL((k_expert_place<I, SORT_SCANNED>), grid, threads, lds, s, p, r.slots, n, bits, r, counts);   \
  } while (0)
  if (id_bytes == 8) {
    MUON_SORT(int64_t);
  } else {
    MUON_SORT(int32_t);
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
  MUON_MOVE(k_expert_gather, blocks_of(a.tokens, runs));
}
hipError_t launch_expert_combine(const MoveArgs& a, int dt, bool vec, hipStream_t s) {
  MUON_MOVE(k_expert_combine, blocks_of(a.tokens, runs));
}
hipError_t launch_expert_combine_grad(const MoveArgs& a, int dt, bool vec, hipStream_t s) {
  const bool wide = a.width / (vec ? (dt == DT_BF16 ? 8 : 4) : 1) > 128;
  const int64_t blocks = std::min<int64_t>(kMaxBlocks, wide ? a.tokens : (a.tokens + 3) / 4);
  // (One by one against together: 1009 tokens of three choices, 769 float32,
  // 6.7 us against 7.7; 2048 of six, 2048 bf16, 17.4 against 20.0; 8192 of
  // four, 96 bf16, 8.0 against 9.2; 16384 of six, 2048 bf16, 178 against 171.)
  const bool one = blocks <= 2048;
  const int n = one ? 1 : kAtOnce;
  const dim3 grid(static_cast<uint32_t>(blocks), static_cast<uint32_t>((a.top + n - 1) / n));
#define MUON_GRAD(T, VEC)                                                                                              \
  do {                                                                                                                 \
    const int runs = runs_of<T>(a, VEC);                                                                               \
    if (wide && one)                                                                                                   \
      hipLaunchKernelGGL((k_expert_combine_grad<T, VEC, 4, 1>), grid, dim3(kMoveThreads), 0, s, a, runs);              \
    else if (wide)                                                                                                     \
      hipLaunchKernelGGL((k_expert_combine_grad<T, VEC, 4, kAtOnce>), grid, dim3(kMoveThreads), 0, s, a, runs);        \
    else if (one)                                                                                                      \
      hipLaunchKernelGGL((k_expert_combine_grad<T, VEC, 1, 1>), grid, dim3(kMoveThreads), 0, s, a, runs);              \
    else                                                                                                               \
      hipLaunchKernelGGL((k_expert_combine_grad<T, VEC, 1, kAtOnce>), grid, dim3(kMoveThreads), 0, s, a, runs);        \
  } while (0)
  if (dt == DT_BF16) {
    if (vec) MUON_GRAD(uint16_t, true); else MUON_GRAD(uint16_t, false);
  } else {
    if (vec) MUON_GRAD(float, true); else MUON_GRAD(float, false);
  }
#undef MUON_GRAD
  return hipGetLastError();
}
#undef MUON_MOVE

}  // namespace muon
