// Products over groups of rows, with bias, activation and residual, and their
// gradients.  Group g holds the rows offsets[g] .. offsets[g+1]-1 and has a
// weight W_g (out x in) of its own; a plain layer is one group.
//
//   forward        C(m, n) = sum_k x[m][k] W[n][k]     k-contiguous operands
//   input gradient C(m, n) = sum_k dz[m][k] W[k][n]    W k-major
//   weight gradient C(m, n) = sum_k dz[k][m] x[k][n]   both k-major, k the group's rows
//
// A BM x BN tile per workgroup; both operands go from global memory straight
// into a ring of LDS units, stages of 128 bytes of k per row (64 bf16 or 32
// float32 values; whole lines: half lines cost the forward product 10%).
// Buffer loads carry the bounds: their descriptor ends with the operand, so
// that rows behind a group's last one, columns behind the matrix and the
// ragged end of k arrive as zeros and no operand is padded.  The products run
// with W's (or x's) fragment first, so that a lane holds runs of four output
// columns of one row.
//
// What bounds the large tiles (256 x 256, four waves of 128 x 128, one per
// SIMD): per stage and CU 2048 cycles of MFMA, 1024 of fragment reads and 512
// of loads into LDS.  Eight waves of 128 x 64 read half as much again and
// were held by the LDS.  The products are 16 x 16 x 32 (5% faster than
// 32 x 32 x 16: half the accumulator traffic), and every step's order is
// given (pace): without it the compiler put a step's reads behind its
// products, before the wait.  A ring of five units gives one operand two
// stages' time to arrive (8 to 23% of the time at 8192^3).  8192^3 bf16 takes
// 750 us, forward and for either gradient (the library's: 680, 791, 918).  The
// GPU holds about 1.6 GHz there, the matrix units busy 73% of cycles.  A round
// of tiles takes 21 us per 1024 of k, and beside its k 8 to 12 us for the sums
// alone, 15 with an activation, 19 with a residual, 18 added to what dW holds
// and 25 through x_pre.
#include <algorithm>
#include <type_traits>

#include "expert.h"
#include "muon_mi355x.h"

namespace muon {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

#define MUON_LDS __attribute__((address_space(3)))

constexpr uint32_t kNowhere = 0x80000000u;   // an offset behind every descriptor's end

// ---------------------------------------------------------------------------
// Activations, in float32.
// ---------------------------------------------------------------------------
// z Phi(z), with Phi from the complementary error function: no cancellation for negative z.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }
// (1 + tanh(u)) / 2 = sigmoid(2u)
constexpr float kTanhScale = 2.0f * 0.79788456080286536f, kTanhCubic = 0.044715f;

// EXACT (float32 outputs): expf and a true quotient; otherwise the hardware's
// exponential and reciprocal, 1 ulp each (z log2 e rounds to 2^-24 z, so the
// exponential is off by at most 2^-24 |z| + 2 ulps, far below a bf16 step).
template <bool EXACT>
__device__ __forceinline__ float over_one_plus_exp(float z, float u) {   // z / (1 + exp(-u))
  if constexpr (EXACT) return z / (1.0f + expf(-u));
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * u));
}

// The slope's argument: beyond 100 every slope is 0 or 1 in float32, and the
// formulas would multiply 0 by infinity further out; NaN stays.
__device__ __forceinline__ float within_100(float z) { return z > 100.0f ? 100.0f : (z < -100.0f ? -100.0f : z); }

template <int ACT, bool EXACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == LINEAR_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == LINEAR_SILU) return over_one_plus_exp<EXACT>(z, z);
  if constexpr (ACT == LINEAR_GELU) return z * normal_cdf(z);
  return over_one_plus_exp<EXACT>(z, kTanhScale * (z + kTanhCubic * z * z * z));
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float slope(float z) {
  z = within_100(z);
  if constexpr (ACT == LINEAR_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == LINEAR_SILU) {
    const float s = over_one_plus_exp<EXACT>(1.0f, z);
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (ACT == LINEAR_GELU) return normal_cdf(z) + z * 0.39894228040143268f * expf(-0.5f * z * z);
  const float s = over_one_plus_exp<EXACT>(1.0f, kTanhScale * (z + kTanhCubic * z * z * z));
  return s + z * s * (1.0f - s) * kTanhScale * (1.0f + 3.0f * kTanhCubic * z * z);
}

// v = act(v), and v *= act'(z): one branch for H runs of N values.
template <bool EXACT, int H, int N>
__device__ __forceinline__ void activate_runs(int act, float (&v)[H][N]) {
#define MUON_EACH(ACT)            \
  case ACT:                       \
    _Pragma("unroll")             \
    for (int e = 0; e < H * N; ++e) v[e / N][e % N] = activate<ACT, EXACT>(v[e / N][e % N]); \
    break
  switch (act) {
    MUON_EACH(LINEAR_RELU);
    MUON_EACH(LINEAR_SILU);
    MUON_EACH(LINEAR_GELU);
    MUON_EACH(LINEAR_GELU_TANH);
    default: break;
  }
#undef MUON_EACH
}
template <bool EXACT, int H, int N>
__device__ __forceinline__ void times_slopes(int act, const float (&z)[H][N], float (&v)[H][N]) {
#define MUON_EACH(ACT)            \
  case ACT:                       \
    _Pragma("unroll")             \
    for (int e = 0; e < H * N; ++e) v[e / N][e % N] *= slope<ACT, EXACT>(z[e / N][e % N]); \
    break
  switch (act) {
    MUON_EACH(LINEAR_RELU);
    MUON_EACH(LINEAR_SILU);
    MUON_EACH(LINEAR_GELU);
    MUON_EACH(LINEAR_GELU_TANH);
    default: break;
  }
#undef MUON_EACH
}

// ---------------------------------------------------------------------------
// Work of a workgroup
// ---------------------------------------------------------------------------
struct Group {
  int index, lo, hi;   // rows lo .. hi-1
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Workgroups are dealt to the 8 XCDs in turn; runs of `run` neighbouring
// tiles, which share operand panels, go to one XCD and so one L2.
// `turn`: every other round of runs goes to the XCDs in reverse, so that runs
// in order of falling work even out.
__device__ __forceinline__ int tile_of(int bid, int run, bool turn) {
  const int i = bid >> 3, round = i / run;
  const int xcd = turn && (round & 1) ? 7 - (bid & 7) : bid & 7;
  return (round * 8 + xcd) * run + i % run;
}

// Tile idx of the list that has every group's tiles of bm rows x nt columns
// after another: its group and number within the group.  False behind the
// last tile.  The groups' tiles are added up 64 groups at a time over the
// lanes of a wave.
__device__ __forceinline__ bool find_rows(const LinArgs& a, int idx, int bm, int nt, Group& g, int& local) {
  if (!a.offsets) {
    g = {0, 0, a.rows};
    local = idx;
    return idx < (a.rows + bm - 1) / bm * nt;
  }
  const int lane = threadIdx.x & 63;
  const MUON_GLOBAL int32_t* off = gmem(a.offsets);
  int before = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64) {
    const int i = g0 + lane;
    int lo = 0, hi = 0;
    if (i < a.groups) {
      lo = clamped(off[i], 0, a.rows);
      hi = clamped(off[i + 1], lo, a.rows);
    }
    const int tiles = (hi - lo + bm - 1) / bm * nt;
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t past = __ballot(before + sum > idx);
    if (past) {
      const int l = __builtin_ctzll(past);
      g.index = g0 + l;
      g.lo = __builtin_amdgcn_readlane(lo, l);
      g.hi = __builtin_amdgcn_readlane(hi, l);
      local = idx - (before + __builtin_amdgcn_readlane(sum - tiles, l));
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// The group with the p-th most rows, of at most kRanked groups (ties: the
// lower number first): a wave ranks them all.
constexpr int kRanked = 128;
__device__ __forceinline__ int group_by_size(const LinArgs& a, int p) {
  const int lane = threadIdx.x & 63;
  const MUON_GLOBAL int32_t* off = gmem(a.offsets);
  int n[kRanked / 64], rank[kRanked / 64];
#pragma unroll
  for (int j = 0; j < kRanked / 64; ++j) {
    const int g = 64 * j + lane;
    n[j] = -1;
    rank[j] = 0;
    if (g < a.groups) {
      const int lo = clamped(off[g], 0, a.rows);
      n[j] = clamped(off[g + 1], lo, a.rows) - lo;
    }
  }
#pragma unroll
  for (int h = 0; h < kRanked / 64; ++h)
    if (64 * h < a.groups)
      for (int l = 0; l < 64; ++l) {
        const int other = __builtin_amdgcn_readlane(n[h], l), g = 64 * h + l;
#pragma unroll
        for (int j = 0; j < kRanked / 64; ++j)
          rank[j] += other > n[j] || (other == n[j] && g < 64 * j + lane) ? 1 : 0;
      }
#pragma unroll
  for (int j = 0; j < kRanked / 64; ++j) {
    const uint64_t hit = __ballot(rank[j] == p);
    if (hit) return 64 * j + __builtin_ctzll(hit);
  }
  return p;
}

// Tile `local` of mt x nt: blocks of up to eight row tiles by all columns,
// rows first, so that neighbours share panels of both operands.
__device__ __forceinline__ void block_order(int local, int mt, int nt, int& rt, int& ct) {
  const int per = 8 * nt, b = local / per, r = local - b * per, rows = min(8, mt - 8 * b);
  rt = 8 * b + r % rows;
  ct = r / rows;
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
// WR x WC waves, each with (BM / WR) x (BN / WC) of the tile in 16 x 16
// blocks.  Stages have KB = 128 bytes of k of every row; a ring of U units
// holds the stages' operands in turn, P_0 Q_0 P_1 Q_1 ..., so that with five
// units one operand's loads have two stages' time to arrive.
template <int BM_, int BN_, int WR_, int WC_, int U_, int UNIT_ = (BM_ > BN_ ? BM_ : BN_) * 128>
struct Geo {
  static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_, U = U_, UNIT = UNIT_;   // UNIT: bytes
  static constexpr int NW = WR * WC, NT = 64 * NW, WM = BM / WR, WN = BN / WC, MS = WM / 16, NS = WN / 16;
  // A wave's strip of 32 output rows (where they lie on no 16-byte borders).
  static constexpr int SP = WN + 4, STRIP = 32 * SP * 4;
};
constexpr int KB = 128, NQ = 2;   // a stage's k: bytes, and steps of 32 (bf16) or 16 (f32) values

// k-contiguous operand, rows of KB bytes: 16-byte chunk c of row r sits in
// slot c ^ swz(r), so that the 16 rows of a fragment read's phase fall on
// distinct banks.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
// k-major operand, k-rows of B values: 16-byte chunk c of k-row r sits in slot
// c ^ kswz(r).  bf16: the four k-rows of a transposing read (32 bytes of each),
// and those of the 16 lanes beside, eight k-rows on, on distinct banks; float32: the k-rows of a wave's four quarters.
template <bool F32, int B>
__device__ __forceinline__ int kswz(int row) {
  static_assert(B % 128 == 0 || B == 64, "k-rows of whole 64-bank lines, or half of one");
  if constexpr (F32) return 4 * ((row >> 2) & 3);
  return (B == 64 ? 2 : 4) * (row & 3) ^ 2 * ((row >> 3) & 1);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// One operand of a tile: B rows (or columns, k-major) of which `valid` exist.
// AL: bytes of a load.  16: rows on 16-byte borders; 4: on 4-byte borders
// (every float32 matrix); 2: element by element through registers.
template <bool F32, bool KM, int B, int NT, int AL>
struct Operand {
  static constexpr int ES = F32 ? 4 : 2, LBK = KB / ES;
  static constexpr int LINE = KM ? B * ES : KB;            // bytes of an LDS row
  static constexpr int W = AL == 2 ? 16 : AL;              // bytes a thread stages at a time
  static constexpr int L = B * KB / W / NT, PER = LINE / W;   // pieces per thread and unit, and per row
  static_assert(L * NT * W == B * KB && (W != 16 || NT / 8 % 16 == 0), "whole pieces; one swizzle for a thread's rows");
  const char* base;
  uint32_t ld;         // bytes
  int valid, k;
  uint32_t off[L];     // of this thread's pieces within a stage

  // LDS row and byte within the operand's row of piece q.
  static __device__ __forceinline__ void piece(int q, int& row, int& byte) {
    const int i = q * NT + threadIdx.x;
    row = i / PER;
    const int at = i % PER * W, c = (at >> 4) ^ (KM ? kswz<F32, B>(row) : swz(row));
    byte = c * 16 + (at & 15);
  }

  __device__ __forceinline__ Operand(const void* p, int64_t ld_elems, int valid_, int k_)
      : base(static_cast<const char*>(p)), ld(static_cast<uint32_t>(ld_elems * ES)), valid(valid_), k(k_) {
#pragma unroll
    for (int q = 0; q < L; ++q) {
      int r, b;
      piece(q, r, b);
      off[q] = !KM || b < valid * ES ? r * ld + b : kNowhere;
    }
  }

  // Loads of stage st into `buf`.
  __device__ __forceinline__ void issue(int st, char* buf) const {
    const int left = k - st * LBK, here = left < LBK ? left : LBK;
    const char* p = base + (KM ? static_cast<uint64_t>(st) * LBK * ld : static_cast<uint64_t>(st) * KB);
    // (Behind the last stage nothing is read: the descriptor is empty.)
    const uint32_t end = here <= 0 ? 0 : KM ? (here - 1) * ld + valid * ES : (valid - 1) * ld + here * ES;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, end, 0x00020000);
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < L; ++q) {
      uint32_t o = off[q];
      // The ragged end of k: what lies behind it is the next row.
      if (!KM) {
        int r, b;
        piece(W == 16 ? 0 : q, r, b);   // (16-byte pieces: the same chunk in all of the thread's rows)
        o = b < here * ES ? o : kNowhere;
      }
      MUON_LDS void* to = (MUON_LDS void*)(buf + (q * NT + wave * 64) * W);
      if constexpr (W == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 16, o, 0, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 4, o, 0, 0, 0);
    }
  }

  // AL = 2: through registers.
  __device__ __forceinline__ void fetch(int st, u32x4_t (&f)[L]) const {
    const int left = k - st * LBK;
    const char* p = base + (KM ? static_cast<uint64_t>(st) * LBK * ld : static_cast<uint64_t>(st) * KB);
#pragma unroll
    for (int q = 0; q < L; ++q) {
      int r, b;
      piece(q, r, b);
      const int rows = KM ? left : valid, bytes = (KM ? valid : left) * ES;
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = 0;
        if (r < rows && b + 2 * e < bytes)
          v[e] = gmem(reinterpret_cast<const uint16_t*>(p + static_cast<uint64_t>(r) * ld + b))[e];
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) f[q][w] = v[2 * w] | (v[2 * w + 1] << 16);
    }
  }
  __device__ __forceinline__ void put(const u32x4_t (&f)[L], char* buf) const {
#pragma unroll
    for (int q = 0; q < L; ++q) *reinterpret_cast<u32x4_t*>(buf + (q * NT + threadIdx.x) * 16) = f[q];
  }
};

// Fragments of k-step q of N blocks of 16 rows from row0 on.  bf16: lane l
// holds k = 32q + 8 (l / 16) + 0..7 of row l mod 16; float32: k = 16q +
// 4 (l / 16) + 0..3 (element e of both operands is the lane's k-slot of the
// e-th of four products).
template <bool F32, bool KM, int B, int N>
__device__ __forceinline__ void read_frags(const char* buf, int row0, int q, u32x4_t (&f)[N]) {
  const int lane = threadIdx.x & 63, m16 = lane & 15, g16 = lane >> 4;
  if constexpr (!KM) {
    const char* p = buf + (row0 + m16) * KB + (((4 * q + g16) ^ swz(m16)) * 16);
#pragma unroll
    for (int t = 0; t < N; ++t) f[t] = *reinterpret_cast<const u32x4_t*>(p + t * 16 * KB);
  } else if constexpr (F32) {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * q + 4 * g16 + e, col = row0 + t * 16 + m16;
        f[t][e] = *reinterpret_cast<const uint32_t*>(buf + r * B * 4 + ((((col >> 2) ^ kswz<true, B>(r)) << 2) + (col & 3)) * 4);
      }
  } else {
    // Two transposing reads a block: in each group of 16 lanes, lane m
    // receives column m's values of four k-rows, of which lane i reads the
    // four columns 4 (i mod 4) of k-row i / 4.
    const int r = 32 * q + 8 * g16 + (m16 >> 2), sw = kswz<false, B>(r);
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const int col = row0 + t * 16 + 4 * (m16 & 3);
      const char* p = buf + r * B * 2 + ((((col >> 3) ^ sw) << 3) + (col & 7)) * 2;
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS i16x4_t*)(p));
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS i16x4_t*)(p + 4 * B * 2));
      f[t] = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
}

// Fragments read from LDS are in registers at this point of the program (an
// LDS read is otherwise free to move behind the barrier that lets the other
// waves refill its buffer).
template <int N>
__device__ __forceinline__ void in_registers(u32x4_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(r[i]));
}

template <bool F32, int MS, int NS>
__device__ __forceinline__ void multiply(const u32x4_t (&fp)[MS], const u32x4_t (&fq)[NS], f32x4_t (&acc)[MS][NS]) {
#pragma unroll
  for (int s = 0; s < MS; ++s)
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[s][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fq[t][e]), __uint_as_float(fp[s][e]),
                                                           acc[s][t], 0, 0, 0);
      } else {
        acc[s][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fq[t]),
                                                            __builtin_bit_cast(bf16x8_t, fp[s]), acc[s][t], 0, 0, 0);
      }
    }
}

// Order of a k-step's instructions: the next step's fragments are read between
// its first products, so that they are there when it ends, and the loads go
// out between the later ones.
template <bool F32, bool PKM, bool QKM, typename G, int LOADS>
__device__ __forceinline__ void pace() {
  constexpr int M = G::MS * G::NS * (F32 ? 4 : 1), H = M / 2;   // products
  constexpr int R = G::MS * (PKM ? (F32 ? 4 : 2) : 1) + G::NS * (QKM ? (F32 ? 4 : 2) : 1);   // reads
#pragma unroll
  for (int i = 0; i < H; ++i) {
#pragma unroll
    for (int j = i * R / H; j < (i + 1) * R / H; ++j) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < M - H; ++i) {
#pragma unroll
    for (int j = i * LOADS / (M - H); j < (i + 1) * LOADS / (M - H); ++j)
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
}

// acc += P Q over k.
template <bool F32, bool PKM, bool QKM, typename G, int AL>
__device__ __forceinline__ void product(const Operand<F32, PKM, G::BM, G::NT, AL>& P,
                                        const Operand<F32, QKM, G::BN, G::NT, AL>& Q, int k, char* const (&ring)[G::U],
                                        int row_p, int row_q, f32x4_t (&acc)[G::MS][G::NS]) {
  constexpr int LBK = KB / (F32 ? 4 : 2), U = G::U;
  const int nk = (k + LBK - 1) / LBK;
  if (nk == 0) return;
  u32x4_t fp[2][G::MS], fq[2][G::NS];
  auto read = [&](const char* bp, const char* bq, int q) {
    read_frags<F32, PKM, G::BM, G::MS>(bp, row_p, q, fp[q & 1]);
    read_frags<F32, QKM, G::BN, G::NS>(bq, row_q, q, fq[q & 1]);
  };
  auto mul = [&](int q) { multiply<F32, G::MS, G::NS>(fp[q & 1], fq[q & 1], acc); };
  constexpr int LP = G::BM * KB / (AL == 2 ? 16 : AL) / G::NT, LQ = G::BN * KB / (AL == 2 ? 16 : AL) / G::NT;
  if constexpr (AL == 2) {
    u32x4_t rp[LP], rq[LQ];
    P.fetch(0, rp);
    Q.fetch(0, rq);
    for (int st = 0; st < nk; ++st) {
      __syncthreads();
      P.put(rp, ring[0]);
      Q.put(rq, ring[1]);
      __syncthreads();
      if (st + 1 < nk) {
        P.fetch(st + 1, rp);
        Q.fetch(st + 1, rq);
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        read(ring[0], ring[1], q);
        mul(q);
      }
    }
  } else {
    static_assert(NQ % 2 == 0, "fragment sets alternate");
    // Loads of this wave in units first .. U-1 of the order P Q P Q ...
    constexpr auto loads_from = [](int first) {
      int n = 0;
      for (int u = first; u < U; ++u) n += u % 2 ? LQ : LP;
      return n;
    };
    auto issue = [&](int st, int operand, char* buf) {
      if (operand == 0) P.issue(st, buf);
      else Q.issue(st, buf);
    };
    // The stage's reads are complete and the next stage has landed, the loads
    // behind it still in flight: behind this point the stage's units may be
    // refilled.
    auto sync = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      in_registers(fp[(NQ - 1) & 1]);
      in_registers(fq[(NQ - 1) & 1]);
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      wait_vm<loads_from(4)>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      issue(u / 2, u % 2, ring[u]);
      if (u % 2) __builtin_amdgcn_s_barrier();   // every wave's loads of a stage go out before any of the next
    }
    wait_vm<loads_from(2)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    read(ring[0], ring[1], 0);
#pragma unroll
    for (int q = 1; q < NQ; ++q) {
      read(ring[0], ring[1], q);
      mul(q - 1);
    }
    sync();
    // From the sync after stage st to the next one: its units (c0, c1) take
    // the U-th and U+1-st units behind them (U odd: Q first), while its last
    // step and the next stage's (units n0, n1) others are multiplied.
    constexpr bool ODD = U % 2;
    auto step = [&](char* c0, char* c1, const char* n0, const char* n1, int st) {
      read(n0, n1, 0);
      issue(st + U / 2, ODD, c0);
      mul(NQ - 1);
      pace<F32, PKM, QKM, G, ODD ? LQ : LP>();
      read(n0, n1, 1);
      issue(st + U / 2 + ODD, !ODD, c1);
      mul(0);
      pace<F32, PKM, QKM, G, ODD ? LP : LQ>();
#pragma unroll
      for (int q = 2; q < NQ; ++q) {
        read(n0, n1, q);
        mul(q - 1);
        pace<F32, PKM, QKM, G, 0>();
      }
      sync();
    };
    constexpr int PERIOD = ODD ? U : U / 2;   // stages until the units' order repeats
    for (int st = 0; st < nk - 1; st += PERIOD) {
#pragma unroll
      for (int b = 0; b < PERIOD; ++b) {
        if (st + b >= nk - 1) break;
        step(ring[2 * b % U], ring[(2 * b + 1) % U], ring[(2 * b + 2) % U], ring[(2 * b + 3) % U], st + b);
      }
    }
    mul(NQ - 1);
    // No load may still be writing the ring when the epilogue uses it.
    wait_vm<0>();
  }
}

// Eight values of one (bf16) or two 16-byte loads.
template <int W>
__device__ __forceinline__ void unpack8(const u32x4_t (&u)[W], bool f32, float (&v)[8]) {
  if (W == 2 && f32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float(u[0][e]);
      v[4 + e] = __uint_as_float(u[W - 1][e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[0][e] << 16);
      v[2 * e + 1] = __uint_as_float(u[0][e] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  u32x4_t u;
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  return u;
}
// Lanes 8-15 of each row of 16 take u[1] of the lane eight below, lanes 0-7
// u[0] of the lane eight above (its own inverse).
__device__ __forceinline__ void exchange8(u32x4_t (&u)[2]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int x = static_cast<int>(u[0][e]), y = static_cast<int>(u[1][e]);
    u[0][e] = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false));   // row_ror:8
    u[1][e] = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false));
  }
}
__device__ __forceinline__ void store8(void* p, const float (&v)[8], bool f32) {
  MUON_GLOBAL u32x4_t* q = reinterpret_cast<MUON_GLOBAL u32x4_t*>(gmem(static_cast<char*>(p)));
  if (f32) {
    u32x4_t a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __float_as_uint(v[e]);
      b[e] = __float_as_uint(v[4 + e]);
    }
    q[0] = a;
    q[1] = b;
  } else {
    q[0] = pack8(v);
  }
}

// A run of N values from element `at` on: eight on 16-byte borders, or one.
template <int N>
__device__ __forceinline__ void load_run(const void* p, int64_t at, bool f32, float (&v)[N]) {
  if constexpr (N == 8) {
    const MUON_GLOBAL u32x4_t* q =
        reinterpret_cast<const MUON_GLOBAL u32x4_t*>(gmem(static_cast<const char*>(p) + at * (f32 ? 4 : 2)));
    u32x4_t u[2] = {q[0], q[0]};
    if (f32) u[1] = q[1];
    unpack8(u, f32, v);
  } else {
    v[0] = load_elem(p, at, f32 ? DT_F32 : DT_BF16);
  }
}
template <int N>
__device__ __forceinline__ void store_run(void* p, int64_t at, bool f32, const float (&v)[N]) {
  if constexpr (N == 8) store8(static_cast<char*>(p) + at * (f32 ? 4 : 2), v, f32);
  else store_elem(p, at, f32 ? DT_F32 : DT_BF16, v[0]);
}

// What a product's result is combined with, element by element: the residual
// (forward), x_pre (input gradient), what dW holds (weight gradient,
// accumulated).
template <bool F32, int MODE>
struct Old {
  const void* p;   // NULL: none
  int64_t ld, at;
  bool f32;
  __device__ __forceinline__ Old(const LinArgs& a, int g) {
    if constexpr (MODE == LIN_WEIGHT) {
      p = a.accumulate && a.parts == 1 ? a.c : nullptr;
      ld = a.ldc;
      at = g * a.gc;
      f32 = a.c_dt == DT_F32;
    } else {
      p = a.aux;
      ld = a.ldaux;
      at = 0;
      f32 = F32;
    }
  }
};

// What becomes of N sums of row m (of the operands' rows; of the weight
// gradient: an output feature) from column n on, in group g.
template <bool F32, int MODE, int N>
__device__ __forceinline__ void finish(const LinArgs& a, int g, int part, int64_t m, int n, float (&run)[1][N],
                                       const float (&bias)[N], bool has_old, const float (&old)[1][N]) {
  float (&v)[N] = run[0];
  auto add = [&](const float (&b)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += b[e];
  };
  if constexpr (MODE == LIN_FORWARD) {
    if (a.bias) add(bias);
    if (a.pre) store_run(a.pre, m * a.ldpre + n, F32, v);
    activate_runs<F32>(a.act, run);
    if (has_old) add(old[0]);
    store_run(a.c, m * a.ldc + n, F32, v);
  } else if constexpr (MODE == LIN_INPUT) {
    if (has_old) times_slopes<F32>(a.act, old, run);
    store_run(a.c, m * a.ldc + n, F32, v);
  } else if (a.parts > 1) {
    const int64_t at = (static_cast<int64_t>(part) * a.groups + g) * a.m + m;
    store_run(a.part, at * a.n + n, true, v);
  } else {
    if (has_old) add(old[0]);
    store_run(a.c, g * a.gc + m * a.ldc + n, a.c_dt == DT_F32, v);
  }
}

// What a workgroup's part of a product reads and writes.
struct Tile {
  const char *p, *q;
  int group, part, k;
  int m_valid, n_valid, n0;
  int64_t row0;   // of c: a row (forward, input gradient) or an output feature
};

// A tile's part of a matrix in memory: rows m_valid, columns up to a.n; what
// lies outside is neither read nor written (no branches, so that the stores
// of one row of blocks need not end before the next one's begin).
struct Window {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t ld;     // bytes
  bool f32;
  __device__ __forceinline__ Window(const void* p, int64_t at, int64_t ld_elems, bool f32_, const LinArgs& a, const Tile& w)
      : ld(static_cast<uint32_t>(ld_elems) * (f32_ ? 4 : 2)), f32(f32_) {
    const uint32_t es = f32 ? 4 : 2, end = (w.m_valid - 1) * ld + (a.n - w.n0) * es;
    rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(p)) + (at + w.row0 * ld_elems + w.n0) * es, 0, end, 0x00020000);
  }
  // Byte of row r, column n of the tile (at columns behind the matrix: nowhere).
  __device__ __forceinline__ uint32_t at(int r, int n, int columns) const {
    return n < columns ? r * ld + n * (f32 ? 4 : 2) : kNowhere;
  }
};

// A tile's results from the accumulators to memory, where rows lie on 16-byte
// borders.
//
// A lane holds columns 4 (l / 16) .. + 3 of row l mod 16 of each 16 x 16
// block.  Swapping the odd rows of 16 lanes of one block with the even ones of
// the next gives every lane a run of eight columns, without a way through LDS.
// Two such runs, 32 columns apart, are handled together: in bf16 their halves
// are exchanged (exchange8), so that an access covers whole 128-byte lines of
// eight rows instead of half lines of sixteen.
//
// Old values come through the ring: every lane's go straight into LDS slots of
// its own, a batch of block rows at a time, before the batch's first store.
// The loop then waits for no memory: a wait for loads between the stores would
// wait for the stores too (one counter), 1 us for each of a tile's block rows.
// PLAIN: the sums alone are the results, and all block rows are unrolled (the
// loop's branches take half of its time).
template <bool F32, int MODE, typename G, bool PLAIN>
__device__ __forceinline__ void leave(const LinArgs& a, const Tile& w, const Old<F32, MODE>& old, char* const (&ring)[G::U],
                                      int row_p, int row_q, const f32x4_t (&acc)[G::MS][G::NS]) {
  constexpr int RUNS = G::NS / 2, H = RUNS >= 2 ? 2 : 1, OW = F32 || MODE == LIN_WEIGHT ? 2 : 1;
  constexpr int FIT = G::UNIT / (RUNS * OW * 1024), BATCH = FIT < G::MS ? FIT : G::MS;   // block rows in a unit
  static_assert(BATCH >= 1 && G::U >= G::NW, "a unit per wave");
  const int lane = threadIdx.x & 63, r16 = lane & 15, columns = a.n - w.n0;
  const int c8 = row_q + 16 * (lane >> 4 & 1) + 8 * (lane >> 5);   // of the lane's first run
  // Runs i .. i+H-1 of the 16 rows from block row s on: f(which, byte).  In
  // halves (bf16, two runs): after exchange8.
  auto each = [&](const Window& m, int s, int i, auto&& f) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const bool x = H == 2 && !m.f32;
      f(h, m.at(row_p + s * 16 + (x ? (r16 & 7) + 8 * h : r16), c8 + 32 * (i + (x ? r16 >> 3 : h)), columns));
    }
  };
  auto put = [&](const Window& m, int s, int i, const float (&v)[H][8]) {
    u32x4_t u[H];
    if (m.f32) {
      each(m, s, i, [&](int h, uint32_t at) {
        u32x4_t lo, hi;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = __float_as_uint(v[h][e]);
          hi[e] = __float_as_uint(v[h][4 + e]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(lo, m.rs, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(hi, m.rs, at, 16, 0);
      });
      return;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) u[h] = pack8(v[h]);
    if constexpr (H == 2) exchange8(u);
    each(m, s, i, [&](int h, uint32_t at) { __builtin_amdgcn_raw_buffer_store_b128(u[h], m.rs, at, 0, 0); });
  };
  // Runs i .. i+H-1 of a row of blocks.
  auto turn = [&](const f32x4_t (&row)[G::NS], int i, float (&v)[H][8]) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(row[2 * (i + h)][e]),
                                                        __float_as_uint(row[2 * (i + h) + 1][e]), false, false);
        v[h][e] = __uint_as_float(x[0]);
        v[h][4 + e] = __uint_as_float(x[1]);
      }
  };
  const bool parts = MODE == LIN_WEIGHT && a.parts > 1;
  const Window to = parts ? Window(a.part, (static_cast<int64_t>(w.part) * a.groups + w.group) * a.m * a.n, a.n, true, a, w)
                          : Window(a.c, MODE == LIN_WEIGHT ? w.group * a.gc : 0, a.ldc, MODE == LIN_WEIGHT ? a.c_dt == DT_F32 : F32, a, w);
  const bool has_pre = MODE == LIN_FORWARD && a.pre;
  const Window pre(has_pre ? a.pre : a.c, 0, a.ldpre, F32, a, w);
  const Window from(old.p ? old.p : a.c, old.at, old.ld, old.f32, a, w);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t unit = 0;
#pragma unroll
  for (int b = 0; b < G::NW; ++b)
    unit = wave == b ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MUON_LDS char*)ring[b])) : unit;
  auto slot = [&](int s, int i, int o) { return unit + ((s % BATCH * RUNS + i) * OW + o) * 1024; };
  float bias[MODE == LIN_FORWARD ? RUNS : 1][8];
#pragma unroll
  for (int i = 0; i < (MODE == LIN_FORWARD ? RUNS : 1); ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[i][e] = 0.0f;
    const int n = w.n0 + c8 + 32 * i;
    if (MODE == LIN_FORWARD && a.bias && n < a.n) load_run(a.bias, static_cast<int64_t>(w.group) * a.n + n, F32, bias[i]);
  }
  if (old.p) __syncthreads();   // (the other waves have read the ring's last stage)
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): the bias is here
  if constexpr (PLAIN) {
#pragma unroll
    for (int s = 0; s < G::MS; ++s) {
#pragma unroll
      for (int i = 0; i < RUNS; i += H) {
        float v[H][8];
        turn(acc[s], i, v);
        put(to, s, i, v);
      }
    }
    return;
  }
  // (One copy of what follows the sums, for all rows of blocks.)
#pragma unroll 1
  for (int s = 0; s < G::MS; ++s) {
    if (row_p + s * 16 >= w.m_valid) break;
    if (old.p && s % BATCH == 0) {
#pragma unroll 1
      for (int t = s; t < s + BATCH; ++t)
#pragma unroll
        for (int i = 0; i < RUNS; i += H)
          each(from, t, i, [&](int h, uint32_t at) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from.rs, (MUON_LDS void*)static_cast<uintptr_t>(slot(t, i + h, 0)), 16,
                                                     at, 0, 0, 0);
            if constexpr (OW == 2) {
              if (from.f32)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from.rs, (MUON_LDS void*)static_cast<uintptr_t>(slot(t, i + h, 1)),
                                                         16, at + 16, 0, 0, 0);
            }
          });
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    }
    // Accumulators have no run-time index.  A switch is the shorter way to
    // them (300 rows, 768 x 768: 7.9 instead of 8.7 us), but left the Large
    // kernels short of registers: their main loops moved accumulators and
    // spilled (the input gradient through x_pre 1125 instead of 603 us, 8192^3
    // 1597 instead of 789).
    f32x4_t row[G::NS];
    auto take = [&](auto b) {
#pragma unroll
      for (int t = 0; t < G::NS; ++t) row[t] = acc[b][t];
    };
    if constexpr (G::MS * G::NS > 16) {
#pragma unroll
      for (int b = 0; b < G::MS; ++b)
        if (b == s) {
#pragma unroll
          for (int t = 0; t < G::NS; ++t) row[t] = acc[b][t];
        }
    } else {
      static_assert(G::MS <= 4, "a case per row of blocks");
      switch (s) {
        case 0: take(std::integral_constant<int, 0>{}); break;
        case 1: take(std::integral_constant<int, 1>{}); break;
        case 2: take(std::integral_constant<int, (G::MS > 2 ? 2 : 0)>{}); break;
        default: take(std::integral_constant<int, (G::MS > 3 ? 3 : 0)>{}); break;
      }
    }
#pragma unroll
    for (int i = 0; i < RUNS; i += H) {
      float v[H][8], o[H][8];
      turn(row, i, v);
      if (old.p) {
        u32x4_t u[OW][H];
#pragma unroll
        for (int q = 0; q < OW; ++q)
#pragma unroll
          for (int h = 0; h < H; ++h)
            u[q][h] = *(const MUON_LDS u32x4_t*)static_cast<uintptr_t>(slot(s, i + h, q) + lane * 16);
        if constexpr (H == 2) {
          if (!from.f32) exchange8(u[0]);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const u32x4_t both[2] = {u[0][h], u[OW - 1][h]};
          unpack8(both, from.f32, o[h]);
        }
      }
      auto add = [&](const float (&x)[8], int h) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[h][e] += x[e];
      };
      if constexpr (MODE == LIN_INPUT) {
        if (old.p) times_slopes<F32>(a.act, o, v);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if constexpr (MODE == LIN_FORWARD) add(bias[i + h], h);
        if constexpr (MODE == LIN_WEIGHT) {
          if (old.p) add(o[h], h);
        }
      }
      if (has_pre) put(pre, s, i, v);
      if constexpr (MODE == LIN_FORWARD) {
        activate_runs<F32>(a.act, v);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (old.p) add(o[h], h);
      }
      put(to, s, i, v);
    }
  }
}

// One tile of at most G::BM x G::BN.
template <bool F32, int MODE, typename G, int AL, bool PLAIN>
__device__ __forceinline__ void tile(const LinArgs& a, const Tile& w, char* const (&ring)[G::U]) {
  constexpr bool PKM = MODE == LIN_WEIGHT, QKM = MODE != LIN_FORWARD;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row_p = (wave / G::WC) * G::WM, row_q = (wave % G::WC) * G::WN;
  f32x4_t acc[G::MS][G::NS];
#pragma unroll
  for (int s = 0; s < G::MS; ++s)
#pragma unroll
    for (int t = 0; t < G::NS; ++t) acc[s][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const Operand<F32, PKM, G::BM, G::NT, AL> P(w.p, a.ldp, w.m_valid, w.k);
  const Operand<F32, QKM, G::BN, G::NT, AL> Q(w.q, a.ldq, w.n_valid, w.k);
  product<F32, PKM, QKM, G, AL>(P, Q, w.k, ring, row_p, row_q, acc);

  const Old<F32, MODE> old(a, w.group);
  if constexpr (AL == 16) {
    leave<F32, MODE, G, PLAIN>(a, w, old, ring, row_p, row_q, acc);
  } else {
    // Rows on no 16-byte borders: through LDS, 32 rows at a time in a strip of
    // the wave's own, then a lane per column.
    __syncthreads();
    constexpr int PER = G::UNIT / G::STRIP;   // strips of a unit
    static_assert(PER * G::U >= G::NW, "strips fit the ring");
    uint32_t base = 0;
#pragma unroll
    for (int b = 0; b < G::U; ++b)
      base = wave / PER == b ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MUON_LDS char*)ring[b])) : base;
    MUON_LDS float* strip = (MUON_LDS float*)(static_cast<uintptr_t>(base + (wave % PER) * G::STRIP));
#pragma unroll 1
    for (int s = 0; s < G::MS / 2; ++s) {
      const int ms = row_p + s * 32;
      if (ms >= w.m_valid) break;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int b = 0; b < G::MS; ++b)
        if (b / 2 == s) {
#pragma unroll
          for (int t = 0; t < G::NS; ++t)
            *(MUON_LDS f32x4_t*)(strip + (b % 2 * 16 + (lane & 15)) * G::SP + t * 16 + 4 * (lane >> 4)) = acc[b][t];
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 4
      for (int i = lane; i < 32 * G::WN; i += 64) {
        const int r = i / G::WN, c = i % G::WN;
        const int n = w.n0 + row_q + c;
        if (ms + r >= w.m_valid || n >= a.n) continue;
        float v[1][1] = {{strip[r * G::SP + c]}}, b1[1] = {0.0f}, o1[1][1] = {{0.0f}};
        const int64_t m = w.row0 + ms + r;
        if (MODE == LIN_FORWARD && a.bias) load_run(a.bias, static_cast<int64_t>(w.group) * a.n + n, F32, b1);
        if (old.p) load_run(old.p, old.at + m * old.ld + n, old.f32, o1[0]);
        finish<F32, MODE, 1>(a, w.group, w.part, m, n, v, b1, old.p != nullptr, o1);
      }
    }
  }
}

// (Medium tiles run two workgroups on a CU.)
template <bool F32, int MODE, typename G, int AL, bool PLAIN>
__global__ __launch_bounds__(G::NT, G::UNIT * G::U <= 81920 ? 2 : 1) void k_linear(LinArgs a, int run) {
  constexpr int ES = F32 ? 4 : 2, LBK = KB / ES;
  // (Arrays of their own, so that the compiler can tell a read of one unit
  // from a load into another.)
  __shared__ __attribute__((aligned(16))) char unit0[G::UNIT];
  __shared__ __attribute__((aligned(16))) char unit1[G::UNIT];
  __shared__ __attribute__((aligned(16))) char unit2[G::U > 2 ? G::UNIT : 16];
  __shared__ __attribute__((aligned(16))) char unit3[G::U > 3 ? G::UNIT : 16];
  __shared__ __attribute__((aligned(16))) char unit4[G::U > 4 ? G::UNIT : 16];
  __shared__ __attribute__((aligned(16))) char unit5[G::U > 5 ? G::UNIT : 16];
  __shared__ __attribute__((aligned(16))) char unit6[G::U > 6 ? G::UNIT : 16];
  __shared__ __attribute__((aligned(16))) char unit7[G::U > 7 ? G::UNIT : 16];
  const int idx = tile_of(blockIdx.x, run, MODE == LIN_WEIGHT), nt = (a.n + G::BN - 1) / G::BN;
  Group g;
  Tile w;
  int rt, ct;
  w.part = 0;
  if constexpr (MODE == LIN_WEIGHT) {
    const int mt = (a.m + G::BM - 1) / G::BM;
    if (idx >= mt * nt * a.groups * a.parts) return;
    const int gi = idx / (mt * nt);
    w.part = gi / a.groups;
    // Groups with many rows first: a tile's time is its rows, and a long one
    // begun last would run alone.
    g.index = gi % a.groups;
    if (a.offsets && a.groups > 1 && a.groups <= kRanked) g.index = group_by_size(a, g.index);
    g.lo = a.offsets ? clamped(gmem(a.offsets)[g.index], 0, a.rows) : 0;
    g.hi = a.offsets ? clamped(gmem(a.offsets)[g.index + 1], g.lo, a.rows) : a.rows;
    block_order(idx % (mt * nt), mt, nt, rt, ct);
    const int rows = g.hi - g.lo;
    const int per = a.parts > 1 ? ((rows + a.parts - 1) / a.parts + LBK - 1) / LBK * LBK : rows;
    const int first = static_cast<int>(min(static_cast<int64_t>(rows), static_cast<int64_t>(w.part) * per));
    w.k = min(per, rows - first);
    const int64_t from = g.lo + first;
    w.row0 = rt * G::BM;
    w.m_valid = min(G::BM, a.m - rt * G::BM);
    w.p = static_cast<const char*>(a.p) + (from * a.ldp + rt * G::BM) * ES;
    w.q = static_cast<const char*>(a.q) + (from * a.ldq + ct * G::BN) * ES;
  } else {
    int local;
    if (!find_rows(a, idx, G::BM, nt, g, local)) return;
    block_order(local, (g.hi - g.lo + G::BM - 1) / G::BM, nt, rt, ct);
    w.k = a.k;
    w.row0 = g.lo + rt * G::BM;
    w.m_valid = min(G::BM, g.hi - static_cast<int>(w.row0));
    w.p = static_cast<const char*>(a.p) + w.row0 * a.ldp * ES;
    const int64_t at = static_cast<int64_t>(ct) * G::BN;
    w.q = static_cast<const char*>(a.q) + (g.index * a.gq + (MODE == LIN_FORWARD ? at * a.ldq : at)) * ES;
  }
  w.group = g.index;
  w.n0 = ct * G::BN;
  w.n_valid = min(G::BN, a.n - w.n0);
  if constexpr (G::U == 8) {
    char* const ring[8] = {unit0, unit1, unit2, unit3, unit4, unit5, unit6, unit7};
    tile<F32, MODE, G, AL, PLAIN>(a, w, ring);
  } else if constexpr (G::U == 5) {
    char* const ring[5] = {unit0, unit1, unit2, unit3, unit4};
    // A tile that is less than half full in one direction takes half the time.
    if constexpr (G::BM == 256 && G::BN == 256) {
      if (w.n_valid <= 128) {
        tile<F32, MODE, Geo<256, 128, 4, 1, 5, G::UNIT>, AL, PLAIN>(a, w, ring);
        return;
      }
      if (w.m_valid <= 128) {
        tile<F32, MODE, Geo<128, 256, 1, 4, 5, G::UNIT>, AL, PLAIN>(a, w, ring);
        return;
      }
    }
    tile<F32, MODE, G, AL, PLAIN>(a, w, ring);
  } else if constexpr (G::U == 4) {
    char* const ring[4] = {unit0, unit1, unit2, unit3};
    tile<F32, MODE, G, AL, PLAIN>(a, w, ring);
  } else {
    char* const ring[2] = {unit0, unit1};
    tile<F32, MODE, G, AL, PLAIN>(a, w, ring);
  }
}

// ---------------------------------------------------------------------------
// Few rows (serving): the weights are read once and everything else is small.
// A workgroup takes 16 columns of a group's 16 rows; its two waves take the
// 128-byte blocks of k in turn, straight from global memory into MFMA
// fragments (no element is used twice), and add their sums up in LDS.
// ---------------------------------------------------------------------------
constexpr int kThinRows = 16, kThinCols = 16, kThinWaves = 2;

template <bool F32>
__global__ __launch_bounds__(64 * kThinWaves) void k_linear_thin(LinArgs a) {
  constexpr int ES = F32 ? 4 : 2, STEPS = 2, AHEAD = 4;   // k-steps (64 bytes) of a block; blocks in flight
  __shared__ __attribute__((aligned(16))) float sums[kThinWaves][kThinRows][kThinCols + 4];
  const int nt = (a.n + kThinCols - 1) / kThinCols;
  Group g;
  int local;
  if (!find_rows(a, blockIdx.x, kThinRows, nt, g, local)) return;
  const int mt = (g.hi - g.lo + kThinRows - 1) / kThinRows, rt = local % mt, n0 = local / mt * kThinCols;
  const int row0 = g.lo + rt * kThinRows, m_valid = min(kThinRows, g.hi - row0), n_valid = min(kThinCols, a.n - n0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
  const uint32_t bytes = static_cast<uint32_t>(a.k) * ES, blocks = (bytes + 127) / 128;
  const uint32_t ldp = static_cast<uint32_t>(a.ldp) * ES, ldq = static_cast<uint32_t>(a.ldq) * ES;
  char* const p = const_cast<char*>(static_cast<const char*>(a.p)) + static_cast<int64_t>(row0) * a.ldp * ES;
  char* const q = const_cast<char*>(static_cast<const char*>(a.q)) + (g.index * a.gq + n0 * a.ldq) * ES;
  const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(p, 0, (m_valid - 1) * ldp + bytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(q, 0, (n_valid - 1) * ldq + bytes, 0x00020000);
  u32x4_t fp[2][AHEAD][STEPS], fq[2][AHEAD][STEPS];
  auto load = [&](uint32_t b0, u32x4_t (&vp)[AHEAD][STEPS], u32x4_t (&vq)[AHEAD][STEPS]) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const uint32_t k = (b0 + i * kThinWaves) * 128 + s * 64 + (lane >> 4) * 16;
        vq[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rq, k < bytes ? l16 * ldq + k : kNowhere, 0, 0);
        vp[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rp, k < bytes ? l16 * ldp + k : kNowhere, 0, 0);
      }
  };
  f32x4_t acc[1][1] = {{f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}}};
  auto mul = [&](const u32x4_t (&vp)[AHEAD][STEPS], const u32x4_t (&vq)[AHEAD][STEPS]) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const u32x4_t one_p[1] = {vp[i][s]}, one_q[1] = {vq[i][s]};
        multiply<F32, 1, 1>(one_p, one_q, acc);
      }
  };
  constexpr uint32_t HOP = AHEAD * kThinWaves;
  load(wave, fp[0], fq[0]);
  for (uint32_t b = wave; b < blocks; b += 2 * HOP) {
    load(b + HOP, fp[1], fq[1]);   // (behind the end: zeros, without a fetch)
    mul(fp[0], fq[0]);
    load(b + 2 * HOP, fp[0], fq[0]);
    mul(fp[1], fq[1]);
  }
  *reinterpret_cast<f32x4_t*>(&sums[wave][l16][4 * (lane >> 4)]) = acc[0][0];
  __syncthreads();
  const int r = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
  if (r >= m_valid || n0 + c >= a.n) return;
  float v[1][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[0][e] = sums[0][r][c + e];
#pragma unroll
    for (int w = 1; w < kThinWaves; ++w) v[0][e] += sums[w][r][c + e];
  }
  float bias[8], old[1][8];
  if (a.bias) load_run(a.bias, static_cast<int64_t>(g.index) * a.n + n0 + c, F32, bias);
  if (a.aux) load_run(a.aux, static_cast<int64_t>(row0 + r) * a.ldaux + n0 + c, F32, old[0]);
  finish<F32, LIN_FORWARD, 8>(a, g.index, 0, row0 + r, n0 + c, v, bias, a.aux != nullptr, old);
}

// ---------------------------------------------------------------------------
// Elementwise and column passes
// ---------------------------------------------------------------------------
constexpr int kPassThreads = 256;

// Rows that belong to a group (all without offsets).
__device__ __forceinline__ int rows_used(const int32_t* offsets, int groups, int rows) {
  return offsets ? clamped(gmem(offsets)[groups], 0, rows) : rows;
}

// N: values of a thread (eight on 16-byte borders, or one).
template <bool F32, int N>
__global__ __launch_bounds__(kPassThreads) void k_linear_slope(const void* dy, int64_t ld_dy, const void* pre,
                                                              int64_t ld_pre, void* dz, int64_t ld_dz,
                                                              const int32_t* offsets, int groups, int rows, int out,
                                                              int act) {
  const int runs = out / N;
  const int64_t n = static_cast<int64_t>(rows_used(offsets, groups, rows)) * runs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPassThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kPassThreads) {
    const int64_t r = i / runs;
    const int c = static_cast<int>(i % runs) * N;
    float g[1][N], z[1][N];
    load_run(dy, r * ld_dy + c, F32, g[0]);
    load_run(pre, r * ld_pre + c, F32, z[0]);
    times_slopes<F32>(act, z, g);
    store_run(dz, r * ld_dz + c, F32, g[0]);
  }
}

// The same in bf16 where db is wanted too: the terms dy act'(pre) of one tile
// of `per` rows and 64 N columns of a group are summed in float32 as they are
// formed (dz, rounded for the matrix units, is only written; with random
// signs its half steps would be sqrt(rows) 2^-9 of a term in db), and
// k_linear_sums adds a group's tiles up.  Four waves take every fourth row,
// four in flight.  N = 2 where rows lie on 4-byte borders.  Tiles of rows and
// not parts of a group, so that one group with most rows is split as well.
// 98304 rows of 64 groups, 1408 columns, silu: 118 us for db alone (4.7 TB/s;
// with erfc's gelu the slopes bound it, 268); with dz 37 us more than
// k_linear_slope without db.  Reading the rounded dz again took 140 more.
constexpr int kSumThreads = 256;
template <int N>
__global__ __launch_bounds__(kSumThreads) void k_linear_slope_sums(LinArgs a, const void* dy, int64_t ld_dy,
                                                                   const void* pre, int64_t ld_pre, void* dz,
                                                                   int64_t ld_dz, int per, int tiles, float* sums) {
  constexpr int NW = kSumThreads / 64, AHEAD = 4;
  __shared__ float red[NW][64 * N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blocks = (a.n + 64 * N - 1) / (64 * N);
  auto load = [&](const void* p, int64_t at, float (&v)[N][AHEAD], int i) {
    if constexpr (N == 2) {
      const uint32_t u = gmem(static_cast<const uint32_t*>(p))[at / 2];
      v[0][i] = __uint_as_float(u << 16);
      v[1][i] = __uint_as_float(u & 0xffff0000u);
    } else {
      v[0][i] = load_elem(p, at, DT_BF16);
    }
  };
  Group g;
  int local;
  // (Offsets that decrease would name more than `tiles` tiles.)
  for (int idx = blockIdx.x; idx < tiles * blocks && find_rows(a, idx, per, blocks, g, local); idx += gridDim.x) {
    const int first = g.lo + local / blocks * per, last = min(g.hi, first + per), c0 = local % blocks * 64 * N;
    const int c = c0 + lane * N;
    float s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = 0.0f;
    if (c < a.n)
      for (int r0 = first + wave; r0 < last; r0 += NW * AHEAD) {
        float v[N][AHEAD], z[N][AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int64_t r = min(r0 + i * NW, last - 1);   // (behind the last row: read again, not added)
          load(dy, r * ld_dy + c, v, i);
          load(pre, r * ld_pre + c, z, i);
        }
        times_slopes<false>(a.act, z, v);
        if (dz) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            const int64_t r = r0 + i * NW;
            if (r >= last) break;
            if constexpr (N == 2) gmem(static_cast<uint32_t*>(dz))[(r * ld_dz + c) / 2] = pack_bf16x2(v[0][i], v[1][i]);
            else store_elem(dz, r * ld_dz + c, DT_BF16, v[0][i]);
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
#pragma unroll
          for (int i = 1; i < AHEAD; ++i) v[e][i] = r0 + i * NW < last ? v[e][i] : 0.0f;
          s[e] += (v[e][0] + v[e][1]) + (v[e][2] + v[e][3]);
        }
      }
#pragma unroll
    for (int e = 0; e < N; ++e) red[wave][lane * N + e] = s[e];
    __syncthreads();
    if (threadIdx.x < 64 * N && c0 + static_cast<int>(threadIdx.x) < a.n) {
      float sum = red[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < NW; ++w) sum += red[w][threadIdx.x];
      sums[static_cast<int64_t>(idx / blocks) * a.n + c0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// db (+)= the sums of a group's tiles of `per` rows: a workgroup per 64 columns
// of a group, whose sixteen waves take every sixteenth tile, four in flight,
// and are added in wave order.  Each wave counts the tiles before the group's.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void k_linear_sums(LinArgs a, const float* sums, int per, int most) {
  constexpr int NW = kJoinThreads / 64, AHEAD = 4;
  __shared__ float red[NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks = (a.n + 63) / 64, g = blockIdx.x / blocks, c = blockIdx.x % blocks * 64 + lane;
  auto tiles_of = [&](int i) {
    const int lo = a.offsets ? clamped(gmem(a.offsets)[i], 0, a.rows) : 0;
    const int hi = a.offsets ? clamped(gmem(a.offsets)[i + 1], lo, a.rows) : a.rows;
    return (hi - lo + per - 1) / per;
  };
  int before = 0;
  for (int i = lane; i < g; i += 64) before = min(most, before + tiles_of(i));
  for (int d = 1; d < 64; d <<= 1) before = min(most, before + __shfl_xor(before, d));
  const int tiles = min(tiles_of(g), most - before);   // (fewer where offsets decrease)
  float s = 0.0f;
  if (c < a.n)
    for (int t0 = wave; t0 < tiles; t0 += NW * AHEAD) {
      float v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int t = t0 + i * NW;
        v[i] = t < tiles ? gmem(sums)[static_cast<int64_t>(before + t) * a.n + c] : 0.0f;
      }
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.n) {
    s = red[0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += red[w][lane];
    const int64_t at = static_cast<int64_t>(g) * a.n + c;
    if (a.accumulate) s += load_elem(a.c, at, a.c_dt);
    store_elem(a.c, at, a.c_dt, s);
  }
}

// Column sums of a group's rows (or of one part of them): sixteen waves take
// every sixteenth row, 64 columns each, eight rows in flight, and are added in
// wave order.
constexpr int kBiasThreads = 1024;
template <bool F32>
__global__ __launch_bounds__(kBiasThreads) void k_linear_bias(const void* dz, int64_t ld, const int32_t* offsets,
                                                             int rows, int out, void* db, int grad_dt, int accumulate,
                                                             float* part, int parts) {
  constexpr int NW = kBiasThreads / 64, AHEAD = 8;
  __shared__ float red[NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks = (out + 63) / 64, g = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 64 + lane;
  const int lo = offsets ? clamped(gmem(offsets)[g], 0, rows) : 0;
  const int hi = offsets ? clamped(gmem(offsets)[g + 1], lo, rows) : rows;
  const int per = (hi - lo + parts - 1) / parts;
  const int first = static_cast<int>(min(static_cast<int64_t>(hi), lo + static_cast<int64_t>(blockIdx.y) * per));
  const int last = min(hi, first + per);
  float s = 0.0f;
  if (c < out)
    for (int r0 = first + wave; r0 < last; r0 += NW * AHEAD) {
      float v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int r = r0 + i * NW;
        v[i] = r < last ? load_elem(dz, r * ld + c, F32 ? DT_F32 : DT_BF16) : 0.0f;
      }
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < out) {
    s = red[0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += red[w][lane];
    const int64_t at = static_cast<int64_t>(g) * out + c;
    if (parts > 1) {
      part[static_cast<int64_t>(blockIdx.y) * (gridDim.x / blocks) * out + at] = s;
    } else {
      if (accumulate) s += load_elem(db, at, grad_dt);
      store_elem(db, at, grad_dt, s);
    }
  }
}

// c (+)= sum of `parts` arrays of `groups` x m x n, in order.
__global__ __launch_bounds__(kPassThreads) void k_linear_join(const float* part, int parts, int groups, int m, int n,
                                                             void* c, int64_t ldc, int64_t gc, int c_dt,
                                                             int accumulate) {
  const int64_t total = static_cast<int64_t>(groups) * m * n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPassThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kPassThreads) {
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += gmem(part)[p * total + i];
    const int64_t row = i / n, at = row / m * gc + row % m * ldc + i % n;
    if (accumulate) s += load_elem(c, at, c_dt);
    store_elem(c, at, c_dt, s);
  }
}

using Large = Geo<256, 256, 2, 2, 5>;
using Medium = Geo<128, 128, 2, 2, 5>;
using Plain = Geo<128, 128, 2, 2, 2, 2 * Medium::STRIP>;   // operands through registers
using Small = Geo<64, 128, 1, 4, 4>;
using MediumDeep = Geo<128, 128, 2, 2, 8>;
using SmallDeep = Geo<64, 128, 1, 4, 8>;
using Tiny = Geo<64, 64, 2, 2, 8>;

int64_t ceil_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxBlocks = (int64_t{1} << 23) - 1;

// Tiles of a launch at most (the groups' last tiles may be partial).
template <typename G>
int64_t tiles_at_most(const LinArgs& a, int mode) {
  const int64_t nt = ceil_of(a.n, G::BN);
  if (mode == LIN_WEIGHT) return ceil_of(a.m, G::BM) * nt * a.groups * a.parts;
  const int64_t mt = a.offsets ? std::min<int64_t>(a.rows, a.rows / G::BM + a.groups) : ceil_of(a.rows, G::BM);
  return mt * nt;
}

template <bool F32, int MODE, typename G, int AL, bool PLAIN = false>
hipError_t go(const LinArgs& a, bool dry, hipStream_t s) {
  const int64_t tiles = tiles_at_most<G>(a, MODE);
  const int64_t run = std::max<int64_t>(1, std::min<int64_t>(32, tiles / 16));
  const int64_t blocks = ceil_of(tiles, 8 * run) * 8 * run;
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  if (blocks == 0 || dry) return hipSuccess;
  hipLaunchKernelGGL((k_linear<F32, MODE, G, AL, PLAIN>), dim3(static_cast<uint32_t>(blocks)), dim3(G::NT), 0, s, a,
                     static_cast<int>(run));
  return hipGetLastError();
}

template <bool F32>
hipError_t go_thin(const LinArgs& a, bool dry, hipStream_t s) {
  const int64_t mt = a.offsets ? std::min<int64_t>(a.rows, a.rows / kThinRows + a.groups) : ceil_of(a.rows, kThinRows);
  const int64_t blocks = mt * ceil_of(a.n, kThinCols);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  if (dry) return hipSuccess;
  hipLaunchKernelGGL(k_linear_thin<F32>, dim3(static_cast<uint32_t>(blocks)), dim3(64 * kThinWaves), 0, s, a);
  return hipGetLastError();
}

// Rounds that `tiles` take on the GPU (in halves): whole ones while they are few.
int64_t half_rounds(int64_t tiles, int64_t at_once) {
  return tiles <= 4 * at_once ? 2 * ceil_of(tiles, at_once) : 2 * tiles / at_once + 1;
}
// Tiles of a launch as expected: a group's last tile is half full on average.
template <typename G>
int64_t tiles_expected(const LinArgs& a, int mode) {
  const int64_t nt = ceil_of(a.n, G::BN);
  if (mode == LIN_WEIGHT || !a.offsets) return tiles_at_most<G>(a, mode);
  return std::max<int64_t>(1, a.rows / G::BM + a.groups / 2) * nt;
}

// Whether a product's sums alone are its result.
bool plain(const LinArgs& a, int mode) {
  if (mode == LIN_WEIGHT) return a.parts > 1 || !a.accumulate;
  return !a.aux && (mode == LIN_INPUT || (!a.bias && !a.pre && a.act == LINEAR_NONE));
}

// The kernel of a product.  `align`: 16 (rows of whole 16-byte runs on 16-byte
// borders), 4 or 2.
template <int MODE>
hipError_t pick(const LinArgs& a, int dt, int align, bool dry, hipStream_t s) {
  const int64_t small = tiles_expected<Small>(a, MODE), medium = tiles_expected<Medium>(a, MODE);
  const int64_t mean = a.rows / a.groups;   // rows of a group
  if constexpr (MODE == LIN_FORWARD) {
    // Few rows: every 16 of a group's read its weight again (from the L2 or
    // the Infinity Cache).  64 experts of 2048 x 1408: 69 us against 92 (Small)
    // at three rows an expert, 84 against 99 at nine, 95 against 100 at twelve;
    // 4096 x 4096, one group: 18 us against 22 (SmallDeep) at 32 rows, 31
    // against 24 at 64.
    if (align == 16 && (mean <= 10 || (mean <= 40 && small <= 256))) {
      const hipError_t e = dt == DT_F32 ? go_thin<true>(a, dry, s) : go_thin<false>(a, dry, s);
      if (e != hipErrorInvalidValue) return e;   // (more workgroups than a launch has: the tiles are larger)
    }
  }
  if (dt == DT_F32) {
    // A float32 product is slow enough (an eighth of the bf16 rate) that small
    // tiles lose nothing, and few large ones leave CUs idle: 9 groups of 300
    // rows, 517 x 259: 33 us in 64 x 128 tiles.
    if (align == 16) {
      if (small <= 256) return go<true, MODE, Tiny, 16>(a, dry, s);
      return medium <= 512 ? go<true, MODE, Small, 16>(a, dry, s) : go<true, MODE, Medium, 16>(a, dry, s);
    }
    if (small <= 256) return go<true, MODE, Tiny, 4>(a, dry, s);
    return medium <= 512 ? go<true, MODE, Small, 4>(a, dry, s) : go<true, MODE, Medium, 4>(a, dry, s);
  }
  if (align == 4) return medium <= 512 ? go<false, MODE, Small, 4>(a, dry, s) : go<false, MODE, Medium, 4>(a, dry, s);
  if (align != 16) return go<false, MODE, Plain, 2>(a, dry, s);
  if constexpr (MODE != LIN_WEIGHT) {
    // No more tiles than CUs: a ring over most of a CU's LDS (4096 x 4096: 23
    // instead of 40 us at 32 to 96 rows).
    if (small <= 256) return go<false, MODE, SmallDeep, 16>(a, dry, s);
    if (mean <= 96) return go<false, MODE, Small, 16>(a, dry, s);
  }
  if (medium <= 256) return go<false, MODE, MediumDeep, 16>(a, dry, s);
  // Time in units of a Large tile's step of k: a CU runs one Large tile, whose
  // beginning and end take as long as 600 steps, or two Medium ones at once,
  // 7/8 of a step (their fragment reads take the LDS 1.5 times as long as
  // their products the matrix units) and no more.  Experts of 2048 x 1408, 1536
  // rows each: 562 us (Large) against 663, with silu, pre and residual 641
  // against 736; 16384 rows, 768 x 768: 24.5 against 26.9, with silu, pre and
  // residual 35.7 against 33.6.
  const int64_t k = MODE == LIN_WEIGHT ? mean / a.parts : a.k;
  if (half_rounds(tiles_expected<Large>(a, MODE), 256) * (k + 600) <= half_rounds(medium, 512) * (k * 7 / 8))
    return plain(a, MODE) ? go<false, MODE, Large, 16, true>(a, dry, s) : go<false, MODE, Large, 16>(a, dry, s);
  return go<false, MODE, Medium, 16>(a, dry, s);
}

uint32_t pass_blocks(int64_t n) {
  return static_cast<uint32_t>(std::max<int64_t>(1, std::min<int64_t>(1 << 20, ceil_of(n, kPassThreads))));
}

}  // namespace

static hipError_t linear(const LinArgs& a, int mode, int dt, int align, bool dry, hipStream_t s) {
  if (mode == LIN_FORWARD) return pick<LIN_FORWARD>(a, dt, align, dry, s);
  if (mode == LIN_INPUT) return pick<LIN_INPUT>(a, dt, align, dry, s);
  return pick<LIN_WEIGHT>(a, dt, align, dry, s);
}
hipError_t launch_linear(const LinArgs& a, int mode, int dt, int align, hipStream_t s) {
  return linear(a, mode, dt, align, false, s);
}
bool linear_fits(const LinArgs& a, int mode, int dt, int align) {
  return linear(a, mode, dt, align, true, nullptr) == hipSuccess;
}

int linear_weight_parts(int64_t rows, int64_t out, int64_t in, int64_t groups) {
  const int64_t tiles = ceil_of(out, 128) * ceil_of(in, 128) * groups;
  const int64_t most = std::max<int64_t>(1, rows / groups / 512);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most, 512 / tiles, 64})));
}

hipError_t launch_linear_join(const LinArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_linear_join, dim3(pass_blocks(static_cast<int64_t>(a.groups) * a.m * a.n)), dim3(kPassThreads), 0,
                     s, a.part, a.parts, a.groups, a.m, a.n, a.c, a.ldc, a.gc, a.c_dt, a.accumulate);
  return hipGetLastError();
}

hipError_t launch_linear_slope(const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre, void* dz, int64_t ld_dz,
                               const int32_t* offsets, int groups, int64_t rows, int64_t out, int act, int dt, int align,
                               hipStream_t s) {
  const bool runs = align == 16;
  const dim3 grid(pass_blocks(rows * (runs ? out / 8 : out))), threads(kPassThreads);
#define MUON_SLOPE(F32, N)                                                                                           \
  hipLaunchKernelGGL((k_linear_slope<F32, N>), grid, threads, 0, s, dy, ld_dy, pre, ld_pre, dz, ld_dz, offsets,      \
                     groups, (int)rows, (int)out, act)
  if (dt == DT_F32) {
    if (runs) MUON_SLOPE(true, 8); else MUON_SLOPE(true, 1);
  } else {
    if (runs) MUON_SLOPE(false, 8); else MUON_SLOPE(false, 1);
  }
#undef MUON_SLOPE
  return hipGetLastError();
}

// Rows of a tile: 64 while they are few, at most 256.
constexpr int64_t kSumTiles = 2048;
static int slope_rows(int64_t rows, int64_t out) {
  const int64_t blocks = ceil_of(out, 128);
  return static_cast<int>(std::max<int64_t>(64, std::min<int64_t>(256, ceil_of(rows * blocks, kSumTiles * 64) * 64)));
}
// Tiles at most.  (Bounded so that fewer rows never have more: a workspace is
// used for up to so many rows.)
int64_t linear_slope_tiles(int64_t rows, int64_t out, int64_t groups) {
  return std::max(std::min(rows / 64, kSumTiles / ceil_of(out, 128)), rows / 256) + groups;
}

hipError_t launch_linear_slope_sums(const LinArgs& a, const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre,
                                    void* dz, int64_t ld_dz, float* sums, hipStream_t s) {
  const bool pairs = a.n % 2 == 0 && ld_dy % 2 == 0 && ld_pre % 2 == 0 && reinterpret_cast<uintptr_t>(dy) % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(pre) % 4 == 0;
  const int per = slope_rows(a.rows, a.n), tiles = static_cast<int>(linear_slope_tiles(a.rows, a.n, a.groups));
  const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(tiles * ceil_of(a.n, pairs ? 128 : 64), 1 << 16)));
  if (pairs)
    hipLaunchKernelGGL(k_linear_slope_sums<2>, grid, dim3(kSumThreads), 0, s, a, dy, ld_dy, pre, ld_pre, dz, ld_dz, per,
                       tiles, sums);
  else
    hipLaunchKernelGGL(k_linear_slope_sums<1>, grid, dim3(kSumThreads), 0, s, a, dy, ld_dy, pre, ld_pre, dz, ld_dz, per,
                       tiles, sums);
  return hipGetLastError();
}

hipError_t launch_linear_sums(const LinArgs& a, const float* sums, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(ceil_of(a.n, 64) * a.groups));   // (linear_bias_fits)
  hipLaunchKernelGGL(k_linear_sums, grid, dim3(kJoinThreads), 0, s, a, sums, slope_rows(a.rows, a.n),
                     static_cast<int>(linear_slope_tiles(a.rows, a.n, a.groups)));
  return hipGetLastError();
}

// (A launch has fewer than 2^32 threads.)
bool linear_bias_fits(int64_t out, int64_t groups) { return ceil_of(out, 64) * groups * kBiasThreads < int64_t{1} << 32; }

int linear_bias_parts(int64_t rows, int64_t groups) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows / groups / 256, 64)));
}

hipError_t launch_linear_bias(const void* dz, int64_t ld, const int32_t* offsets, int groups, int64_t rows, int64_t out,
                              void* db, int dt, int grad_dt, int accumulate, float* part, int parts, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(ceil_of(out, 64) * groups), static_cast<uint32_t>(parts)), threads(kBiasThreads);
  if (dt == DT_F32)
    hipLaunchKernelGGL(k_linear_bias<true>, grid, threads, 0, s, dz, ld, offsets, (int)rows, (int)out, db, grad_dt,
                       accumulate, part, parts);
  else
    hipLaunchKernelGGL(k_linear_bias<false>, grid, threads, 0, s, dz, ld, offsets, (int)rows, (int)out, db, grad_dt,
                       accumulate, part, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  hipLaunchKernelGGL(k_linear_join, dim3(pass_blocks(out * groups)), dim3(kPassThreads), 0, s, part, parts, groups, 1, (int)out, db,
                     out, out, grad_dt, accumulate);
  return hipGetLastError();
}

}  // namespace muon
