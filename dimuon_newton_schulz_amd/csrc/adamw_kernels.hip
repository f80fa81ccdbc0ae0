// AdamW over many tensors: the step with 32- and 8-bit moments, and the
// moments as values.
#include "adamw.h"

namespace muon {
namespace {

// A workgroup walks pieces blockIdx.x, blockIdx.x + gridDim.x, ...; the
// workgroups running at once stream through neighbouring memory.
constexpr int kGrid32 = 2048, kGrid8 = 2048, kGridState = 2048;

// ---------------------------------------------------------------------------
// Groups of N consecutive elements, element index a multiple of N and the
// base 16-byte aligned; `cnt` of them exist (the others read as zero and are
// not written).
// ---------------------------------------------------------------------------
template <bool BF16, int N>
__device__ __forceinline__ void load_group(const void* p, int64_t i, int cnt, float (&out)[N]) {
  if (cnt >= N) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      float t[4];
      if constexpr (BF16 && N == 8) {
        if (e != 0) continue;
        const uint4 u = *reinterpret_cast<const MUON_GLOBAL uint4*>(gmem(static_cast<const uint16_t*>(p)) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          out[2 * k] = __uint_as_float(w[k] << 16);
          out[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
      } else {
        load4_aligned(p, i + e, BF16 ? DT_BF16 : DT_F32, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[e + k] = t[k];
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) out[e] = e < cnt ? load_elem(p, i + e, BF16 ? DT_BF16 : DT_F32) : 0.0f;
}

template <bool BF16, int N>
__device__ __forceinline__ void store_group(void* p, int64_t i, int cnt, const float (&v)[N]) {
  if (cnt >= N) {
    if constexpr (BF16 && N == 8) {
      uint4 u;
      u.x = pack_bf16x2(v[0], v[1]);
      u.y = pack_bf16x2(v[2], v[3]);
      u.z = pack_bf16x2(v[4], v[5]);
      u.w = pack_bf16x2(v[6], v[7]);
      *reinterpret_cast<MUON_GLOBAL uint4*>(gmem(static_cast<uint16_t*>(p)) + i) = u;
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float t[4] = {v[e], v[e + 1], v[e + 2], v[e + 3]};
        store4_aligned(p, i + e, BF16 ? DT_BF16 : DT_F32, t);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < cnt) store_elem(p, i + e, BF16 ? DT_BF16 : DT_F32, v[e]);
}

__device__ __forceinline__ uint2 load_codes(const void* p, int64_t i, int cnt) {
  const MUON_GLOBAL uint8_t* q = gmem(static_cast<const uint8_t*>(p)) + i;
  if (cnt >= 8) return *reinterpret_cast<const MUON_GLOBAL uint2*>(q);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) w[e >> 2] |= static_cast<uint32_t>(q[e]) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(void* p, int64_t i, int cnt, uint2 c) {
  MUON_GLOBAL uint8_t* q = gmem(static_cast<uint8_t*>(p)) + i;
  if (cnt >= 8) {
    *reinterpret_cast<MUON_GLOBAL uint2*>(q) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) q[e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
}

// ---------------------------------------------------------------------------
// 8-bit moments.  A block of 256 elements is half a wave's: 32 lanes of eight
// elements (16-byte bf16 and 8-byte code accesses; a block's maximum takes
// four DPP steps and one exchange of 16-lane rows).
// ---------------------------------------------------------------------------
constexpr uint32_t kInfBits = 0x7F800000u;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}

// Maximum over each half of the wave, in every lane of it.
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));    // quad_perm [1,0,3,2]
  v = max(v, dpp_u32<0x4E>(v));    // quad_perm [2,3,0,1]
  v = max(v, dpp_u32<0x141>(v));   // row_half_mirror
  v = max(v, dpp_u32<0x140>(v));   // row_mirror
  const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max(static_cast<uint32_t>(rows[0]), static_cast<uint32_t>(rows[1]));
}

// Scales of a block and what its encoding needs, from the bits of the largest
// |m| and v.  The reciprocals (1 ulp) are taken of values that keep them
// normal numbers: v is encoded as y * 2^40 or y * 2^-24, its code's offset
// following (y = v / vs, whose bits give the code).
struct BlockScale {
  float ms, vs, minv, vinv;
  uint32_t voff;   // code offset << 20
};

__device__ __forceinline__ BlockScale block_scale(uint32_t mbits, uint32_t vbits) {
  BlockScale b;
  // Below 2^-118 (0x04800000) 1 / ms would overflow: such a block is zero.
  b.ms = mbits >= 0x04800000u ? __uint_as_float(mbits) * 0x1p-8f : 0.0f;
  b.minv = b.ms > 0.0f ? __builtin_amdgcn_rcpf(b.ms) : 0.0f;
  b.vs = __uint_as_float(vbits);
  const bool big = b.vs >= 1.0f;
  b.vinv = big ? __builtin_amdgcn_rcpf(b.vs * 0x1p-40f) : __builtin_amdgcn_rcpf(b.vs * 0x1p32f) * 0x1p8f;
  if (vbits == 0) b.vinv = 0.0f;
  b.voff = big ? 1088u << 20 : 576u << 20;
  return b;
}

// 16 * (upper half of h) + t, one instruction.
__device__ __forceinline__ uint32_t add_upper16(uint32_t h, uint32_t t) {
  uint32_t r;
  asm("v_mad_u32_u16 %0, %1, 16, %2 op_sel:[1,0,0,0]" : "=v"(r) : "v"(h), "v"(t));
  return r;
}

// 1 if x is not zero.  (As a minimum: the compiler makes a compare and a
// select of it.)
__device__ __forceinline__ int nonzero(float x) {
  int r;
  asm("v_min_u32 %0, 1, %1" : "=v"(r) : "v"(x));
  return r;
}

// Rounds eight elements to codes (those that do not exist are zero).  idx is
// the first one's index in the batch.
//
// Rounding adds to the 20 float32 mantissa bits that a code drops: 16 r + 8
// (stochastic) or half of their range (nearest), then cuts.  For m,
// v_cvt_sr_fp8_f32 does that with the upper 20 bits of its random operand,
// subnormal codes included (checked against the addition written out, over
// 4M values: equal in the normal range, and within 2^-20 of a code step of
// the border below it).  The block's largest |m| and v are a few ulp off
// their code's value at most, which neither rounding can carry to the next
// code.
template <bool STOCHASTIC>
__device__ __forceinline__ void encode8(const float (&m)[8], const float (&v)[8], uint32_t key, int64_t idx,
                                        uint2& mc, uint2& vc, float& ms, float& vs) {
  uint32_t mmax = 0, vmax = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mmax = max(mmax, __float_as_uint(m[e]) & 0x7FFFFFFFu);
    vmax = max(vmax, __float_as_uint(v[e]));
  }
  mmax = half_max(mmax);
  vmax = half_max(vmax);
  // NaN, Inf and negative v have bits from kInfBits on: then the maxima are
  // taken over the other elements, and those get the codes of NaN.
  const bool odd = __any(mmax >= kInfBits || vmax >= kInfBits);
  uint32_t mbad = 0, vbad = 0;
  if (odd) {
    mmax = 0;
    vmax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t mb = __float_as_uint(m[e]) & 0x7FFFFFFFu, vb = __float_as_uint(v[e]);
      if (mb >= kInfBits) mbad |= 1u << e; else mmax = max(mmax, mb);
      if (vb >= kInfBits) vbad |= 1u << e; else vmax = max(vmax, vb);
    }
    mmax = half_max(mmax);
    vmax = half_max(vmax);
  }
  const BlockScale b = block_scale(mmax, vmax);
  ms = b.ms;
  vs = b.vs;
  const uint32_t vadd = (STOCHASTIC ? 8u : 0x80000u) - b.voff;
  uint32_t hi = 0;
  if constexpr (STOCHASTIC)
    hi = adam_mix(key + static_cast<uint32_t>(static_cast<uint64_t>(idx) >> 32)) + static_cast<uint32_t>(idx);
  int q[2] = {0, 0};
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t rm = 0x80000000u, t = __float_as_uint(v[e] * b.vinv) + vadd;
    if constexpr (STOCHASTIC) {
      const uint32_t h = adam_mix(hi + e);
      rm = h << 16 | 0x8000u;
      t = add_upper16(h, t);
    }
    const float y = m[e] * b.minv;
    int& w = q[e >> 2];
    switch (e & 3) {
      case 0: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 0); break;
      case 1: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 1); break;
      case 2: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 2); break;
      default: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 3); break;
    }
    c[e] = static_cast<uint32_t>(max(static_cast<int>(t) >> 20, nonzero(v[e])));   // v > 0 has a code above 0
  }
  mc = make_uint2(static_cast<uint32_t>(q[0]), static_cast<uint32_t>(q[1]));
  if (odd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t byte = 0xFFu << (8 * (e & 3)), nan = 0x7Fu << (8 * (e & 3));
      uint32_t& w = e < 4 ? mc.x : mc.y;
      if (mbad >> e & 1) w = (w & ~byte) | nan;
      if (vbad >> e & 1) c[e] = 255;
    }
  }
  vc = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// Unscaled values of eight codes.
__device__ __forceinline__ void decode8(uint2 mc, uint2 vc, float (&m)[8], float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mc.x), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mc.x), true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mc.y), false);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(mc.y), true);
  m[0] = a.x; m[1] = a.y; m[2] = b.x; m[3] = b.y;
  m[4] = c.x; m[5] = c.y; m[6] = d.x; m[7] = d.y;
  // u(c) has the bits (c << 20) + 768 << 20, but for c = 0 and 255, which few
  // waves hold.  A zero byte of x has the upper bit of
  // (x - 0x01010101) & ~x & 0x80808080 set, a byte 255 is one of ~x.
  const uint32_t w[2] = {vc.x, vc.y};
  uint32_t rare = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    rare |= (((w[k] - 0x01010101u) & ~w[k]) | ((~w[k] - 0x01010101u) & w[k])) & 0x80808080u;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = __uint_as_float(((w[e >> 2] >> (8 * (e & 3)) & 0xFFu) << 20) + 0x30000000u);
  if (__any(rare != 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t k = w[e >> 2] >> (8 * (e & 3)) & 0xFFu;
      v[e] = k == 0 ? 0.0f : k == 255 ? __builtin_nanf("") : v[e];
    }
  }
}

// ---------------------------------------------------------------------------
// One step
// ---------------------------------------------------------------------------
struct StepValues {
  float b1, b2, eps, lr, rb1, rb2;
  float cm, cv;   // factors of the gradient in m, and of its square's root in v
  uint32_t key;
};

__device__ __forceinline__ StepValues step_values(const AdamArgs& a) {
  StepValues s;
  s.b1 = static_cast<float>(a.beta1);
  s.b2 = static_cast<float>(a.beta2);
  s.eps = a.eps;
  s.lr = a.ctl->lr;
  s.rb1 = a.ctl->rb1;
  s.rb2 = a.ctl->rb2;
  s.key = a.ctl->key;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  s.cm = a.c1 * gs;
  s.cv = a.root_c2 * gs;
  return s;
}

// One element: m and v hold the old moments before their factors (fm, fv:
// beta times the block's scale, or beta) and the new ones after; returns the
// new weight.  `adam` and `decay` are lr * lr_scale / (1 - beta1^t) and
// lr * weight_decay.  Square root and reciprocal are the 1 ulp instructions.
__device__ __forceinline__ float update(const StepValues& s, float g, float w, float fm, float fv, float adam,
                                        float decay, float& m, float& v) {
  m = fm * m + s.cm * g;
  const float z = s.cv * g;
  v = fv * v + z * z;
  const float den = __builtin_amdgcn_sqrtf(v) * s.rb2 + s.eps;
  const float upd = (m * adam) * __builtin_amdgcn_rcpf(den);
  return w - (upd + decay * w);
}

// The last workgroup to have read the step's values writes the next step's.
__device__ __forceinline__ void finish_step(const AdamArgs& a, bool advance) {
  __syncthreads();
  if (!advance || threadIdx.x != 0) return;
  const uint32_t seen = __hip_atomic_fetch_add(&a.ctl->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (seen != gridDim.x - 1) return;
  AdamCtl c = *a.ctl;
  c.t += 1;
  c.b1t *= a.beta1;
  c.b2t *= a.beta2;
  c.ticket = 0;
  adam_derive(c, a.seed);
  *a.ctl = c;
}

// Elements of the group of N from `i` on that lie below n.
template <bool FULL, int N>
__device__ __forceinline__ int count_of(int64_t i, int64_t n) {
  if constexpr (FULL) return N;
  const int64_t k = n - i;
  return k < 0 ? 0 : k > N ? N : static_cast<int>(k);
}

// 32-bit moments.  Four groups of four elements per thread and piece (FULL:
// the piece is whole, and no access is guarded).
template <bool WB, bool GB, bool MASTER, bool FULL>
__device__ __forceinline__ void piece32(const StepValues& s, const AdamDesc& d, int64_t base) {
  constexpr int G = kAdamPiece / (4 * kAdamThreads);
  const float adam = s.lr * d.lr_scale * s.rb1, decay = s.lr * d.weight_decay;
  float g[G][4], w[G][4], m[G][4], v[G][4];
  int cnt[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t i = base + j * 4 * kAdamThreads;
    cnt[j] = count_of<FULL, 4>(i, d.n);
    load_group<GB>(d.g, i, cnt[j], g[j]);
    load_group<false>(d.m, i, cnt[j], m[j]);
    load_group<false>(d.v, i, cnt[j], v[j]);
    if constexpr (MASTER) load_group<false>(d.master, i, cnt[j], w[j]);
    else load_group<WB>(d.w, i, cnt[j], w[j]);
  }
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t i = base + j * 4 * kAdamThreads;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[j][e] = update(s, g[j][e], w[j][e], s.b1, s.b2, adam, decay, m[j][e], v[j][e]);
    store_group<false>(d.m, i, cnt[j], m[j]);
    store_group<false>(d.v, i, cnt[j], v[j]);
    if constexpr (MASTER) store_group<false>(d.master, i, cnt[j], w[j]);
    store_group<WB>(d.w, i, cnt[j], w[j]);
  }
}

template <bool WB, bool GB, bool MASTER>
__global__ __launch_bounds__(kAdamThreads) void k_adamw32(AdamArgs a, bool advance) {
  const StepValues s = step_values(a);
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t at = static_cast<int64_t>(pc.piece) * kAdamPiece;
    if (d.n - at >= kAdamPiece) piece32<WB, GB, MASTER, true>(s, d, at + 4 * threadIdx.x);
    else piece32<WB, GB, MASTER, false>(s, d, at + 4 * threadIdx.x);
  }
  finish_step(a, advance);
}

// 8-bit moments.  Two groups of eight elements per thread and piece.
template <bool WB, bool GB, bool MASTER, bool STOCHASTIC, bool FULL>
__device__ __forceinline__ void piece8(const StepValues& s, const AdamDesc& d, int64_t base) {
  constexpr int G = kAdamPiece / (8 * kAdamThreads);
  const float adam = s.lr * d.lr_scale * s.rb1, decay = s.lr * d.weight_decay;
  float g[G][8], w[G][8], ms[G], vs[G];
  uint2 mc[G], vc[G];
  int cnt[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t i = base + j * 8 * kAdamThreads;
    cnt[j] = count_of<FULL, 8>(i, d.n);
    // Lanes of a block without elements read the scale of the last block.
    const int64_t blk = (cnt[j] > 0 ? i : d.n - 1) / ADAMW_BLOCK;
    ms[j] = gmem(d.m_scale)[blk];
    vs[j] = gmem(d.v_scale)[blk];
    mc[j] = load_codes(d.m, i, cnt[j]);
    vc[j] = load_codes(d.v, i, cnt[j]);
    load_group<GB>(d.g, i, cnt[j], g[j]);
    if constexpr (MASTER) load_group<false>(d.master, i, cnt[j], w[j]);
    else load_group<WB>(d.w, i, cnt[j], w[j]);
  }
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t i = base + j * 8 * kAdamThreads;
    float m[8], v[8];
    decode8(mc[j], vc[j], m, v);
    const float fm = s.b1 * ms[j], fv = s.b2 * vs[j];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[j][e] = update(s, g[j][e], w[j][e], fm, fv, adam, decay, m[e], v[e]);
    if constexpr (MASTER) store_group<false>(d.master, i, cnt[j], w[j]);
    store_group<WB>(d.w, i, cnt[j], w[j]);
    float ms1, vs1;
    encode8<STOCHASTIC>(m, v, s.key, d.first + i, mc[j], vc[j], ms1, vs1);
    store_codes(d.m, i, cnt[j], mc[j]);
    store_codes(d.v, i, cnt[j], vc[j]);
    if ((threadIdx.x & 31) == 0 && cnt[j] > 0) {
      gmem(d.m_scale)[i / ADAMW_BLOCK] = ms1;
      gmem(d.v_scale)[i / ADAMW_BLOCK] = vs1;
    }
  }
}

template <bool WB, bool GB, bool MASTER, bool STOCHASTIC>
__global__ __launch_bounds__(kAdamThreads) void k_adamw8(AdamArgs a, bool advance) {
  const StepValues s = step_values(a);
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t at = static_cast<int64_t>(pc.piece) * kAdamPiece;
    if (d.n - at >= kAdamPiece) piece8<WB, GB, MASTER, STOCHASTIC, true>(s, d, at + 8 * threadIdx.x);
    else piece8<WB, GB, MASTER, STOCHASTIC, false>(s, d, at + 8 * threadIdx.x);
  }
  finish_step(a, advance);
}

__global__ void k_ctl(AdamCtl* ctl, AdamCtl value, bool set_step) {
  if (set_step) {
    ctl->b1t = value.b1t;
    ctl->b2t = value.b2t;
    ctl->t = value.t;
    ctl->rb1 = value.rb1;
    ctl->rb2 = value.rb2;
    ctl->key = value.key;
  } else {
    ctl->lr = value.lr;
  }
}

// ---------------------------------------------------------------------------
// The moments as values
// ---------------------------------------------------------------------------
template <bool BLOCK8, bool BF16, bool FULL>
__device__ __forceinline__ void piece_get(const AdamDesc& d, int64_t base, void* m_out, void* v_out) {
#pragma unroll
  for (int j = 0; j < kAdamPiece / (8 * kAdamThreads); ++j) {
    const int64_t i = base + j * 8 * kAdamThreads;
    const int cnt = count_of<FULL, 8>(i, d.n);
    float m[8], v[8];
    if constexpr (BLOCK8) {
      const int64_t blk = (cnt > 0 ? i : d.n - 1) / ADAMW_BLOCK;
      const float ms = gmem(d.m_scale)[blk], vs = gmem(d.v_scale)[blk];
      decode8(load_codes(d.m, i, cnt), load_codes(d.v, i, cnt), m, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] *= ms;
        v[e] *= vs;
      }
    } else {
      load_group<false>(d.m, i, cnt, m);
      load_group<false>(d.v, i, cnt, v);
    }
    store_group<BF16>(m_out, d.first + i, cnt, m);
    store_group<BF16>(v_out, d.first + i, cnt, v);
  }
}

template <bool BLOCK8, bool BF16>
__global__ __launch_bounds__(kAdamThreads) void k_get(AdamArgs a, void* m_out, void* v_out) {
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t at = static_cast<int64_t>(pc.piece) * kAdamPiece;
    if (d.n - at >= kAdamPiece) piece_get<BLOCK8, BF16, true>(d, at + 8 * threadIdx.x, m_out, v_out);
    else piece_get<BLOCK8, BF16, false>(d, at + 8 * threadIdx.x, m_out, v_out);
  }
}

template <bool BLOCK8, bool BF16, bool FULL>
__device__ __forceinline__ void piece_set(const AdamDesc& d, int64_t base, const void* m_in, const void* v_in) {
#pragma unroll
  for (int j = 0; j < kAdamPiece / (8 * kAdamThreads); ++j) {
    const int64_t i = base + j * 8 * kAdamThreads;
    const int cnt = count_of<FULL, 8>(i, d.n);
    float m[8], v[8];
    load_group<BF16>(m_in, d.first + i, cnt, m);
    load_group<BF16>(v_in, d.first + i, cnt, v);
    if constexpr (BLOCK8) {
      uint2 mc, vc;
      float ms, vs;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += 0.0f;   // -0 becomes +0
      encode8<false>(m, v, 0, 0, mc, vc, ms, vs);
      store_codes(d.m, i, cnt, mc);
      store_codes(d.v, i, cnt, vc);
      if ((threadIdx.x & 31) == 0 && cnt > 0) {
        gmem(d.m_scale)[i / ADAMW_BLOCK] = ms;
        gmem(d.v_scale)[i / ADAMW_BLOCK] = vs;
      }
    } else {
      store_group<false>(d.m, i, cnt, m);
      store_group<false>(d.v, i, cnt, v);
    }
  }
}

template <bool BLOCK8, bool BF16>
__global__ __launch_bounds__(kAdamThreads) void k_set(AdamArgs a, const void* m_in, const void* v_in) {
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t at = static_cast<int64_t>(pc.piece) * kAdamPiece;
    if (d.n - at >= kAdamPiece) piece_set<BLOCK8, BF16, true>(d, at + 8 * threadIdx.x, m_in, v_in);
    else piece_set<BLOCK8, BF16, false>(d, at + 8 * threadIdx.x, m_in, v_in);
  }
}

// At most `most` workgroups; a batch without elements still takes its step
// (the step number advances).
unsigned grid_of(const AdamArgs& a, int most) {
  return static_cast<unsigned>(a.npieces < 1 ? 1 : a.npieces < most ? a.npieces : most);
}

template <bool WB, bool GB, bool MASTER>
void launch_step(const AdamArgs& a, bool advance, hipStream_t s) {
  const dim3 threads(kAdamThreads);
  if (!a.block8)
    hipLaunchKernelGGL((k_adamw32<WB, GB, MASTER>), dim3(grid_of(a, kGrid32)), threads, 0, s, a, advance);
  else if (a.stochastic)
    hipLaunchKernelGGL((k_adamw8<WB, GB, MASTER, true>), dim3(grid_of(a, kGrid8)), threads, 0, s, a, advance);
  else
    hipLaunchKernelGGL((k_adamw8<WB, GB, MASTER, false>), dim3(grid_of(a, kGrid8)), threads, 0, s, a, advance);
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, bool advance, hipStream_t s) {
  const bool wb = a.w_dt == DT_BF16, gb = a.g_dt == DT_BF16;
  if (a.has_master) {
    if (gb) launch_step<true, true, true>(a, advance, s);
    else launch_step<true, false, true>(a, advance, s);
  } else if (wb) {
    if (gb) launch_step<true, true, false>(a, advance, s);
    else launch_step<true, false, false>(a, advance, s);
  } else {
    if (gb) launch_step<false, true, false>(a, advance, s);
    else launch_step<false, false, false>(a, advance, s);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_ctl(AdamCtl* ctl, const AdamCtl& value, bool set_step, hipStream_t s) {
  hipLaunchKernelGGL(k_ctl, dim3(1), dim3(1), 0, s, ctl, value, set_step);
  return hipGetLastError();
}

hipError_t launch_adamw_get(const AdamArgs& a, void* m, void* v, int32_t dt, hipStream_t s) {
  if (!a.npieces) return hipSuccess;
  const dim3 grid(grid_of(a, kGridState)), threads(kAdamThreads);
  const bool bf16 = dt == DT_BF16;
  if (a.block8) {
    if (bf16) hipLaunchKernelGGL((k_get<true, true>), grid, threads, 0, s, a, m, v);
    else hipLaunchKernelGGL((k_get<true, false>), grid, threads, 0, s, a, m, v);
  } else {
    if (bf16) hipLaunchKernelGGL((k_get<false, true>), grid, threads, 0, s, a, m, v);
    else hipLaunchKernelGGL((k_get<false, false>), grid, threads, 0, s, a, m, v);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_set(const AdamArgs& a, const void* m, const void* v, int32_t dt, hipStream_t s) {
  if (!a.npieces) return hipSuccess;
  const dim3 grid(grid_of(a, kGridState)), threads(kAdamThreads);
  const bool bf16 = dt == DT_BF16;
  if (a.block8) {
    if (bf16) hipLaunchKernelGGL((k_set<true, true>), grid, threads, 0, s, a, m, v);
    else hipLaunchKernelGGL((k_set<true, false>), grid, threads, 0, s, a, m, v);
  } else {
    if (bf16) hipLaunchKernelGGL((k_set<false, true>), grid, threads, 0, s, a, m, v);
    else hipLaunchKernelGGL((k_set<false, false>), grid, threads, 0, s, a, m, v);
  }
  return hipGetLastError();
}

}  // namespace muon
