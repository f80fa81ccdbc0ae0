// AdamW over many tensors: the step with 32- and 8-bit moments, and the
// moments as values.
#include "adamw.h"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// Eight elements per thread of a group, raw as loaded.  p is the group's base
// (the same for the whole workgroup) and `lane` the thread in it.  In a group
// that is not WHOLE, only `cnt` of the eight exist; the others read as zero
// and are not written.
//
// The eight are consecutive: 16 bytes of bf16 or 32 of float32, eight code
// bytes.  With SPLIT (whole groups only) a thread has four elements in each
// half of the group, so that a float32 access takes 16 bytes from each lane
// and neighbouring lanes touch neighbouring bytes.  Float32 stores of 32 bytes
// a lane in two halves fill half a line each: writing 39M moments as float32
// took 127 us that way with non-temporal stores and 103 us with plain ones,
// and takes 57 us with SPLIT.  The 8-bit step keeps its eight together, which
// makes its code accesses eight bytes long.
//
// Stores are non-temporal: nothing that a step writes is read again by it.
// 39M elements with 8-bit moments and float32 master weights: 172 us with
// plain stores, 153 us with these; loads past the caches were slower (215
// against 238 us with 32-bit moments).
// ---------------------------------------------------------------------------
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename V>
__device__ __forceinline__ V load_vec(const void* p, int k) {
  return reinterpret_cast<const MUON_GLOBAL V*>(gmem(static_cast<const char*>(p)))[k];
}

template <typename V>
__device__ __forceinline__ void store_vec(void* p, int k, V v) {
  __builtin_nontemporal_store(v, reinterpret_cast<MUON_GLOBAL V*>(gmem(static_cast<char*>(p))) + k);
}

template <bool BF16>
struct Raw8;
template <>
struct Raw8<true> {
  u32x4 a;
};
template <>
struct Raw8<false> {
  u32x4 a, b;
};

template <bool BF16, bool WHOLE, bool SPLIT = false>
__device__ __forceinline__ Raw8<BF16> load8(const void* p, int lane, int cnt) {
  Raw8<BF16> r;
  if constexpr (WHOLE && SPLIT) {
    if constexpr (BF16) {
      const u32x2 x = load_vec<u32x2>(p, lane), y = load_vec<u32x2>(p, lane + kAdamThreads);
      r.a = u32x4{x[0], x[1], y[0], y[1]};
    } else {
      r.a = load_vec<u32x4>(p, lane);
      r.b = load_vec<u32x4>(p, lane + kAdamThreads);
    }
    return r;
  }
  if (WHOLE || cnt == 8) {
    if constexpr (BF16) {
      r.a = load_vec<u32x4>(p, lane);
    } else {
      r.a = load_vec<u32x4>(p, 2 * lane);
      r.b = load_vec<u32x4>(p, 2 * lane + 1);
    }
    return r;
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 0;
    if (e >= cnt) continue;
    if constexpr (BF16) w[e] = gmem(static_cast<const uint16_t*>(p))[8 * lane + e];
    else w[e] = gmem(static_cast<const uint32_t*>(p))[8 * lane + e];
  }
  if constexpr (BF16) {
    r.a = u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
  } else {
    r.a = u32x4{w[0], w[1], w[2], w[3]};
    r.b = u32x4{w[4], w[5], w[6], w[7]};
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void floats8(const Raw8<BF16>& r, float (&out)[8]) {
  if constexpr (BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      out[2 * k] = __uint_as_float(r.a[k] << 16);
      out[2 * k + 1] = __uint_as_float(r.a[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      out[k] = __uint_as_float(r.a[k]);
      out[4 + k] = __uint_as_float(r.b[k]);
    }
  }
}

template <bool BF16, bool WHOLE, bool SPLIT = false>
__device__ __forceinline__ void store8(void* p, int lane, int cnt, const float (&v)[8]) {
  if (WHOLE || cnt == 8) {
    if constexpr (BF16 && WHOLE && SPLIT) {
      store_vec(p, lane, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
      store_vec(p, lane + kAdamThreads, u32x2{pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
    } else if constexpr (BF16) {
      store_vec(p, lane, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7])});
    } else {
      u32x4 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = __float_as_uint(v[k]);
        b[k] = __float_as_uint(v[4 + k]);
      }
      store_vec(p, WHOLE && SPLIT ? lane : 2 * lane, a);
      store_vec(p, WHOLE && SPLIT ? lane + kAdamThreads : 2 * lane + 1, b);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) store_elem(p, 8 * lane + e, BF16 ? DT_BF16 : DT_F32, v[e]);
}

template <bool WHOLE>
__device__ __forceinline__ u32x2 load_codes(const void* p, int lane, int cnt) {
  if (WHOLE || cnt == 8) return load_vec<u32x2>(p, lane);
  u32x2 w = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) w[e >> 2] |= static_cast<uint32_t>(gmem(static_cast<const uint8_t*>(p))[8 * lane + e]) << (8 * (e & 3));
  return w;
}

template <bool WHOLE>
__device__ __forceinline__ void store_codes(void* p, int lane, int cnt, u32x2 c) {
  if (WHOLE || cnt == 8) {
    store_vec(p, lane, c);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) gmem(static_cast<uint8_t*>(p))[8 * lane + e] = static_cast<uint8_t>(c[e >> 2] >> (8 * (e & 3)));
}

// Elements of this thread in a group of `left` elements.
__device__ __forceinline__ int count_of(int left) {
  const int k = left - 8 * static_cast<int>(threadIdx.x);
  return k < 0 ? 0 : k > 8 ? 8 : k;
}

// Address of element `at` of a tensor.
__device__ __forceinline__ void* elem_at(void* p, int64_t at, int size) { return static_cast<char*>(p) + at * size; }
__device__ __forceinline__ const void* elem_at(const void* p, int64_t at, int size) {
  return static_cast<const char*>(p) + at * size;
}

// ---------------------------------------------------------------------------
// 8-bit moments.  A block of 256 elements is half a wave's: 32 lanes of eight
// elements (16-byte bf16 and 8-byte code accesses; a block's maximum takes
// four DPP steps and one exchange of 16-lane rows, no LDS and no barrier).
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
  float vden;      // 1 / vinv: vs * 2^-40 or vs * 2^24
  uint32_t voff;   // code offset << 20
};

__device__ __forceinline__ BlockScale block_scale(uint32_t mbits, uint32_t vbits) {
  BlockScale b;
  // Below 2^-118 (0x04800000) 1 / ms would overflow: such a block is zero.
  b.ms = mbits >= 0x04800000u ? __uint_as_float(mbits) * 0x1p-8f : 0.0f;
  b.minv = b.ms > 0.0f ? __builtin_amdgcn_rcpf(b.ms) : 0.0f;
  b.vs = __uint_as_float(vbits);
  const bool big = b.vs >= 1.0f;
  b.vden = b.vs * (big ? 0x1p-40f : 0x1p24f);
  b.vinv = big ? __builtin_amdgcn_rcpf(b.vden) : __builtin_amdgcn_rcpf(b.vs * 0x1p32f) * 0x1p8f;
  if (vbits == 0) b.vinv = 0.0f;
  b.voff = big ? 1088u << 20 : 576u << 20;
  return b;
}

// x * inv, and with EXACT the quotient x / den that it stands for, to the last
// bit but for rare halfway cases (one correction by the remainder).
template <bool EXACT>
__device__ __forceinline__ float quotient(float x, float den, float inv) {
  const float q = x * inv;
  if constexpr (!EXACT) return q;
  return copysignf(__builtin_fmaf(__builtin_fmaf(-q, den, x), inv, q), x);   // -0 stays -0
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

// Rounds eight elements to codes (those that do not exist are zero).  `hash0`
// is what the first one's hash mixes; the next ones follow it.
//
// Rounding adds to the 20 float32 mantissa bits that a code drops: 16 r + 8
// (stochastic) or half of their range (nearest), then cuts.  For m,
// v_cvt_sr_fp8_f32 does that with the upper 20 bits of its random operand,
// subnormal codes included (checked against the addition written out, over
// 4M values: equal in the normal range, and within 2^-20 of a code step of
// the border below it).  The block's largest |m| and v are a few ulp off
// their code's value at most, which neither rounding can carry to the next
// code.  A stochastic rounding may take quotients that are an ulp off
// (its random number is coarser); nearest rounding takes exact ones, so that
// values halfway between two codes (bf16 ones often are) round as stated.
template <bool STOCHASTIC>
__device__ __forceinline__ void encode8(const float (&m)[8], const float (&v)[8], uint32_t hash0, u32x2& mc,
                                        u32x2& vc, float& ms, float& vs) {
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
  int q[2] = {0, 0};
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t rm = 0x80000000u, t = __float_as_uint(quotient<!STOCHASTIC>(v[e], b.vden, b.vinv)) + vadd;
    if constexpr (STOCHASTIC) {
      const uint32_t h = adam_mix(hash0 + e);
      rm = h << 16 | 0x8000u;
      t = add_upper16(h, t);
    }
    const float y = quotient<!STOCHASTIC>(m[e], b.ms, b.minv);
    int& w = q[e >> 2];
    switch (e & 3) {
      case 0: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 0); break;
      case 1: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 1); break;
      case 2: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 2); break;
      default: w = __builtin_amdgcn_cvt_sr_fp8_f32(y, rm, w, 3); break;
    }
    c[e] = static_cast<uint32_t>(max(static_cast<int>(t) >> 20, nonzero(v[e])));   // v > 0 has a code above 0
  }
  mc = u32x2{static_cast<uint32_t>(q[0]), static_cast<uint32_t>(q[1])};
  if (odd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t byte = 0xFFu << (8 * (e & 3)), nan = 0x7Fu << (8 * (e & 3));
      if (mbad >> e & 1) mc[e >> 2] = (mc[e >> 2] & ~byte) | nan;
      if (vbad >> e & 1) c[e] = 255;
    }
  }
  vc = u32x2{c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
}

// Unscaled values of eight codes.
__device__ __forceinline__ void decode8(u32x2 mc, u32x2 vc, float (&m)[8], float (&v)[8]) {
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

__device__ __forceinline__ StepValues step_values(const AdamArgs& a, const AdamCtl& c) {
  StepValues s;
  s.b1 = static_cast<float>(a.beta1);
  s.b2 = static_cast<float>(a.beta2);
  s.eps = a.eps;
  s.lr = c.lr;
  s.rb1 = c.rb1;
  s.rb2 = c.rb2;
  s.key = c.key;
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

// Counts the workgroups that hold the step's values: called by every thread
// (a barrier that waits for scalar loads only).  The count is looked at after
// the step's work.
__device__ __forceinline__ uint32_t have_values(const AdamArgs& a, const AdamCtl& c, bool advance) {
  if (!advance) return 0;   // nobody will write the next step's
  asm volatile("s_waitcnt lgkmcnt(0)" ::"s"(c.lr), "s"(c.rb1), "s"(c.rb2), "s"(c.key) : "memory");
  __builtin_amdgcn_s_barrier();
  return threadIdx.x == 0 ? ticket_take(a.tickets) : 0;
}

// The last workgroup to have read the step's values writes the next step's.
__device__ __forceinline__ void advance_step(const AdamArgs& a, AdamCtl c, uint32_t seen) {
  if (threadIdx.x != 0 || !ticket_last(a.tickets, seen)) return;
  c.t += 1;
  c.b1t *= a.beta1;
  c.b2t *= a.beta2;
  adam_derive(c, a.seed);
  *a.ctl = c;
}

// A group's operands as loaded (kAdamGroup elements from element `at` of its
// tensor on, `left` of them in a group that is not WHOLE).
template <bool WB, bool GB, bool MASTER>
struct Group32 {
  static constexpr bool kBlock8 = false;
  Raw8<GB> g;
  Raw8<WB && !MASTER> w;
  Raw8<false> m, v;
};

template <bool WB, bool GB, bool MASTER, bool WHOLE>
__device__ __forceinline__ void load_group(const AdamDesc& d, int64_t at, int left, Group32<WB, GB, MASTER>& x) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  x.g = load8<GB, WHOLE, true>(elem_at(d.g, at, GB ? 2 : 4), lane, cnt);
  if constexpr (MASTER) x.w = load8<false, WHOLE, true>(elem_at(d.master, at, 4), lane, cnt);
  else x.w = load8<WB, WHOLE, true>(elem_at(d.w, at, WB ? 2 : 4), lane, cnt);
  x.m = load8<false, WHOLE, true>(elem_at(d.m, at, 4), lane, cnt);
  x.v = load8<false, WHOLE, true>(elem_at(d.v, at, 4), lane, cnt);
}

template <bool WB, bool GB, bool MASTER, bool STOCHASTIC, bool WHOLE>
__device__ __forceinline__ void step_group(const StepValues& s, const AdamDesc& d, int64_t at, int left,
                                           const Group32<WB, GB, MASTER>& x) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  const float adam = s.lr * d.lr_scale * s.rb1, decay = s.lr * d.weight_decay;
  float g[8], w[8], m[8], v[8];
  floats8(x.g, g);
  floats8(x.w, w);
  floats8(x.m, m);
  floats8(x.v, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = update(s, g[e], w[e], s.b1, s.b2, adam, decay, m[e], v[e]);
  if constexpr (MASTER) store8<false, WHOLE, true>(elem_at(d.master, at, 4), lane, cnt, w);
  store8<WB, WHOLE, true>(elem_at(d.w, at, WB ? 2 : 4), lane, cnt, w);
  store8<false, WHOLE, true>(elem_at(d.m, at, 4), lane, cnt, m);
  store8<false, WHOLE, true>(elem_at(d.v, at, 4), lane, cnt, v);
}

template <bool WB, bool GB, bool MASTER>
struct Group8 {
  static constexpr bool kBlock8 = true;
  Raw8<GB> g;
  Raw8<WB && !MASTER> w;
  u32x2 m, v;
  float ms, vs;
};

template <bool WB, bool GB, bool MASTER, bool WHOLE>
__device__ __forceinline__ void load_group(const AdamDesc& d, int64_t at, int left, Group8<WB, GB, MASTER>& x) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  x.g = load8<GB, WHOLE>(elem_at(d.g, at, GB ? 2 : 4), lane, cnt);
  if constexpr (MASTER) x.w = load8<false, WHOLE>(elem_at(d.master, at, 4), lane, cnt);
  else x.w = load8<WB, WHOLE>(elem_at(d.w, at, WB ? 2 : 4), lane, cnt);
  x.m = load_codes<WHOLE>(elem_at(d.m, at, 1), lane, cnt);
  x.v = load_codes<WHOLE>(elem_at(d.v, at, 1), lane, cnt);
  // A lane without elements takes the scale of the tensor's last block.
  const int blk = (WHOLE || cnt > 0 ? 8 * lane : left - 1) / ADAMW_BLOCK;
  x.ms = gmem(d.m_scale + at / ADAMW_BLOCK)[blk];
  x.vs = gmem(d.v_scale + at / ADAMW_BLOCK)[blk];
}

// What the hash of this thread's first element of the group mixes.
__device__ __forceinline__ uint32_t hash_base(const StepValues& s, const AdamDesc& d, int64_t at) {
  const uint64_t id = static_cast<uint64_t>(d.first + at);
  const uint32_t lo = static_cast<uint32_t>(id), hi = static_cast<uint32_t>(id >> 32);
  uint32_t k = adam_mix(s.key + hi);   // the same for the whole group, unless it passes a multiple of 2^32
  const uint32_t mine = lo + 8 * threadIdx.x;
  if (lo > 0xFFFFFFFFu - kAdamGroup && mine < lo) k = adam_mix(s.key + hi + 1);
  return mine + k;
}

template <bool WB, bool GB, bool MASTER, bool STOCHASTIC, bool WHOLE>
__device__ __forceinline__ void step_group(const StepValues& s, const AdamDesc& d, int64_t at, int left,
                                           const Group8<WB, GB, MASTER>& x) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  const float adam = s.lr * d.lr_scale * s.rb1, decay = s.lr * d.weight_decay;
  float g[8], w[8], m[8], v[8];
  floats8(x.g, g);
  floats8(x.w, w);
  decode8(x.m, x.v, m, v);
  const float fm = s.b1 * x.ms, fv = s.b2 * x.vs;
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = update(s, g[e], w[e], fm, fv, adam, decay, m[e], v[e]);
  if constexpr (MASTER) store8<false, WHOLE>(elem_at(d.master, at, 4), lane, cnt, w);
  store8<WB, WHOLE>(elem_at(d.w, at, WB ? 2 : 4), lane, cnt, w);
  u32x2 mc, vc;
  float ms, vs;
  encode8<STOCHASTIC>(m, v, STOCHASTIC ? hash_base(s, d, at) : 0, mc, vc, ms, vs);
  store_codes<WHOLE>(elem_at(d.m, at, 1), lane, cnt, mc);
  store_codes<WHOLE>(elem_at(d.v, at, 1), lane, cnt, vc);
  if ((lane & 31) == 0 && (WHOLE || cnt > 0)) {
    gmem(d.m_scale + at / ADAMW_BLOCK)[lane >> 5] = ms;
    gmem(d.v_scale + at / ADAMW_BLOCK)[lane >> 5] = vs;
  }
}

// The step reads and writes each element once and does 17 (32-bit moments) to
// 48 (8-bit, stochastic) vector instructions on it: memory bounds it, and for
// 8-bit moments the vector units are about three quarters busy beside it (the
// square root, the reciprocal and the hash's two products run at a quarter of
// the rate).
//   369M elements, bf16 weights and gradients
//     32-bit moments, 22 bytes an element   1337 us, 6.1 TB/s
//      8-bit moments, 10 bytes an element    610 us, 6.1 TB/s
//   39M elements, bf16 with float32 master weights
//     32-bit moments, 28 bytes               192 us, 5.8 TB/s
//      8-bit moments, 16 bytes               109 us, 5.8 TB/s
// A kernel that only streams through four arrays and writes three of them back
// reaches 6.0 TB/s on the same card.  (Cards differ: on another one the large
// 32-bit step took 1511 us and that kernel reached 5.4 TB/s.)
//
// One workgroup per unit, in the order of memory: measured against workgroups
// that walk several units each (1024 to 16384 of them, interleaved, the next
// unit's operands loaded ahead), which reached 4.6 to 5.1 TB/s where this
// reached 5.4.  Two groups a unit against one: 32-bit 1515 against 1540 us,
// 8-bit with its values 1076 against 1122 us (the slower card).
template <bool WB, bool GB, bool MASTER, bool STOCHASTIC, typename Group>
__device__ __forceinline__ void adamw_unit(const AdamArgs& a, bool advance) {
  const AdamCtl ctl = *a.ctl;
  const StepValues s = step_values(a, ctl);
  const AdamUnit u = a.units[blockIdx.x];
  const AdamDesc d = a.desc[u.tensor];
  const int64_t at = static_cast<int64_t>(u.unit) * kAdamUnit;
  Group x[kAdamGroups];
  // 32-bit moments count once the operands' loads are under way (against
  // counting before them: 50 vectors of 768 in 4.3 instead of 4.6 us, 39M
  // elements in 207 instead of 214), 8-bit ones before (4M elements: 16.7
  // against 18.1 us with the moments' values).
  constexpr bool kLate = !Group::kBlock8;
  uint32_t seen = 0;
  if constexpr (!kLate) seen = have_values(a, ctl, advance);
  if (blockIdx.x < a.nwhole) {
#pragma unroll
    for (int j = 0; j < kAdamGroups; ++j)
      load_group<WB, GB, MASTER, true>(d, at + j * kAdamGroup, kAdamGroup, x[j]);
    if constexpr (kLate) seen = have_values(a, ctl, advance);
#pragma unroll
    for (int j = 0; j < kAdamGroups; ++j)
      step_group<WB, GB, MASTER, STOCHASTIC, true>(s, d, at + j * kAdamGroup, kAdamGroup, x[j]);
  } else {
    int64_t from = at;
    int left = static_cast<int>(d.n - at);
    load_group<WB, GB, MASTER, false>(d, from, left, x[0]);
    if constexpr (kLate) seen = have_values(a, ctl, advance);
    for (;;) {
      step_group<WB, GB, MASTER, STOCHASTIC, false>(s, d, from, left, x[0]);
      from += kAdamGroup;
      left -= kAdamGroup;
      if (left <= 0) break;
      load_group<WB, GB, MASTER, false>(d, from, left, x[0]);
    }
  }
  if (advance) advance_step(a, ctl, seen);
}

template <bool WB, bool GB, bool MASTER>
__global__ __launch_bounds__(kAdamThreads) void k_adamw32(AdamArgs a, bool advance) {
  adamw_unit<WB, GB, MASTER, false, Group32<WB, GB, MASTER>>(a, advance);
}

template <bool WB, bool GB, bool MASTER, bool STOCHASTIC>
__global__ __launch_bounds__(kAdamThreads) void k_adamw8(AdamArgs a, bool advance) {
  adamw_unit<WB, GB, MASTER, STOCHASTIC, Group8<WB, GB, MASTER>>(a, advance);
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
// The moments as values.  Memory bounds both directions.
//   8-bit codes of 39M elements to float32: 56 us, 7.0 TB/s (the Infinity Cache
//     takes part of the writes)
//   8-bit codes of 369M elements to bf16: 357 us, 6.2 TB/s
//   float32 values of 369M elements to codes: 613 us, 6.0 TB/s
// ---------------------------------------------------------------------------
template <bool BLOCK8, bool BF16, bool WHOLE>
__device__ __forceinline__ void get_group(const AdamDesc& d, int64_t at, int left, void* m_out, void* v_out) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  constexpr int size = BF16 ? 2 : 4;
  constexpr bool kSplit = !BF16;   // float32 values: four elements in each half of the group
  float m[8], v[8];
  if constexpr (BLOCK8) {
    const float *msp = d.m_scale + at / ADAMW_BLOCK, *vsp = d.v_scale + at / ADAMW_BLOCK;
    float ms[2], vs[2];
    if constexpr (WHOLE && kSplit) {
      const void *mp = elem_at(d.m, at, 1), *vp = elem_at(d.v, at, 1);
      decode8(u32x2{load_vec<uint32_t>(mp, lane), load_vec<uint32_t>(mp, lane + kAdamThreads)},
              u32x2{load_vec<uint32_t>(vp, lane), load_vec<uint32_t>(vp, lane + kAdamThreads)}, m, v);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int blk = 4 * (lane + h * kAdamThreads) / ADAMW_BLOCK;
        ms[h] = gmem(msp)[blk];
        vs[h] = gmem(vsp)[blk];
      }
    } else {
      decode8(load_codes<WHOLE>(elem_at(d.m, at, 1), lane, cnt), load_codes<WHOLE>(elem_at(d.v, at, 1), lane, cnt), m,
              v);
      const int blk = (WHOLE || cnt > 0 ? 8 * lane : left - 1) / ADAMW_BLOCK;
      ms[0] = ms[1] = gmem(msp)[blk];
      vs[0] = vs[1] = gmem(vsp)[blk];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      m[e] *= ms[e >> 2];
      v[e] *= vs[e >> 2];
    }
  } else {
    floats8(load8<false, WHOLE, kSplit>(elem_at(d.m, at, 4), lane, cnt), m);
    floats8(load8<false, WHOLE, kSplit>(elem_at(d.v, at, 4), lane, cnt), v);
  }
  store8<BF16, WHOLE, kSplit>(elem_at(m_out, d.first + at, size), lane, cnt, m);
  store8<BF16, WHOLE, kSplit>(elem_at(v_out, d.first + at, size), lane, cnt, v);
}

template <bool BLOCK8, bool BF16, bool WHOLE>
__device__ __forceinline__ void set_group(const AdamDesc& d, int64_t at, int left, const void* m_in, const void* v_in) {
  const int lane = threadIdx.x, cnt = WHOLE ? 8 : count_of(left);
  constexpr int size = BF16 ? 2 : 4;
  float m[8], v[8];
  floats8(load8<BF16, WHOLE>(elem_at(m_in, d.first + at, size), lane, cnt), m);
  floats8(load8<BF16, WHOLE>(elem_at(v_in, d.first + at, size), lane, cnt), v);
  if constexpr (BLOCK8) {
    u32x2 mc, vc;
    float ms, vs;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += 0.0f;   // -0 becomes +0
    encode8<false>(m, v, 0, mc, vc, ms, vs);
    store_codes<WHOLE>(elem_at(d.m, at, 1), lane, cnt, mc);
    store_codes<WHOLE>(elem_at(d.v, at, 1), lane, cnt, vc);
    if ((lane & 31) == 0 && cnt > 0) {
      gmem(d.m_scale + at / ADAMW_BLOCK)[lane >> 5] = ms;
      gmem(d.v_scale + at / ADAMW_BLOCK)[lane >> 5] = vs;
    }
  } else {
    store8<false, WHOLE>(elem_at(d.m, at, 4), lane, cnt, m);
    store8<false, WHOLE>(elem_at(d.v, at, 4), lane, cnt, v);
  }
}

// Calls whole(desc, at) or part(desc, at, left) for this workgroup's group
// (kAdamGroups workgroups to a unit).
template <typename Whole, typename Part>
__device__ __forceinline__ void one_group(const AdamArgs& a, Whole whole, Part part) {
  const uint32_t k = blockIdx.x / kAdamGroups;
  const AdamUnit u = a.units[k];
  const AdamDesc d = a.desc[u.tensor];
  const int64_t at = static_cast<int64_t>(u.unit) * kAdamUnit + blockIdx.x % kAdamGroups * kAdamGroup;
  if (k < a.nwhole) whole(d, at);
  else if (d.n > at) part(d, at, static_cast<int>(min(d.n - at, static_cast<int64_t>(kAdamGroup))));
}

template <bool BLOCK8, bool BF16>
__global__ __launch_bounds__(kAdamThreads) void k_get(AdamArgs a, void* m, void* v) {
  one_group(
      a, [&](const AdamDesc& d, int64_t at) { get_group<BLOCK8, BF16, true>(d, at, kAdamGroup, m, v); },
      [&](const AdamDesc& d, int64_t at, int left) { get_group<BLOCK8, BF16, false>(d, at, left, m, v); });
}

template <bool BLOCK8, bool BF16>
__global__ __launch_bounds__(kAdamThreads) void k_set(AdamArgs a, const void* m, const void* v) {
  one_group(
      a, [&](const AdamDesc& d, int64_t at) { set_group<BLOCK8, BF16, true>(d, at, kAdamGroup, m, v); },
      [&](const AdamDesc& d, int64_t at, int left) { set_group<BLOCK8, BF16, false>(d, at, left, m, v); });
}

// A batch without elements still takes its step: one thread advances the
// step number.
__global__ void k_adamw_empty(AdamArgs a) { advance_step(a, *a.ctl, ticket_take(a.tickets)); }

template <bool WB, bool GB, bool MASTER>
void launch_step(const AdamArgs& a, bool advance, hipStream_t s) {
  const dim3 grid(a.nunits), threads(kAdamThreads);
  if (!a.block8) hipLaunchKernelGGL((k_adamw32<WB, GB, MASTER>), grid, threads, 0, s, a, advance);
  else if (a.stochastic) hipLaunchKernelGGL((k_adamw8<WB, GB, MASTER, true>), grid, threads, 0, s, a, advance);
  else hipLaunchKernelGGL((k_adamw8<WB, GB, MASTER, false>), grid, threads, 0, s, a, advance);
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, bool advance, hipStream_t s) {
  if (a.nunits == 0) {
    if (advance) hipLaunchKernelGGL(k_adamw_empty, dim3(1), dim3(1), 0, s, a);
    return hipGetLastError();
  }
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
  if (a.nunits == 0) return hipSuccess;
  const dim3 grid(a.nunits * kAdamGroups), threads(kAdamThreads);
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
  if (a.nunits == 0) return hipSuccess;
  const dim3 grid(a.nunits * kAdamGroups), threads(kAdamThreads);
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
