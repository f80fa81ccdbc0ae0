// AdamW over many tensors: the step with 32- and 8-bit moments, and the
// moments as values.
#include "adamw.h"

namespace muon {
namespace {

constexpr float kMTop = 256.0f;   // code value of a block's largest |m|

// ---------------------------------------------------------------------------
// 8-bit codes.  `add` is what rounding adds to the 20 float32 mantissa bits
// that a code drops.
// ---------------------------------------------------------------------------
constexpr uint32_t kNearestAdd = 0x80000u;
__device__ __forceinline__ uint32_t add_of(uint32_t r16) { return r16 * 16u + 8u; }

__device__ __forceinline__ bool finite_f32(float x) { return fabsf(x) < __builtin_inff(); }

// e4m3 value of m at scale ms: below 2^-6 the step of e4m3 stays 2^-9, which
// is its step in [2^-6, 2^-5), so those values are rounded after adding 2^-6.
__device__ __forceinline__ uint8_t encode_m(float m, float ms, uint32_t add) {
  if (!finite_f32(m)) return 0x7F;
  const float y = ms > 0.0f ? fminf(fabsf(m) / ms, 448.0f) : 0.0f;
  const float off = y < 0.015625f ? 0.015625f : 0.0f;
  float q = __uint_as_float((__float_as_uint(y + off) + add) & 0xFFF00000u) - off;
  q = copysignf(q, m);
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xFF);   // exact
}

__device__ __forceinline__ float decode_m(uint8_t c, float ms) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 0) * ms;
}

__device__ __forceinline__ uint8_t encode_v(float v, float vs, uint32_t add) {
  if (!finite_f32(v) || v < 0.0f) return 255;
  if (v == 0.0f) return 0;
  const float y = fminf(v / vs, 1.0f);   // vs >= v > 0
  const int c = static_cast<int>((__float_as_uint(y) + add) >> 20) - 768;
  return static_cast<uint8_t>(c < 1 ? 1 : c);
}

__device__ __forceinline__ float decode_v(uint8_t c, float vs) {
  if (c == 0) return 0.0f;
  if (c == 255) return __builtin_nanf("");
  return __uint_as_float((static_cast<uint32_t>(c) + 768u) << 20) * vs;
}

// What an element adds to its block's maxima.
__device__ __forceinline__ float max_m_of(float m) { return finite_f32(m) ? fabsf(m) : 0.0f; }
__device__ __forceinline__ float max_v_of(float v) { return finite_f32(v) && v > 0.0f ? v : 0.0f; }

// ---------------------------------------------------------------------------
// One step
// ---------------------------------------------------------------------------
struct StepValues {
  float b1, c1, b2, c2, eps, lr, rb1, rb2, gs;
  uint32_t key;
};

__device__ __forceinline__ StepValues step_values(const AdamArgs& a) {
  StepValues s;
  s.b1 = static_cast<float>(a.beta1);
  s.c1 = static_cast<float>(1.0 - a.beta1);
  s.b2 = static_cast<float>(a.beta2);
  s.c2 = static_cast<float>(1.0 - a.beta2);
  s.eps = a.eps;
  s.lr = a.ctl->lr;
  s.rb1 = a.ctl->rb1;
  s.rb2 = a.ctl->rb2;
  s.key = a.ctl->key;
  s.gs = a.grad_scale ? *a.grad_scale : 1.0f;
  return s;
}

__device__ __forceinline__ float moments(const StepValues& s, float g, float w, float& m, float& v, float lr_scale,
                                         float wd) {
  const float y = g * s.gs;
  m = s.b1 * m + s.c1 * y;
  v = s.b2 * v + s.c2 * (y * y);
  const float upd = (m * s.rb1) / (sqrtf(v) * s.rb2 + s.eps);
  return w - s.lr * (lr_scale * upd + wd * w);
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

__global__ __launch_bounds__(kAdamThreads) void k_adamw(AdamArgs a, bool advance) {
  const StepValues s = step_values(a);
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t base = static_cast<int64_t>(pc.piece) * kAdamPiece;
    const int64_t end = base + kAdamPiece < d.n ? base + kAdamPiece : d.n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // One wave per block of 256, four elements per lane.
    for (int64_t b = base + wave * ADAMW_BLOCK; b < end; b += 4 * ADAMW_BLOCK) {
      float m[4], v[4];
      float mmax = 0.0f, vmax = 0.0f;
      const int64_t blk = b / ADAMW_BLOCK;
      const float ms = a.block8 ? d.m_scale[blk] : 0.0f, vs = a.block8 ? d.v_scale[blk] : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = b + 4 * lane + e;
        m[e] = 0.0f;
        v[e] = 0.0f;
        if (i >= end) continue;
        if (a.block8) {
          m[e] = decode_m(static_cast<const uint8_t*>(d.m)[i], ms);
          v[e] = decode_v(static_cast<const uint8_t*>(d.v)[i], vs);
        } else {
          m[e] = static_cast<const float*>(d.m)[i];
          v[e] = static_cast<const float*>(d.v)[i];
        }
        const float g = load_elem(d.g, i, a.g_dt);
        const float w = d.master ? d.master[i] : load_elem(d.w, i, a.w_dt);
        const float w1 = moments(s, g, w, m[e], v[e], d.lr_scale, d.weight_decay);
        if (d.master) d.master[i] = w1;
        store_elem(d.w, i, a.w_dt, w1);
        if (!a.block8) {
          static_cast<float*>(d.m)[i] = m[e];
          static_cast<float*>(d.v)[i] = v[e];
        }
        mmax = fmaxf(mmax, max_m_of(m[e]));
        vmax = fmaxf(vmax, max_v_of(v[e]));
      }
      if (!a.block8) continue;
      const float ms1 = wave_max(mmax) * (1.0f / kMTop), vs1 = wave_max(vmax);
      if (lane == 0) {
        d.m_scale[blk] = ms1;
        d.v_scale[blk] = vs1;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = b + 4 * lane + e;
        if (i >= end) continue;
        uint32_t am = kNearestAdd, av = kNearestAdd;
        if (a.stochastic) {
          const uint64_t id = static_cast<uint64_t>(d.first + i);
          const uint32_t h = adam_mix(static_cast<uint32_t>(id) +
                                      adam_mix(s.key + static_cast<uint32_t>(id >> 32)));
          am = add_of(h & 0xFFFFu);
          av = add_of(h >> 16);
        }
        static_cast<uint8_t*>(d.m)[i] = encode_m(m[e], ms1, am);
        static_cast<uint8_t*>(d.v)[i] = encode_v(v[e], vs1, av);
      }
    }
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
__global__ __launch_bounds__(kAdamThreads) void k_get(AdamArgs a, void* m_out, void* v_out, int32_t dt) {
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t base = static_cast<int64_t>(pc.piece) * kAdamPiece;
    const int64_t end = base + kAdamPiece < d.n ? base + kAdamPiece : d.n;
    for (int64_t i = base + threadIdx.x; i < end; i += kAdamThreads) {
      float m, v;
      if (a.block8) {
        m = decode_m(static_cast<const uint8_t*>(d.m)[i], d.m_scale[i / ADAMW_BLOCK]);
        v = decode_v(static_cast<const uint8_t*>(d.v)[i], d.v_scale[i / ADAMW_BLOCK]);
      } else {
        m = static_cast<const float*>(d.m)[i];
        v = static_cast<const float*>(d.v)[i];
      }
      store_elem(m_out, d.first + i, dt, m);
      store_elem(v_out, d.first + i, dt, v);
    }
  }
}

__global__ __launch_bounds__(kAdamThreads) void k_set(AdamArgs a, const void* m_in, const void* v_in, int32_t dt) {
  for (int64_t p = blockIdx.x; p < a.npieces; p += gridDim.x) {
    const AdamPiece pc = a.pieces[p];
    const AdamDesc& d = a.desc[pc.tensor];
    const int64_t base = static_cast<int64_t>(pc.piece) * kAdamPiece;
    const int64_t end = base + kAdamPiece < d.n ? base + kAdamPiece : d.n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t b = base + wave * ADAMW_BLOCK; b < end; b += 4 * ADAMW_BLOCK) {
      float m[4], v[4];
      float mmax = 0.0f, vmax = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = b + 4 * lane + e;
        m[e] = i < end ? load_elem(m_in, d.first + i, dt) : 0.0f;
        v[e] = i < end ? load_elem(v_in, d.first + i, dt) : 0.0f;
        mmax = fmaxf(mmax, max_m_of(m[e]));
        vmax = fmaxf(vmax, max_v_of(v[e]));
        if (i < end && !a.block8) {
          static_cast<float*>(d.m)[i] = m[e];
          static_cast<float*>(d.v)[i] = v[e];
        }
      }
      if (!a.block8) continue;
      const float ms = wave_max(mmax) * (1.0f / kMTop), vs = wave_max(vmax);
      if (lane == 0) {
        d.m_scale[b / ADAMW_BLOCK] = ms;
        d.v_scale[b / ADAMW_BLOCK] = vs;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = b + 4 * lane + e;
        if (i >= end) continue;
        static_cast<uint8_t*>(d.m)[i] = encode_m(m[e], ms, kNearestAdd);
        static_cast<uint8_t*>(d.v)[i] = encode_v(v[e], vs, kNearestAdd);
      }
    }
  }
}

unsigned grid_of(const AdamArgs& a) { return static_cast<unsigned>(a.npieces < 2048 ? a.npieces : 2048); }

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, bool advance, hipStream_t s) {
  // A batch without elements still takes its step (the step number advances).
  const unsigned grid = a.npieces ? grid_of(a) : 1;
  hipLaunchKernelGGL(k_adamw, dim3(grid), dim3(kAdamThreads), 0, s, a, advance);
  return hipGetLastError();
}

hipError_t launch_adamw_ctl(AdamCtl* ctl, const AdamCtl& value, bool set_step, hipStream_t s) {
  hipLaunchKernelGGL(k_ctl, dim3(1), dim3(1), 0, s, ctl, value, set_step);
  return hipGetLastError();
}

hipError_t launch_adamw_get(const AdamArgs& a, void* m, void* v, int32_t dt, hipStream_t s) {
  if (!a.npieces) return hipSuccess;
  hipLaunchKernelGGL(k_get, dim3(grid_of(a)), dim3(kAdamThreads), 0, s, a, m, v, dt);
  return hipGetLastError();
}

hipError_t launch_adamw_set(const AdamArgs& a, const void* m, const void* v, int32_t dt, hipStream_t s) {
  if (!a.npieces) return hipSuccess;
  hipLaunchKernelGGL(k_set, dim3(grid_of(a)), dim3(kAdamThreads), 0, s, a, m, v, dt);
  return hipGetLastError();
}

}  // namespace muon
