// AdamW and the global gradient norm: structures shared by the host planner
// and the kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "muon_mi355x.h"

namespace muon {

// Work is dealt in units of kAdamUnit elements of one tensor, a workgroup
// each (256 threads, kAdamGroups times eight elements per thread; the last
// unit of a tensor may be shorter).  A unit is a multiple of ADAMW_BLOCK, so a
// block of the 8-bit moments never spans two.
constexpr int kAdamThreads = 256;
constexpr int kAdamGroups = 2;
constexpr int kAdamGroup = 8 * kAdamThreads;
constexpr int kAdamUnit = kAdamGroups * kAdamGroup;

// Per-tensor descriptor (uploaded once per batch into the workspace).
struct alignas(16) AdamDesc {
  void* w;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t n;
  int64_t first;          // index of the tensor's first element in the batch (a multiple of ADAMW_BLOCK)
  float lr_scale;
  float weight_decay;
};

// One unit of work.  The whole units of all tensors come first, in memory
// order, then the tensors' short last ones.
struct alignas(8) AdamUnit {
  uint32_t tensor, unit;
};

// State of a plan's step sequence, in the workspace.  b1t, b2t and the values
// derived from them are those of the step to come; the last workgroup of a
// step advances them, so a captured step replays as the next one.
struct alignas(16) AdamCtl {
  double b1t, b2t;        // beta1^t, beta2^t
  int64_t t;              // number of the step to come, from 1 on
  float lr;
  float rb1;              // 1 / (1 - beta1^t)
  float rb2;              // 1 / sqrt(1 - beta2^t)
  uint32_t key;           // key of the rounding hash for step t
};

// Counts the workgroups of a launch, to find the last one.  An agent-scope
// add to one address takes about 14 ns whoever issues it (measured: 2048 of
// them held a launch back by 25 us), so the workgroups are spread over groups
// of kTicketGroup, each with a counter in a line of its own, and the last one
// of a group counts the group.  Ticket 0 counts the groups.
constexpr int kTicketGroup = 64;
struct alignas(128) Ticket {
  uint32_t count;
};
inline int64_t tickets_of(int64_t workgroups) { return 1 + (workgroups + kTicketGroup - 1) / kTicketGroup; }

struct AdamArgs {
  const AdamDesc* desc;
  const AdamUnit* units;
  uint32_t nunits, nwhole;   // all units, whole units
  AdamCtl* ctl;
  Ticket* tickets;
  const float* grad_scale;  // or NULL
  double beta1, beta2;
  uint64_t seed;
  float c1, root_c2;      // 1 - beta1, sqrt(1 - beta2)
  float eps;
  int32_t w_dt, g_dt;
  int32_t block8;         // 8-bit moments
  int32_t stochastic;
  int32_t has_master;
};

// The counter hash of the stochastic rounding: two rounds of xor-shift and
// multiply by odd constants (the fraction bits of sqrt 2 and sqrt 3), after
// which every output bit flips with probability 1/2 +- 0.004 for any flipped
// input bit.
__host__ __device__ inline uint32_t adam_mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

__host__ __device__ inline uint32_t adam_key(uint64_t seed, int64_t t) {
  const uint64_t u = static_cast<uint64_t>(t);
  uint32_t k = adam_mix(static_cast<uint32_t>(u >> 32) ^ 0x3C6EF372u);
  k = adam_mix(static_cast<uint32_t>(u) ^ k);
  k = adam_mix(static_cast<uint32_t>(seed >> 32) ^ k);
  return adam_mix(static_cast<uint32_t>(seed) ^ k);
}

#if defined(__HIPCC__)
// Adds this workgroup to its group; one thread calls it.  The counter's value
// before says whether it is the group's last.
__device__ __forceinline__ uint32_t ticket_take(Ticket* t) {
  return __hip_atomic_fetch_add(&t[1 + blockIdx.x / kTicketGroup].count, 1u, __ATOMIC_RELAXED,
                                __HIP_MEMORY_SCOPE_AGENT);
}

// Whether the workgroup that took `seen` is the launch's last.  The counters
// are zero again after the last one's call.
__device__ __forceinline__ bool ticket_last(Ticket* t, uint32_t seen) {
  const uint32_t groups = (gridDim.x + kTicketGroup - 1) / kTicketGroup, mine = blockIdx.x / kTicketGroup;
  const uint32_t members = mine + 1 < groups ? kTicketGroup : gridDim.x - mine * kTicketGroup;
  if (seen != members - 1) return false;
  __hip_atomic_store(&t[1 + mine].count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (groups == 1) return true;
  if (__hip_atomic_fetch_add(&t[0].count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != groups - 1) return false;
  __hip_atomic_store(&t[0].count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}
#endif

// Values of the step t = ctl.t, from b1t and b2t.
__host__ __device__ inline void adam_derive(AdamCtl& c, uint64_t seed) {
  c.rb1 = static_cast<float>(1.0 / (1.0 - c.b1t));
  c.rb2 = static_cast<float>(1.0 / sqrt(1.0 - c.b2t));
  c.key = adam_key(seed, c.t);
}

hipError_t launch_adamw(const AdamArgs& a, bool advance, hipStream_t s);
// Writes the step values (`set_step`) or only the learning rate.
hipError_t launch_adamw_ctl(AdamCtl* ctl, const AdamCtl& value, bool set_step, hipStream_t s);
hipError_t launch_adamw_get(const AdamArgs& a, void* m, void* v, int32_t dt, hipStream_t s);
hipError_t launch_adamw_set(const AdamArgs& a, const void* m, const void* v, int32_t dt, hipStream_t s);

// ---------------------------------------------------------------------------
// Global gradient norm
// ---------------------------------------------------------------------------
// Every workgroup sums a stretch of one tensor (a leaf).  The sums meet in a
// tree of nodes with at most 128 children: the last child to store its sum
// adds up its siblings', two per lane, and goes on to the parent.  A tensor's
// sum is the value of one leaf or node.  A level costs about 1 us, and a
// node's counter 14 ns a child where all arrive at once.  With 64, 128 and 256
// children a node (three sets of gradients in turn): 128 tensors of 4 leaves
// take 8.3 us (three levels), 7.5 (two) and 7.6; 129 of them 8.5, 8.7 and 7.6;
// 256 of them 10.7, 11.3 and 11.1; one tensor of 512 leaves 7.2, 7.9 and 9.4;
// 128 tensors of 176 leaves 117, 116 and 118.
constexpr int kNormThreads = 256;
constexpr int kNormLeafBytes = 32768;
constexpr int kNormChildren = 128;
constexpr uint32_t kNone = 0xFFFFFFFFu;

struct alignas(32) NormLeaf {
  const void* g;          // first element of the stretch
  uint32_t count;         // elements
  int32_t dt;
  uint32_t slot;          // where its sum goes
  uint32_t parent;        // node, or kNone
  uint32_t tensor;        // the tensor whose whole sum this is, or kNone
  uint32_t reserved0;
};

struct alignas(32) NormNode {
  uint32_t first, children;   // the children's sums are in slots first, first + 1, ...
  uint32_t slot, parent, tensor;
  uint32_t reserved0[3];
};

struct NormArgs {
  const NormLeaf* leaves;
  const NormNode* nodes;
  Ticket* arrived;             // per node: children that have stored their sums
  double* sums;                // by slot
  float* out;
  float* tensor_norms;         // or NULL
  float max_norm;
  uint32_t nleaves;
  int32_t stream;              // the gradients do not fit the Infinity Cache
};

hipError_t launch_grad_norm(const NormArgs& a, hipStream_t s);

}  // namespace muon
