// Host side of AdamW and of the global gradient norm: argument validation,
// descriptor tables, launches, plans.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <stdexcept>
#include <vector>

#include "adamw.h"
#include "host.h"
#include "muon_mi355x.h"

namespace muon {
namespace {

constexpr int64_t kMaxTensors = int64_t{1} << 20;
constexpr int64_t kMaxElems = int64_t{1} << 40;
// Workgroups of one launch: its threads, 256 times as many, are below 2^32.
constexpr int64_t kMaxLeaves = (int64_t{1} << 24) - 1, kMaxUnits = kMaxLeaves / kAdamGroups;
constexpr int64_t kMaxStep = int64_t{1} << 62;

// Makes a plan's device current for one call.
struct DeviceGuard {
  int before = -1;
  hipError_t err;
  explicit DeviceGuard(int dev) {
    int cur = -1;
    err = hipGetDevice(&cur);
    if (err == hipSuccess && cur != dev) {
      err = hipSetDevice(dev);
      if (err == hipSuccess) before = cur;
    }
  }
  ~DeviceGuard() {
    if (before >= 0) (void)hipSetDevice(before);
  }
};

// No C++ exception leaves a C entry point.
template <typename F>
muon_status_t guarded(F&& f) {
  try {
    g_last_error.clear();
    return f();
  } catch (const std::bad_alloc&) {
  } catch (const std::length_error&) {
  }
  return fail(MUON_ERR_MEMORY, "host memory exhausted");
}

// A copy from a staging buffer that is used again cannot be part of a
// captured graph: calls that upload a table are refused under capture, before
// they touch a staging buffer.
muon_status_t refuse_capture(hipStream_t s) {
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  MUON_HIP_TRY(hipStreamIsCapturing(s, &cap));
  if (cap != hipStreamCaptureStatusNone)
    return fail(MUON_ERR_UNSUPPORTED, "the descriptor upload cannot be captured: create a plan before the capture");
  return MUON_OK;
}

muon_status_t check_workspace(void* ws, size_t have, size_t need, std::vector<Range>& rs) {
  if (!ws) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign != 0) return fail(MUON_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (have < need) return fail(MUON_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", have, need);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(ws), hi = lo + need;
  for (const Range& r : rs)
    if (r.lo < hi && lo < r.hi)
      return fail(MUON_ERR_ALIAS, "%s of tensor %lld overlaps the workspace", r.what, (long long)r.mat);
  return MUON_OK;
}

muon_status_t add_buffer(std::vector<Range>& rs, int64_t i, const void* p, size_t bytes, size_t align,
                         const char* what, bool writable) {
  if (!p) return fail(MUON_ERR_INVALID_ARG, "tensor %lld: %s is NULL", (long long)i, what);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (lo % align != 0)
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: %s is not %zu-byte aligned", (long long)i, what, align);
  rs.push_back({lo, lo + bytes, i, what, writable});
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
struct AdamTable {
  std::vector<AdamDesc> desc;
  std::vector<AdamUnit> units;
  int64_t nunits = 0, nwhole = 0, elems = 0;
  bool has_master = false;
  size_t ticket_off = 0, desc_off = 0, unit_off = 0, bytes = 0;
  std::vector<Range> buffers;
};

muon_status_t adam_check_config(const adamw_config_t* cfg) {
  if (!cfg) return fail(MUON_ERR_INVALID_ARG, "cfg is NULL");
  for (int32_t dt : {static_cast<int32_t>(cfg->w_dtype), static_cast<int32_t>(cfg->g_dtype)})
    if (dt != MUON_F32 && dt != MUON_BF16) return fail(MUON_ERR_DTYPE, "unknown dtype %d", dt);
  if (cfg->state != ADAMW_STATE_F32 && cfg->state != ADAMW_STATE_BLOCK8)
    return fail(MUON_ERR_DTYPE, "unknown moment format %d", cfg->state);
  if (cfg->rounding != ADAMW_ROUND_NEAREST && cfg->rounding != ADAMW_ROUND_STOCHASTIC)
    return fail(MUON_ERR_INVALID_ARG, "unknown rounding %d", cfg->rounding);
  for (double b : {cfg->beta1, cfg->beta2})
    if (!(b >= 0.0 && b < 1.0)) return fail(MUON_ERR_INVALID_ARG, "beta %g outside [0, 1)", b);
  if (!finite(cfg->lr)) return fail(MUON_ERR_INVALID_ARG, "lr must be finite");
  if (!finite(cfg->eps) || cfg->eps < 0.0f) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (reinterpret_cast<uintptr_t>(cfg->grad_scale) % 4 != 0)
    return fail(MUON_ERR_INVALID_ARG, "grad_scale is not 4-byte aligned");
  return MUON_OK;
}

// Sizes only: the workspace layout of a batch.
template <typename T>
muon_status_t check_count(const T* items, int64_t count) {
  if (!items) return fail(MUON_ERR_INVALID_ARG, "the tensor list is NULL");
  if (count < 1) return fail(MUON_ERR_INVALID_ARG, "count %lld < 1", (long long)count);
  if (count > kMaxTensors) return fail(MUON_ERR_UNSUPPORTED, "count %lld above %lld", (long long)count,
                                       (long long)kMaxTensors);
  for (int64_t i = 0; i < count; ++i) {
    if (items[i].n < 0) return fail(MUON_ERR_INVALID_ARG, "tensor %lld: n %lld < 0", (long long)i, (long long)items[i].n);
    if (items[i].n > kMaxElems) return fail(MUON_ERR_UNSUPPORTED, "tensor %lld: n %lld above %lld", (long long)i,
                                            (long long)items[i].n, (long long)kMaxElems);
  }
  return MUON_OK;
}

muon_status_t adam_layout(const adamw_tensor_t* ts, int64_t count, AdamTable& t) {
  muon_status_t st;
  if ((st = check_count(ts, count)) != MUON_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    t.nunits += ceil_div(ts[i].n, kAdamUnit);
    t.nwhole += ts[i].n / kAdamUnit;
    t.elems += round_up(ts[i].n, ADAMW_BLOCK);
  }
  if (t.nunits > kMaxUnits) return fail(MUON_ERR_UNSUPPORTED, "the batch is too large");
  t.ticket_off = round_up(sizeof(AdamCtl), kAlign);
  t.desc_off = round_up(t.ticket_off + sizeof(Ticket) * tickets_of(std::max<int64_t>(1, t.nunits)), kAlign);
  t.unit_off = round_up(t.desc_off + sizeof(AdamDesc) * count, kAlign);
  t.bytes = round_up(t.unit_off + sizeof(AdamUnit) * t.nunits, kAlign);
  return MUON_OK;
}

muon_status_t adam_prepare(const adamw_tensor_t* ts, int64_t count, const adamw_config_t* cfg, int64_t done,
                           void* ws, size_t ws_bytes, AdamTable& t, AdamCtl& ctl, std::vector<unsigned char>& table) {
  muon_status_t st;
  if ((st = adam_check_config(cfg)) != MUON_OK) return st;
  if ((st = adam_layout(ts, count, t)) != MUON_OK) return st;
  const bool block8 = cfg->state == ADAMW_STATE_BLOCK8;
  const size_t wsz = dtype_size(cfg->w_dtype), gsz = dtype_size(cfg->g_dtype), ssz = block8 ? 1 : 4;
  t.buffers.reserve(count * 7 + 1);
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    const adamw_tensor_t& x = ts[i];
    if (!finite(x.lr_scale) || !finite(x.weight_decay))
      return fail(MUON_ERR_INVALID_ARG, "tensor %lld: lr_scale and weight_decay must be finite", (long long)i);
    if (x.n == 0) continue;
    const size_t n = static_cast<size_t>(x.n), blocks = ceil_div(x.n, ADAMW_BLOCK);
    if ((st = add_buffer(t.buffers, i, x.w, n * wsz, 16, "w", true)) != MUON_OK ||
        (st = add_buffer(t.buffers, i, x.g, n * gsz, 16, "g", false)) != MUON_OK ||
        (st = add_buffer(t.buffers, i, x.m, n * ssz, 16, "m", true)) != MUON_OK ||
        (st = add_buffer(t.buffers, i, x.v, n * ssz, 16, "v", true)) != MUON_OK)
      return st;
    if (block8 && ((st = add_buffer(t.buffers, i, x.m_scale, blocks * 4, 4, "m_scale", true)) != MUON_OK ||
                   (st = add_buffer(t.buffers, i, x.v_scale, blocks * 4, 4, "v_scale", true)) != MUON_OK))
      return st;
    const bool master = x.master != nullptr;
    if (master && cfg->w_dtype != MUON_BF16)
      return fail(MUON_ERR_DTYPE, "tensor %lld: master weights go with bf16 weights", (long long)i);
    if (any && master != t.has_master)
      return fail(MUON_ERR_INVALID_ARG, "tensor %lld: either all tensors have master weights or none", (long long)i);
    t.has_master = master;
    any = true;
    if (master && (st = add_buffer(t.buffers, i, x.master, n * 4, 16, "master", true)) != MUON_OK) return st;
  }
  if (cfg->grad_scale) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(cfg->grad_scale);
    t.buffers.push_back({lo, lo + 4, 0, "grad_scale", false});
  }
  if ((st = check_overlaps(t.buffers, "tensor")) != MUON_OK) return st;
  if ((st = check_workspace(ws, ws_bytes, t.bytes, t.buffers)) != MUON_OK) return st;

  t.desc.reserve(count);
  t.units.reserve(t.nunits);
  int64_t first = 0;
  for (int64_t i = 0; i < count; ++i) {
    const adamw_tensor_t& x = ts[i];
    t.desc.push_back({x.w, x.g, x.m, x.v, x.m_scale, x.v_scale, x.master, x.n, first, x.lr_scale, x.weight_decay});
    first += round_up(x.n, ADAMW_BLOCK);
    for (int64_t u = 0; u < x.n / kAdamUnit; ++u) t.units.push_back({static_cast<uint32_t>(i), static_cast<uint32_t>(u)});
  }
  for (int64_t i = 0; i < count; ++i)
    if (ts[i].n % kAdamUnit)
      t.units.push_back({static_cast<uint32_t>(i), static_cast<uint32_t>(ts[i].n / kAdamUnit)});

  ctl = AdamCtl{};
  ctl.t = done + 1;
  ctl.b1t = std::pow(cfg->beta1, static_cast<double>(ctl.t));
  ctl.b2t = std::pow(cfg->beta2, static_cast<double>(ctl.t));
  ctl.lr = cfg->lr;
  adam_derive(ctl, cfg->seed);
  table.assign(t.bytes, 0);
  std::memcpy(table.data(), &ctl, sizeof(ctl));
  std::memcpy(table.data() + t.desc_off, t.desc.data(), sizeof(AdamDesc) * count);
  if (t.nunits) std::memcpy(table.data() + t.unit_off, t.units.data(), sizeof(AdamUnit) * t.nunits);
  return MUON_OK;
}

AdamArgs adam_args(const AdamTable& t, const adamw_config_t& cfg, void* ws) {
  char* base = static_cast<char*>(ws);
  AdamArgs a{};
  a.desc = reinterpret_cast<const AdamDesc*>(base + t.desc_off);
  a.units = reinterpret_cast<const AdamUnit*>(base + t.unit_off);
  a.nunits = static_cast<uint32_t>(t.nunits);
  a.nwhole = static_cast<uint32_t>(t.nwhole);
  a.ctl = reinterpret_cast<AdamCtl*>(base);
  a.tickets = reinterpret_cast<Ticket*>(base + t.ticket_off);
  a.grad_scale = cfg.grad_scale;
  a.beta1 = cfg.beta1;
  a.beta2 = cfg.beta2;
  a.seed = cfg.seed;
  a.c1 = static_cast<float>(1.0 - cfg.beta1);
  a.root_c2 = static_cast<float>(std::sqrt(1.0 - cfg.beta2));
  a.eps = cfg.eps;
  a.w_dt = cfg.w_dtype;
  a.g_dt = cfg.g_dtype;
  a.block8 = cfg.state == ADAMW_STATE_BLOCK8 ? 1 : 0;
  a.stochastic = cfg.rounding == ADAMW_ROUND_STOCHASTIC ? 1 : 0;
  a.has_master = t.has_master ? 1 : 0;
  return a;
}

#define MUON_ONE_LAUNCH(kind, expr)                      \
  do {                                                   \
    g_hook.next = 0;                                     \
    MUON_HIP_TRY(hook_record(MUON_LAUNCH_START, s));     \
    MUON_HIP_TRY(expr);                                  \
    MUON_HIP_TRY(hook_record((kind), s));                \
    g_hook.last_count = g_hook.next;                     \
  } while (0)

// ---------------------------------------------------------------------------
// Gradient norm
// ---------------------------------------------------------------------------
struct NormTable {
  std::vector<NormLeaf> leaves;
  std::vector<NormNode> nodes;
  size_t nslots = 0;
  int64_t grad_bytes = 0;
  size_t leaf_off = 0, node_off = 0, arrived_off = 0, sum_off = 0, table_bytes = 0, bytes = 0;
};

// Links `count` sums in slots first .. first + count - 1, whose owners write
// their parent through set_parent(i, node), under one node (or, for one sum,
// no new node), whose sum goes to slot `top` of `tensor`.
template <typename SetParent>
void norm_tree(NormTable& t, uint32_t first, uint32_t count, uint32_t top, uint32_t tensor, SetParent set_parent) {
  std::vector<uint32_t> below;   // nodes of the level below; empty: the owners themselves
  for (;;) {
    const uint32_t groups = static_cast<uint32_t>(ceil_div(count, kNormChildren));
    std::vector<uint32_t> level;
    const uint32_t slots = static_cast<uint32_t>(t.nslots);
    if (groups > 1) t.nslots += groups;
    for (uint32_t k = 0; k < groups; ++k) {
      const uint32_t id = static_cast<uint32_t>(t.nodes.size()), c0 = k * kNormChildren;
      const uint32_t n = std::min<uint32_t>(kNormChildren, count - c0);
      NormNode node{first + c0, n, groups > 1 ? slots + k : top, kNone, groups > 1 ? kNone : tensor, {0, 0, 0}};
      t.nodes.push_back(node);
      for (uint32_t c = c0; c < c0 + n; ++c) {
        if (below.empty()) set_parent(c, id);
        else t.nodes[below[c]].parent = id;
      }
      level.push_back(id);
    }
    if (groups == 1) return;
    first = slots;
    count = groups;
    below.swap(level);
  }
}

muon_status_t norm_layout(const muon_grad_t* gs, int64_t count, NormTable& t) {
  muon_status_t st;
  if ((st = check_count(gs, count)) != MUON_OK) return st;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (gs[i].dtype != MUON_F32 && gs[i].dtype != MUON_BF16)
      return fail(MUON_ERR_DTYPE, "tensor %lld: unknown dtype %d", (long long)i, static_cast<int>(gs[i].dtype));
    total += std::max<int64_t>(1, ceil_div(gs[i].n, kNormLeafBytes / static_cast<int64_t>(dtype_size(gs[i].dtype))));
  }
  if (total > kMaxLeaves) return fail(MUON_ERR_UNSUPPORTED, "the batch is too large");
  t.leaves.reserve(total);
  // Slots 0 .. count - 1 hold the tensors' sums.
  t.nslots = count;
  struct Owner { uint32_t leaf, node; };   // what writes a tensor's sum
  std::vector<Owner> owner(count);
  for (int64_t i = 0; i < count; ++i) {
    const int64_t size = dtype_size(gs[i].dtype), most = kNormLeafBytes / size;
    t.grad_bytes += gs[i].n * size;
    const uint32_t n = static_cast<uint32_t>(std::max<int64_t>(1, ceil_div(gs[i].n, most)));
    const uint32_t leaf0 = static_cast<uint32_t>(t.leaves.size()), slot0 = static_cast<uint32_t>(t.nslots);
    const uint32_t ti = static_cast<uint32_t>(i);
    if (n > 1) t.nslots += n;
    for (uint32_t k = 0; k < n; ++k) {
      const int64_t at = k * most;
      t.leaves.push_back({static_cast<const char*>(gs[i].g) + at * size,
                          static_cast<uint32_t>(std::min(most, gs[i].n - at)), static_cast<int32_t>(gs[i].dtype),
                          n > 1 ? slot0 + k : ti, kNone, n > 1 ? kNone : ti, 0});
    }
    owner[i] = {leaf0, kNone};
    if (n > 1) {
      norm_tree(t, slot0, n, ti, ti, [&](uint32_t c, uint32_t node) { t.leaves[leaf0 + c].parent = node; });
      owner[i].node = static_cast<uint32_t>(t.nodes.size() - 1);
    }
  }
  if (count > 1) {
    const uint32_t top = static_cast<uint32_t>(t.nslots++);
    norm_tree(t, 0, static_cast<uint32_t>(count), top, kNone, [&](uint32_t c, uint32_t node) {
      if (owner[c].node != kNone) t.nodes[owner[c].node].parent = node;
      else t.leaves[owner[c].leaf].parent = node;
    });
  }
  t.arrived_off = 0;
  t.leaf_off = round_up(t.arrived_off + sizeof(Ticket) * t.nodes.size(), kAlign);
  t.node_off = round_up(t.leaf_off + sizeof(NormLeaf) * t.leaves.size(), kAlign);
  t.table_bytes = round_up(t.node_off + sizeof(NormNode) * t.nodes.size(), kAlign);
  t.sum_off = t.table_bytes;
  t.bytes = round_up(t.sum_off + sizeof(double) * t.nslots, kAlign);
  return MUON_OK;
}

muon_status_t norm_prepare(const muon_grad_t* gs, int64_t count, float max_norm, float* out, float* tensor_norms,
                           void* ws, size_t ws_bytes, NormTable& t, std::vector<unsigned char>& table) {
  muon_status_t st;
  if ((st = norm_layout(gs, count, t)) != MUON_OK) return st;
  if (!(max_norm > 0.0f)) return fail(MUON_ERR_INVALID_ARG, "max_norm must be above zero");
  if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
  std::vector<Range> rs;
  rs.reserve(count + 2);
  for (int64_t i = 0; i < count; ++i) {
    if (gs[i].n == 0) continue;
    if ((st = add_buffer(rs, i, gs[i].g, static_cast<size_t>(gs[i].n) * dtype_size(gs[i].dtype), 16, "g", false)) !=
        MUON_OK)
      return st;
  }
  if ((st = add_buffer(rs, 0, out, 8, 4, "out", true)) != MUON_OK) return st;
  if (tensor_norms &&
      (st = add_buffer(rs, 0, tensor_norms, static_cast<size_t>(count) * 4, 4, "tensor_norms", true)) != MUON_OK)
    return st;
  if ((st = check_overlaps(rs, "tensor")) != MUON_OK) return st;
  if ((st = check_workspace(ws, ws_bytes, t.bytes, rs)) != MUON_OK) return st;
  table.assign(t.table_bytes, 0);
  std::memcpy(table.data() + t.leaf_off, t.leaves.data(), sizeof(NormLeaf) * t.leaves.size());
  if (!t.nodes.empty()) std::memcpy(table.data() + t.node_off, t.nodes.data(), sizeof(NormNode) * t.nodes.size());
  return MUON_OK;
}

NormArgs norm_args(const NormTable& t, float max_norm, float* out, float* tensor_norms, void* ws) {
  char* base = static_cast<char*>(ws);
  NormArgs a{};
  a.leaves = reinterpret_cast<const NormLeaf*>(base + t.leaf_off);
  a.nodes = reinterpret_cast<const NormNode*>(base + t.node_off);
  a.arrived = reinterpret_cast<Ticket*>(base + t.arrived_off);
  a.sums = reinterpret_cast<double*>(base + t.sum_off);
  a.out = out;
  a.tensor_norms = tensor_norms;
  a.max_norm = max_norm;
  a.nleaves = static_cast<uint32_t>(t.leaves.size());
  a.stream = t.grad_bytes > (int64_t{256} << 20) ? 1 : 0;
  return a;
}

}  // namespace
}  // namespace muon

struct adamw_plan {
  adamw_config_t cfg;
  muon::AdamArgs args;
  std::vector<muon::Range> buffers;   // every buffer of the batch and the workspace
  int64_t elems = 0;
  int device = 0;
  muon::Staging staging;
};

struct muon_grad_norm_plan {
  muon::NormArgs args;
  int device = 0;
  muon::Staging staging;
};

namespace muon {
namespace {

muon_status_t check_values(const adamw_plan* plan, const void* m, const void* v, muon_dtype_t dtype) {
  if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
  if (dtype != MUON_F32 && dtype != MUON_BF16) return fail(MUON_ERR_DTYPE, "unknown dtype %d", static_cast<int>(dtype));
  if (plan->elems == 0) return MUON_OK;   // nothing is read or written
  const size_t bytes = static_cast<size_t>(plan->elems) * dtype_size(dtype);
  uintptr_t lo[2];
  const void* ps[2] = {m, v};
  for (int k = 0; k < 2; ++k) {
    lo[k] = reinterpret_cast<uintptr_t>(ps[k]);
    if (!ps[k]) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", k ? "v" : "m");
    if (lo[k] % 16 != 0) return fail(MUON_ERR_INVALID_ARG, "%s is not 16-byte aligned", k ? "v" : "m");
    for (const Range& r : plan->buffers)
      if (r.lo < lo[k] + bytes && lo[k] < r.hi)
        return fail(MUON_ERR_ALIAS, "the %s values overlap %s of tensor %lld", k ? "v" : "m", r.what, (long long)r.mat);
  }
  if (lo[0] < lo[1] + bytes && lo[1] < lo[0] + bytes) return fail(MUON_ERR_ALIAS, "the m and v values overlap");
  return MUON_OK;
}

}  // namespace
}  // namespace muon

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
extern "C" {

void adamw_config_default(adamw_config_t* cfg) {
  if (!cfg) return;
  std::memset(cfg, 0, sizeof(*cfg));
  cfg->beta1 = 0.9;
  cfg->beta2 = 0.999;
  cfg->lr = 1e-3f;
  cfg->eps = 1e-8f;
  cfg->w_dtype = MUON_BF16;
  cfg->g_dtype = MUON_BF16;
  cfg->state = ADAMW_STATE_F32;
  cfg->rounding = ADAMW_ROUND_STOCHASTIC;
}

muon_status_t adamw_workspace_bytes(const adamw_tensor_t* tensors, int64_t count, const adamw_config_t* cfg,
                                    size_t* bytes) {
  using namespace muon;
  return guarded([&] {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    muon_status_t st;
    AdamTable t;
    if ((st = adam_check_config(cfg)) != MUON_OK) return st;
    if ((st = adam_layout(tensors, count, t)) != MUON_OK) return st;
    *bytes = t.bytes;
    return MUON_OK;
  });
}

muon_status_t adamw_state_elems(const adamw_tensor_t* tensors, int64_t count, int64_t* elems) {
  using namespace muon;
  return guarded([&] {
    if (!elems) return fail(MUON_ERR_INVALID_ARG, "elems is NULL");
    AdamTable t;
    const muon_status_t st = adam_layout(tensors, count, t);
    if (st == MUON_OK) *elems = t.elems;
    return st;
  });
}

muon_status_t adamw_step(const adamw_tensor_t* tensors, int64_t count, const adamw_config_t* cfg, int64_t step,
                         void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (step < 1 || step > kMaxStep) return fail(MUON_ERR_INVALID_ARG, "step %lld outside [1, 2^62]", (long long)step);
    AdamTable t;
    AdamCtl ctl;
    std::vector<unsigned char> table;
    muon_status_t st = adam_prepare(tensors, count, cfg, step - 1, workspace, workspace_bytes, t, ctl, table);
    if (st != MUON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = refuse_capture(s)) != MUON_OK) return st;
    if ((st = g_pool.take()->upload(table, workspace, s)) != MUON_OK) return st;
    MUON_ONE_LAUNCH(MUON_LAUNCH_ADAMW, launch_adamw(adam_args(t, *cfg, workspace), false, s));
    return MUON_OK;
  });
}

muon_status_t adamw_plan_create(const adamw_tensor_t* tensors, int64_t count, const adamw_config_t* cfg,
                                int64_t steps_done, void* workspace, size_t workspace_bytes, void* stream,
                                adamw_plan_t** plan) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (steps_done < 0 || steps_done >= kMaxStep)
      return fail(MUON_ERR_INVALID_ARG, "steps_done %lld outside [0, 2^62)", (long long)steps_done);
    AdamTable t;
    AdamCtl ctl;
    std::vector<unsigned char> table;
    muon_status_t st = adam_prepare(tensors, count, cfg, steps_done, workspace, workspace_bytes, t, ctl, table);
    if (st != MUON_OK) return st;
    if ((st = refuse_capture(static_cast<hipStream_t>(stream))) != MUON_OK) return st;
    std::unique_ptr<adamw_plan, void (*)(adamw_plan*)> pl(new adamw_plan(), adamw_plan_destroy);
    const hipError_t e = hipGetDevice(&pl->device);
    if (e != hipSuccess) return fail(MUON_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if ((st = pl->staging.upload(table, workspace, static_cast<hipStream_t>(stream))) != MUON_OK) return st;
    pl->cfg = *cfg;
    pl->args = adam_args(t, *cfg, workspace);
    pl->elems = t.elems;
    pl->buffers.swap(t.buffers);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace);
    pl->buffers.push_back({lo, lo + t.bytes, 0, "workspace", true});
    *plan = pl.release();
    return MUON_OK;
  });
}

muon_status_t adamw_plan_step(adamw_plan_t* plan, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_ONE_LAUNCH(MUON_LAUNCH_ADAMW, launch_adamw(plan->args, true, s));
    return MUON_OK;
  });
}

muon_status_t adamw_plan_set_lr(adamw_plan_t* plan, float lr, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    if (!finite(lr)) return fail(MUON_ERR_INVALID_ARG, "lr must be finite");
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    AdamCtl c{};
    c.lr = lr;
    MUON_HIP_TRY(launch_adamw_ctl(plan->args.ctl, c, false, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  });
}

muon_status_t adamw_plan_set_step(adamw_plan_t* plan, int64_t steps_done, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    if (steps_done < 0 || steps_done >= kMaxStep)
      return fail(MUON_ERR_INVALID_ARG, "steps_done %lld outside [0, 2^62)", (long long)steps_done);
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    AdamCtl c{};
    c.t = steps_done + 1;
    c.b1t = std::pow(plan->cfg.beta1, static_cast<double>(c.t));
    c.b2t = std::pow(plan->cfg.beta2, static_cast<double>(c.t));
    adam_derive(c, plan->cfg.seed);
    MUON_HIP_TRY(launch_adamw_ctl(plan->args.ctl, c, true, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  });
}

muon_status_t adamw_plan_get_state(adamw_plan_t* plan, void* m, void* v, muon_dtype_t dtype, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    muon_status_t st = check_values(plan, m, v, dtype);
    if (st != MUON_OK) return st;
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_ONE_LAUNCH(MUON_LAUNCH_STATE_GET, launch_adamw_get(plan->args, m, v, dtype, s));
    return MUON_OK;
  });
}

muon_status_t adamw_plan_set_state(adamw_plan_t* plan, const void* m, const void* v, muon_dtype_t dtype,
                                   void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    muon_status_t st = check_values(plan, m, v, dtype);
    if (st != MUON_OK) return st;
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_ONE_LAUNCH(MUON_LAUNCH_STATE_SET, launch_adamw_set(plan->args, m, v, dtype, s));
    return MUON_OK;
  });
}

void adamw_plan_destroy(adamw_plan_t* plan) {
  if (!plan) return;
  plan->staging.release();
  delete plan;
}

muon_status_t muon_grad_norm_workspace_bytes(const muon_grad_t* grads, int64_t count, size_t* bytes) {
  using namespace muon;
  return guarded([&] {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    NormTable t;
    const muon_status_t st = norm_layout(grads, count, t);
    if (st == MUON_OK) *bytes = t.bytes;
    return st;
  });
}

muon_status_t muon_grad_norm(const muon_grad_t* grads, int64_t count, float max_norm, float* out,
                             float* tensor_norms, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    NormTable t;
    std::vector<unsigned char> table;
    muon_status_t st = norm_prepare(grads, count, max_norm, out, tensor_norms, workspace, workspace_bytes, t, table);
    if (st != MUON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = refuse_capture(s)) != MUON_OK) return st;
    if ((st = g_pool.take()->upload(table, workspace, s)) != MUON_OK) return st;
    MUON_ONE_LAUNCH(MUON_LAUNCH_GRAD_NORM, launch_grad_norm(norm_args(t, max_norm, out, tensor_norms, workspace), s));
    return MUON_OK;
  });
}

muon_status_t muon_grad_norm_plan_create(const muon_grad_t* grads, int64_t count, float max_norm, float* out,
                                         float* tensor_norms, void* workspace, size_t workspace_bytes, void* stream,
                                         muon_grad_norm_plan_t** plan) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    NormTable t;
    std::vector<unsigned char> table;
    muon_status_t st = norm_prepare(grads, count, max_norm, out, tensor_norms, workspace, workspace_bytes, t, table);
    if (st != MUON_OK) return st;
    if ((st = refuse_capture(static_cast<hipStream_t>(stream))) != MUON_OK) return st;
    std::unique_ptr<muon_grad_norm_plan, void (*)(muon_grad_norm_plan*)> pl(new muon_grad_norm_plan(), muon_grad_norm_plan_destroy);
    const hipError_t e = hipGetDevice(&pl->device);
    if (e != hipSuccess) return fail(MUON_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if ((st = pl->staging.upload(table, workspace, static_cast<hipStream_t>(stream))) != MUON_OK) return st;
    pl->args = norm_args(t, max_norm, out, tensor_norms, workspace);
    *plan = pl.release();
    return MUON_OK;
  });
}

muon_status_t muon_grad_norm_plan_run(muon_grad_norm_plan_t* plan, void* stream) {
  using namespace muon;
  return guarded([&]() -> muon_status_t {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    const DeviceGuard dev(plan->device);
    MUON_HIP_TRY(dev.err);
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_ONE_LAUNCH(MUON_LAUNCH_GRAD_NORM, launch_grad_norm(plan->args, s));
    return MUON_OK;
  });
}

void muon_grad_norm_plan_destroy(muon_grad_norm_plan_t* plan) {
  if (!plan) return;
  plan->staging.release();
  delete plan;
}

}  // extern "C"
