// Host side of the experts' operators: argument validation, workspaces and
// launches.
#include <algorithm>
#include <vector>

#include "expert.h"
#include "host.h"
#include "muon_mi355x.h"

namespace muon {
namespace {

constexpr int64_t kMaxSide = 65536, kMaxStride = int64_t{1} << 20, kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxGroups = 4096;

// A buffer of a call: `rows` rows of `width` bytes, `stride` bytes apart, in
// each of `groups` groups.
struct Buffer {
  uintptr_t at;
  int64_t rows, width, stride, groups, group_stride;
  const char* what;
  bool written;

  bool empty() const { return rows == 0 || width == 0 || groups == 0; }
  uintptr_t end() const { return at + (groups - 1) * group_stride + (rows - 1) * stride + width; }
};

// Whether two buffers may share a byte.  Rows of one stride that keep to
// columns of their own (views of one wide buffer) do not; a single row has any
// stride.
bool overlap(const Buffer& a, const Buffer& b) {
  if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
  if ((a.stride == b.stride || a.rows == 1 || b.rows == 1) && a.groups == 1 && b.groups == 1) {
    const Buffer& lo = a.at <= b.at ? a : b;
    const Buffer& hi = a.at <= b.at ? b : a;
    const int64_t stride = a.rows > 1 ? a.stride : b.stride;
    const int64_t d = static_cast<int64_t>((hi.at - lo.at) % static_cast<uintptr_t>(stride));
    if (lo.width <= d && d + hi.width <= stride) return false;
  }
  return true;
}

// Buffers of a call, checked as they are named.
struct Buffers {
  std::vector<Buffer> all;
  bool vec = true, dword = true;   // rows on 16-byte borders, on 4-byte borders

  muon_status_t add(const void* p, const char* what, int64_t rows, int64_t width, int64_t stride, size_t es, bool written,
                    int64_t groups = 1, int64_t group_stride = 0) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % es != 0)
      return fail(MUON_ERR_INVALID_ARG, "%s is not %zu-byte aligned", what, es);
    if (stride < width) return fail(MUON_ERR_INVALID_ARG, "%s: stride %lld < width %lld", what, (long long)stride, (long long)width);
    if (stride > kMaxStride)
      return fail(MUON_ERR_UNSUPPORTED, "%s: stride %lld above %lld", what, (long long)stride, (long long)kMaxStride);
    if (groups > 1 && group_stride < (rows - 1) * stride + width)
      return fail(MUON_ERR_INVALID_ARG, "%s: group stride %lld below a group's size", what, (long long)group_stride);
    if (groups > 1 && group_stride > kMaxSide * kMaxStride)
      return fail(MUON_ERR_UNSUPPORTED, "%s: group stride %lld too large", what, (long long)group_stride);
    const int64_t e = static_cast<int64_t>(es);
    const auto off = [&](int64_t n) {
      return reinterpret_cast<uintptr_t>(p) % n || stride * e % n || (groups > 1 && group_stride * e % n);
    };
    if (off(16)) vec = false;
    if (off(4)) dword = false;
    all.push_back({reinterpret_cast<uintptr_t>(p), rows, width * e, stride * e, groups, group_stride * e, what, written});
    return MUON_OK;
  }
  // A list of n values.
  muon_status_t list(const void* p, const char* what, int64_t n, size_t es, bool written) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % es != 0)
      return fail(MUON_ERR_INVALID_ARG, "%s is not %zu-byte aligned", what, es);
    const int64_t bytes = n * static_cast<int64_t>(es);
    all.push_back({reinterpret_cast<uintptr_t>(p), 1, bytes, bytes, 1, 0, what, written});
    return MUON_OK;
  }
  muon_status_t workspace(void* p, size_t have, size_t need) {
    if (need == 0) return MUON_OK;
    if (!p) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(p) % kAlign != 0) return fail(MUON_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (have < need) return fail(MUON_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", have, need);
    return list(p, "the workspace", static_cast<int64_t>(need), 1, true);
  }
  // Alignment of a product's rows (launch_linear).
  int align(int64_t in, int64_t out, size_t es) const {
    if (vec && in % 8 == 0 && out % 8 == 0) return 16;
    return dword && in * es % 4 == 0 && out * es % 4 == 0 ? 4 : 2;
  }
  // `same`: a written buffer that may be the read one itself.
  muon_status_t disjoint(const char* written = nullptr, const char* read = nullptr) const {
    for (size_t i = 0; i < all.size(); ++i)
      for (size_t j = i + 1; j < all.size(); ++j) {
        const Buffer &a = all[i], &b = all[j];
        if (!(a.written || b.written) || !overlap(a, b)) continue;
        const Buffer &w = a.written ? a : b, &r = a.written ? b : a;
        if (written && w.what == written && r.what == read && w.at == r.at && (w.stride == r.stride || w.rows == 1))
          continue;
        return fail(MUON_ERR_ALIAS, "%s overlaps %s", b.what, a.what);
      }
    return MUON_OK;
  }
};

#define MUON_CHECK(expr)                          \
  do {                                            \
    const muon_status_t st_ = (expr);             \
    if (st_ != MUON_OK) return st_;               \
  } while (0)

// Around a call's launches.
#define MUON_HOOK_START()                              \
  do {                                                 \
    g_hook.next = 0;                                   \
    MUON_HIP_TRY(hook_record(MUON_LAUNCH_START, s));   \
  } while (0)
muon_status_t launched() {
  g_hook.last_count = g_hook.next;
  return MUON_OK;
}
// A call that has nothing to launch (and so records no event).
muon_status_t no_launch() {
  g_hook.next = 0;
  return launched();
}

muon_status_t check_dtype(int32_t dt, const char* what) {
  if (dt != MUON_F32 && dt != MUON_BF16) return fail(MUON_ERR_DTYPE, "%s: unknown dtype %d", what, dt);
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------
muon_status_t check_counts(int64_t tokens, int32_t top, int32_t experts) {
  if (tokens < 0) return fail(MUON_ERR_INVALID_ARG, "tokens %lld < 0", (long long)tokens);
  if (top < 1) return fail(MUON_ERR_INVALID_ARG, "top %d < 1", top);
  if (top > kMaxExperts) return fail(MUON_ERR_UNSUPPORTED, "top %d above %d", top, kMaxExperts);
  if (experts < 1) return fail(MUON_ERR_INVALID_ARG, "experts %d < 1", experts);
  if (experts > kMaxExperts) return fail(MUON_ERR_UNSUPPORTED, "experts %d above %d", experts, kMaxExperts);
  if (tokens > kMaxRows / top) return fail(MUON_ERR_UNSUPPORTED, "more than 2^30 slots");
  return MUON_OK;
}

muon_status_t check_routes(const expert_routes_t* r, Buffers& b, bool written) {
  if (!r) return fail(MUON_ERR_INVALID_ARG, "routes is NULL");
  MUON_CHECK(check_counts(r->tokens, r->top, r->experts));
  const int64_t slots = r->tokens * r->top;
  if (written) {
    MUON_CHECK(b.list(r->offsets, "offsets", r->experts + 1, 4, true));
    if (slots) MUON_CHECK(b.list(r->order, "order", slots, 4, true));
  }
  if (slots) MUON_CHECK(b.list(r->place, "place", slots, 4, written));
  return MUON_OK;
}

size_t sort_bytes(int64_t slots, int32_t experts) {
  int64_t per, blocks;
  sort_shape(slots, per, blocks);
  return blocks > 1 ? static_cast<size_t>(round_up((blocks + 1) * (experts + 1) * 4, kAlign)) : 0;
}

muon_status_t check_width(int64_t width) {
  if (width < 1) return fail(MUON_ERR_INVALID_ARG, "width %lld < 1", (long long)width);
  if (width > kMaxSide) return fail(MUON_ERR_UNSUPPORTED, "width %lld above %lld", (long long)width, (long long)kMaxSide);
  return MUON_OK;
}

MoveArgs move_args(const expert_routes_t* r, int64_t width) {
  MoveArgs a{};
  a.place = r->place;
  a.tokens = static_cast<int32_t>(r->tokens);
  a.top = r->top;
  a.width = static_cast<int32_t>(width);
  a.slots = static_cast<int32_t>(r->tokens * r->top);
  return a;
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
template <typename A>
muon_status_t check_sizes(const A* a) {
  if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
  MUON_CHECK(check_dtype(a->dtype, "dtype"));
  if (a->rows < 0) return fail(MUON_ERR_INVALID_ARG, "rows %lld < 0", (long long)a->rows);
  if (a->rows >= kMaxRows) return fail(MUON_ERR_UNSUPPORTED, "rows %lld above 2^30 - 1", (long long)a->rows);
  for (int64_t n : {a->in, a->out}) {
    if (n < 1) return fail(MUON_ERR_INVALID_ARG, "in %lld, out %lld: below 1", (long long)a->in, (long long)a->out);
    if (n > kMaxSide)
      return fail(MUON_ERR_UNSUPPORTED, "in %lld, out %lld: above %lld", (long long)a->in, (long long)a->out,
                  (long long)kMaxSide);
  }
  if (a->groups < 1) return fail(MUON_ERR_INVALID_ARG, "groups %lld < 1", (long long)a->groups);
  if (a->groups > kMaxGroups)
    return fail(MUON_ERR_UNSUPPORTED, "groups %lld above %lld", (long long)a->groups, (long long)kMaxGroups);
  if (!a->offsets && a->groups != 1) return fail(MUON_ERR_INVALID_ARG, "%lld groups need offsets", (long long)a->groups);
  return MUON_OK;
}

muon_status_t check_activation(int32_t act) {
  if (act < LINEAR_NONE || act > LINEAR_SILU) return fail(MUON_ERR_INVALID_ARG, "unknown activation %d", act);
  return MUON_OK;
}

// What linear_grad keeps in its workspace.
struct GradLayout {
  int64_t dz_ld = 0;
  int parts = 1, bias_parts = 1;
  bool slope_sums = false;   // db from the pass that forms dz, whose terms are not rounded yet
  size_t dz = 0, part = 0, bias_part = 0, bytes = 0;
};

muon_status_t grad_layout(const linear_grad_args_t* a, GradLayout& l) {
  MUON_CHECK(check_sizes(a));
  MUON_CHECK(check_dtype(a->grad_dtype, "grad_dtype"));
  MUON_CHECK(check_activation(a->activation));
  MUON_CHECK(check_activation(a->x_activation));
  size_t at = 0;
  if (a->activation != LINEAR_NONE) {
    l.dz_ld = round_up(a->out, 8);
    l.dz = at;
    at += round_up(a->rows * l.dz_ld * static_cast<int64_t>(dtype_size(a->dtype)), kAlign);
  }
  if (a->dw) {
    l.parts = linear_weight_parts(a->rows, a->out, a->in, a->groups);
    l.part = at;
    if (l.parts > 1) at += round_up(l.parts * a->groups * a->out * a->in * 4, kAlign);
  }
  if (a->db && a->activation != LINEAR_NONE && a->dtype == MUON_BF16) {
    l.slope_sums = true;
    l.bias_part = at;
    at += round_up(linear_slope_tiles(a->rows, a->out, a->groups) * a->out * 4, kAlign);
  } else if (a->db) {
    l.bias_parts = linear_bias_parts(a->rows, a->groups);
    l.bias_part = at;
    if (l.bias_parts > 1) at += round_up(l.bias_parts * a->groups * a->out * 4, kAlign);
  }
  l.bytes = at;
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t expert_sort_workspace_bytes(int64_t tokens, int32_t top, int32_t experts, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    MUON_CHECK(check_counts(tokens, top, experts));
    *bytes = sort_bytes(tokens * top, experts);
    return MUON_OK;
  });
}

muon_status_t expert_sort(const void* ids, int32_t id_bytes, const expert_routes_t* routes, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    Buffers b;
    MUON_CHECK(check_routes(routes, b, true));
    if (id_bytes != 4 && id_bytes != 8) return fail(MUON_ERR_DTYPE, "ids of %d bytes", id_bytes);
    const int64_t slots = routes->tokens * routes->top;
    if (slots) MUON_CHECK(b.list(ids, "ids", slots, id_bytes, false));
    const size_t need = sort_bytes(slots, routes->experts);
    MUON_CHECK(b.workspace(workspace, workspace_bytes, need));
    MUON_CHECK(b.disjoint());
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Routes r{routes->offsets, routes->order, routes->place, static_cast<int32_t>(routes->tokens), routes->top,
                   routes->experts, static_cast<int32_t>(slots)};
    MUON_HOOK_START();
    MUON_LAUNCH(MUON_LAUNCH_EXPERT_SORT, launch_expert_sort(ids, id_bytes, r, static_cast<int32_t*>(workspace), s));
    return launched();
  });
}

muon_status_t expert_gather(const void* x, int64_t x_stride, int64_t width, muon_dtype_t dtype,
                            const expert_routes_t* routes, void* xs, int64_t xs_stride, void* stream) {
  return guarded([&]() -> muon_status_t {
    Buffers b;
    MUON_CHECK(check_dtype(dtype, "dtype"));
    MUON_CHECK(check_routes(routes, b, false));
    MUON_CHECK(check_width(width));
    MoveArgs a = move_args(routes, width);
    if (a.slots == 0) return no_launch();
    const size_t es = dtype_size(dtype);
    MUON_CHECK(b.add(x, "x", a.tokens, width, x_stride, es, false));
    MUON_CHECK(b.add(xs, "xs", a.slots, width, xs_stride, es, true));
    MUON_CHECK(b.disjoint());
    a.tok = x;
    a.tok_ld = x_stride;
    a.rows_out = xs;
    a.rows_out_ld = xs_stride;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_HOOK_START();
    MUON_LAUNCH(MUON_LAUNCH_EXPERT_GATHER, launch_expert_gather(a, dtype, b.vec && width * es % 16 == 0, s));
    return launched();
  });
}

muon_status_t expert_combine(const void* ys, int64_t ys_stride, int64_t width, muon_dtype_t dtype,
                             const expert_routes_t* routes, const void* weights, muon_dtype_t weights_dtype,
                             const void* residual, int64_t residual_stride, void* y, int64_t y_stride, void* stream) {
  return guarded([&]() -> muon_status_t {
    Buffers b;
    MUON_CHECK(check_dtype(dtype, "dtype"));
    MUON_CHECK(check_routes(routes, b, false));
    MUON_CHECK(check_width(width));
    MoveArgs a = move_args(routes, width);
    if (a.slots == 0) return no_launch();
    const size_t es = dtype_size(dtype);
    MUON_CHECK(b.add(ys, "ys", a.slots, width, ys_stride, es, false));
    if (weights) {
      MUON_CHECK(check_dtype(weights_dtype, "weights_dtype"));
      MUON_CHECK(b.list(weights, "weights", a.slots, dtype_size(weights_dtype), false));
    }
    static const char kResidual[] = "residual", kY[] = "y";
    if (residual) MUON_CHECK(b.add(residual, kResidual, a.tokens, width, residual_stride, es, false));
    MUON_CHECK(b.add(y, kY, a.tokens, width, y_stride, es, true));
    MUON_CHECK(b.disjoint(kY, kResidual));
    a.rows = ys;
    a.rows_ld = ys_stride;
    a.weights = weights;
    a.w_dt = weights_dtype;
    a.tok = residual;
    a.tok_ld = residual_stride;
    a.tok_out = y;
    a.tok_out_ld = y_stride;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_HOOK_START();
    MUON_LAUNCH(MUON_LAUNCH_EXPERT_COMBINE, launch_expert_combine(a, dtype, b.vec && width * es % 16 == 0, s));
    return launched();
  });
}

muon_status_t expert_combine_grad(const void* dy, int64_t dy_stride, const void* ys, int64_t ys_stride, int64_t width,
                                  muon_dtype_t dtype, const expert_routes_t* routes, const void* weights,
                                  muon_dtype_t weights_dtype, void* dys, int64_t dys_stride, void* dweights,
                                  void* stream) {
  return guarded([&]() -> muon_status_t {
    Buffers b;
    MUON_CHECK(check_dtype(dtype, "dtype"));
    MUON_CHECK(check_dtype(weights_dtype, "weights_dtype"));
    MUON_CHECK(check_routes(routes, b, false));
    MUON_CHECK(check_width(width));
    MoveArgs a = move_args(routes, width);
    if (a.slots == 0) return no_launch();
    const size_t es = dtype_size(dtype), ws = dtype_size(weights_dtype);
    MUON_CHECK(b.add(dy, "dy", a.tokens, width, dy_stride, es, false));
    MUON_CHECK(b.add(ys, "ys", a.slots, width, ys_stride, es, false));
    MUON_CHECK(b.list(weights, "weights", a.slots, ws, false));
    MUON_CHECK(b.add(dys, "dys", a.slots, width, dys_stride, es, true));
    MUON_CHECK(b.list(dweights, "dweights", a.slots, ws, true));
    MUON_CHECK(b.disjoint());
    a.tok = dy;
    a.tok_ld = dy_stride;
    a.rows = ys;
    a.rows_ld = ys_stride;
    a.rows_out = dys;
    a.rows_out_ld = dys_stride;
    a.weights = weights;
    a.dweights = dweights;
    a.w_dt = weights_dtype;
    hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_HOOK_START();
    MUON_LAUNCH(MUON_LAUNCH_EXPERT_COMBINE_GRAD, launch_expert_combine_grad(a, dtype, b.vec && width * es % 16 == 0, s));
    return launched();
  });
}

muon_status_t linear_forward(const linear_args_t* p, void* stream) {
  return guarded([&]() -> muon_status_t {
    MUON_CHECK(check_sizes(p));
    MUON_CHECK(check_activation(p->activation));
    if (p->rows == 0) return no_launch();
    const size_t es = dtype_size(p->dtype);
    Buffers b;
    if (p->offsets) MUON_CHECK(b.list(p->offsets, "offsets", p->groups + 1, 4, false));
    MUON_CHECK(b.add(p->x, "x", p->rows, p->in, p->x_stride, es, false));
    MUON_CHECK(b.add(p->w, "w", p->out, p->in, p->w_stride, es, false, p->groups, p->w_group_stride));
    if (p->bias) MUON_CHECK(b.add(p->bias, "bias", p->groups, p->out, p->out, es, false));
    static const char kResidual[] = "residual", kY[] = "y";
    if (p->residual) MUON_CHECK(b.add(p->residual, kResidual, p->rows, p->out, p->residual_stride, es, false));
    MUON_CHECK(b.add(p->y, kY, p->rows, p->out, p->y_stride, es, true));
    if (p->pre) MUON_CHECK(b.add(p->pre, "pre", p->rows, p->out, p->pre_stride, es, true));
    MUON_CHECK(b.disjoint(kY, kResidual));
    LinArgs a{};
    a.p = p->x;
    a.ldp = p->x_stride;
    a.q = p->w;
    a.ldq = p->w_stride;
    a.gq = p->w_group_stride;
    a.c = p->y;
    a.ldc = p->y_stride;
    a.pre = p->pre;
    a.ldpre = p->pre_stride;
    a.bias = p->bias;
    a.aux = p->residual;
    a.ldaux = p->residual_stride;
    a.offsets = p->offsets;
    a.rows = static_cast<int32_t>(p->rows);
    a.n = static_cast<int32_t>(p->out);
    a.k = static_cast<int32_t>(p->in);
    a.groups = static_cast<int32_t>(p->groups);
    a.act = p->activation;
    a.parts = 1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int align = b.align(p->in, p->out, es);
    if (!linear_fits(a, LIN_FORWARD, p->dtype, align)) return fail(MUON_ERR_UNSUPPORTED, "the product is too large");
    MUON_HOOK_START();
    MUON_LAUNCH(MUON_LAUNCH_LINEAR, launch_linear(a, LIN_FORWARD, p->dtype, align, s));
    return launched();
  });
}

muon_status_t linear_grad_workspace_bytes(const linear_grad_args_t* args, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    GradLayout l;
    MUON_CHECK(grad_layout(args, l));
    *bytes = l.bytes;
    return MUON_OK;
  });
}

muon_status_t linear_grad(const linear_grad_args_t* p, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    GradLayout l;
    MUON_CHECK(grad_layout(p, l));
    // (dx of no rows is an empty buffer, whose address may be NULL.)
    if (!p->dx && !p->dw && !p->db && p->rows == 0) return no_launch();
    if (!p->dx && !p->dw && !p->db) return fail(MUON_ERR_INVALID_ARG, "none of dx, dw and db is given");
    const bool has_act = p->activation != LINEAR_NONE;
    const size_t es = dtype_size(p->dtype), gs = dtype_size(p->grad_dtype);
    Buffers b;
    if (p->offsets) MUON_CHECK(b.list(p->offsets, "offsets", p->groups + 1, 4, false));
    if (p->rows) {
      MUON_CHECK(b.add(p->dy, "dy", p->rows, p->out, p->dy_stride, es, false));
      if (has_act) MUON_CHECK(b.add(p->pre, "pre", p->rows, p->out, p->pre_stride, es, false));
      if (p->dw) MUON_CHECK(b.add(p->x, "x", p->rows, p->in, p->x_stride, es, false));
      if (p->dx) {
        MUON_CHECK(b.add(p->w, "w", p->out, p->in, p->w_stride, es, false, p->groups, p->w_group_stride));
        MUON_CHECK(b.add(p->dx, "dx", p->rows, p->in, p->dx_stride, es, true));
        if (p->x_activation != LINEAR_NONE)
          MUON_CHECK(b.add(p->x_pre, "x_pre", p->rows, p->in, p->x_pre_stride, es, false));
      }
    }
    if (p->dw) MUON_CHECK(b.add(p->dw, "dw", p->out, p->in, p->dw_stride, gs, true, p->groups, p->dw_group_stride));
    if (p->db) MUON_CHECK(b.list(p->db, "db", p->groups * p->out, gs, true));
    MUON_CHECK(b.workspace(workspace, workspace_bytes, l.bytes));
    MUON_CHECK(b.disjoint());
    const int align = b.align(p->in, p->out, es);
    char* ws = static_cast<char*>(workspace);
    const void* dz = has_act ? ws + l.dz : p->dy;
    const int64_t dz_ld = has_act ? l.dz_ld : p->dy_stride;
    hipStream_t s = static_cast<hipStream_t>(stream);
    LinArgs in{}, wt{};
    in.offsets = wt.offsets = p->offsets;
    in.rows = wt.rows = static_cast<int32_t>(p->rows);
    in.groups = wt.groups = static_cast<int32_t>(p->groups);
    in.n = wt.n = static_cast<int32_t>(p->in);
    in.p = wt.p = dz;
    in.ldp = wt.ldp = dz_ld;
    in.k = static_cast<int32_t>(p->out);
    in.q = p->w;
    in.ldq = p->w_stride;
    in.gq = p->w_group_stride;
    in.c = p->dx;
    in.ldc = p->dx_stride;
    in.act = p->x_activation;
    in.aux = p->x_activation != LINEAR_NONE ? p->x_pre : nullptr;
    in.ldaux = p->x_pre_stride;
    in.parts = 1;
    wt.m = static_cast<int32_t>(p->out);
    wt.q = p->x;
    wt.ldq = p->x_stride;
    wt.c = p->dw;
    wt.ldc = p->dw_stride;
    wt.gc = p->dw_group_stride;
    wt.c_dt = p->grad_dtype;
    wt.accumulate = p->accumulate;
    wt.parts = l.parts;
    wt.part = reinterpret_cast<float*>(ws + l.part);
    if ((p->dx && !linear_fits(in, LIN_INPUT, p->dtype, align)) || (p->dw && !linear_fits(wt, LIN_WEIGHT, p->dtype, align)))
      return fail(MUON_ERR_UNSUPPORTED, "the product is too large");
    if ((p->db && !linear_bias_fits(p->out, p->groups)) ||
        (l.slope_sums && linear_slope_tiles(p->rows, p->out, p->groups) * ceil_div(p->out, 64) >= int64_t{1} << 30))
      return fail(MUON_ERR_UNSUPPORTED, "the bias is too large");
    LinArgs bias{};
    bias.offsets = p->offsets;
    bias.rows = in.rows;
    bias.groups = in.groups;
    bias.n = static_cast<int32_t>(p->out);
    bias.act = p->activation;
    bias.c = p->db;
    bias.c_dt = p->grad_dtype;
    bias.accumulate = p->accumulate;
    float* const sums = reinterpret_cast<float*>(ws + l.bias_part);
    MUON_HOOK_START();
    if (l.slope_sums && p->rows)
      MUON_LAUNCH(MUON_LAUNCH_LINEAR_SLOPE,
                  launch_linear_slope_sums(bias, p->dy, p->dy_stride, p->pre, p->pre_stride,
                                           p->dx || p->dw ? ws + l.dz : nullptr, dz_ld, sums, s));
    else if (has_act && p->rows)
      MUON_LAUNCH(MUON_LAUNCH_LINEAR_SLOPE,
                  launch_linear_slope(p->dy, p->dy_stride, p->pre, p->pre_stride, ws + l.dz, dz_ld, p->offsets,
                                      in.groups, p->rows, p->out, p->activation, p->dtype, align, s));
    if (p->dx && p->rows) MUON_LAUNCH(MUON_LAUNCH_LINEAR_INPUT, launch_linear(in, LIN_INPUT, p->dtype, align, s));
    if (p->dw) {
      MUON_HIP_TRY(launch_linear(wt, LIN_WEIGHT, p->dtype, align, s));
      if (l.parts > 1) MUON_HIP_TRY(launch_linear_join(wt, s));
      MUON_HIP_TRY(hook_record(MUON_LAUNCH_LINEAR_WEIGHT, s));
    }
    if (l.slope_sums)
      MUON_LAUNCH(MUON_LAUNCH_LINEAR_BIAS, launch_linear_sums(bias, sums, s));
    else if (p->db)
      MUON_LAUNCH(MUON_LAUNCH_LINEAR_BIAS,
                  launch_linear_bias(dz, dz_ld, p->offsets, in.groups, p->rows, p->out, p->db, p->dtype, p->grad_dtype,
                                     p->accumulate, sums, l.bias_parts, s));
    return launched();
  });
}

}  // extern "C"
