// Host-side pieces shared by the C ABI's translation units: the error message,
// the launch-event hook, the overlap check and the descriptor upload.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <stdexcept>
#include <string>
#include <vector>

#include "common.h"
#include "muon_mi355x.h"

namespace muon {

inline thread_local std::string g_last_error;

// Launch-event hook (timing only).
struct EventHook {
  void* const* events = nullptr;
  int32_t* kinds = nullptr;
  int32_t n = 0;
  int32_t next = 0;
  int32_t last_count = 0;
};
inline thread_local EventHook g_hook;

inline hipError_t hook_record(int32_t kind, hipStream_t s) {
  if (!g_hook.events || g_hook.next >= g_hook.n) return hipSuccess;
  hipError_t e = hipEventRecord(static_cast<hipEvent_t>(g_hook.events[g_hook.next]), s);
  if (g_hook.kinds) g_hook.kinds[g_hook.next] = kind;
  ++g_hook.next;
  return e;
}

inline muon_status_t fail(muon_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

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

constexpr size_t kAlign = 256;

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline size_t dtype_size(int32_t dt) { return dt == DT_F32 ? 4 : 2; }

inline bool finite(float x) { return std::isfinite(x); }

struct Range { uintptr_t lo, hi; int64_t mat; const char* what; bool writable; };

// Any overlap between two ranges of which one is written is an error.
inline muon_status_t check_overlaps(std::vector<Range>& rs, const char* noun) {
  std::sort(rs.begin(), rs.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  // Any overlap that involves a written buffer is an error.  Scanning in
  // address order, keep the written range reaching furthest and the range
  // (of any kind) reaching furthest.
  const Range* far_any = nullptr;
  const Range* far_wr = nullptr;
  for (const Range& r : rs) {
    const Range* hit = nullptr;
    if (r.writable && far_any && far_any->hi > r.lo) hit = far_any;
    else if (far_wr && far_wr->hi > r.lo) hit = far_wr;
    if (hit)
      return fail(MUON_ERR_ALIAS, "%s %lld %s overlaps %s %lld %s", noun, (long long)r.mat, r.what, noun,
                  (long long)hit->mat, hit->what);
    if (!far_any || r.hi > far_any->hi) far_any = &r;
    if (r.writable && (!far_wr || r.hi > far_wr->hi)) far_wr = &r;
  }
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Descriptor upload: the table is copied from a pinned host buffer into the
// workspace prefix on the step's stream.  An event records when the copy has
// consumed the host buffer, so the buffer is never overwritten early.
// ---------------------------------------------------------------------------
struct Staging {
  void* host = nullptr;
  size_t cap = 0;
  hipEvent_t ev = nullptr;
  int device = -1;   // of the event, which can be recorded on that device's streams only
  bool pending = false;

  // True when the buffer may be written: no copy from it is in flight.
  bool idle() {
    if (!pending) return true;
    if (hipEventQuery(ev) == hipSuccess) pending = false;
    return !pending;
  }

  muon_status_t upload(const std::vector<unsigned char>& table, void* dst, hipStream_t s) {
    hipError_t err;
    if (pending) {
      if ((err = hipEventSynchronize(ev)) != hipSuccess)
        return fail(MUON_ERR_HIP, "hipEventSynchronize: %s", hipGetErrorString(err));
      pending = false;
    }
    if (cap < table.size()) {
      if (host) (void)hipHostFree(host);
      host = nullptr;
      cap = 0;
      if ((err = hipHostMalloc(&host, table.size(), hipHostMallocDefault)) != hipSuccess) {
        host = nullptr;
        return fail(MUON_ERR_HIP, "hipHostMalloc(%zu): %s", table.size(), hipGetErrorString(err));
      }
      cap = table.size();
    }
    int current = -1;
    if ((err = hipGetDevice(&current)) != hipSuccess)
      return fail(MUON_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(err));
    if (ev && device != current) {   // a thread that steps on several devices
      (void)hipEventDestroy(ev);
      ev = nullptr;
    }
    if (!ev && (err = hipEventCreateWithFlags(&ev, hipEventDisableTiming)) != hipSuccess) {
      ev = nullptr;
      return fail(MUON_ERR_HIP, "hipEventCreate: %s", hipGetErrorString(err));
    }
    device = current;
    std::memcpy(host, table.data(), table.size());
    if ((err = hipMemcpyAsync(dst, host, table.size(), hipMemcpyHostToDevice, s)) != hipSuccess)
      return fail(MUON_ERR_HIP, "hipMemcpyAsync: %s", hipGetErrorString(err));
    if ((err = hipEventRecord(ev, s)) != hipSuccess)
      return fail(MUON_ERR_HIP, "hipEventRecord: %s", hipGetErrorString(err));
    pending = true;
    return MUON_OK;
  }

  void release() {
    if (pending && ev) (void)hipEventSynchronize(ev);
    if (ev) (void)hipEventDestroy(ev);
    if (host) (void)hipHostFree(host);
    host = nullptr;
    ev = nullptr;
    cap = 0;
    pending = false;
  }
};

// Staging buffers of the stateless calls, per host thread.  A call takes an
// idle buffer (its previous copy has completed), or a new one while the
// thread holds fewer than kPoolMax; only a thread with kPoolMax copies in
// flight waits, for its oldest.  The buffers are freed when the thread exits.
constexpr size_t kPoolMax = 64;
struct StagingPool {
  std::vector<Staging*> slots;
  size_t oldest = 0;   // slot waited on when every slot is busy

  Staging* take() {
    for (Staging* st : slots)
      if (st->idle()) return st;
    if (slots.size() < kPoolMax) {
      slots.push_back(new Staging());
      return slots.back();
    }
    Staging* st = slots[oldest];
    oldest = (oldest + 1) % slots.size();
    return st;   // upload() waits for its copy
  }

  ~StagingPool() {
    for (Staging* st : slots) {
      st->release();
      delete st;
    }
  }
};
inline thread_local StagingPool g_pool;

#define MUON_HIP_TRY(expr)                                                                 \
  do {                                                                                     \
    hipError_t e_ = (expr);                                                                \
    if (e_ != hipSuccess) return fail(MUON_ERR_HIP, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

// Launch, then record the hook's event for this launch kind.
#define MUON_LAUNCH(kind, expr)              \
  do {                                       \
    MUON_HIP_TRY(expr);                      \
    MUON_HIP_TRY(hook_record((kind), s));    \
  } while (0)

}  // namespace muon
