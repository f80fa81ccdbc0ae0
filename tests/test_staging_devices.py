"""The descriptor upload of host.h against a stand-in for the HIP runtime that
knows several devices (host code only, built with g++): an event may be
recorded only on streams of the device it was created on."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#define __host__
#define __device__
struct float4 { float x, y, z, w; };
enum hipError_t { hipSuccess = 0, hipErrorInvalidHandle = 400, hipErrorNotReady = 600 };
struct Stream { int device; };
struct Event { int device; bool recorded; };
typedef Stream* hipStream_t;
typedef Event* hipEvent_t;
inline int g_device = 0, g_events = 0, g_hosts = 0;
inline bool g_busy = false;
constexpr unsigned hipEventDisableTiming = 2, hipHostMallocDefault = 0;
enum hipMemcpyKind { hipMemcpyHostToDevice };
inline const char* hipGetErrorString(hipError_t e) { return e == hipErrorInvalidHandle ? "invalid handle" : "error"; }
inline hipError_t hipGetDevice(int* d) { *d = g_device; return hipSuccess; }
inline hipError_t hipHostMalloc(void** p, size_t n, unsigned) { *p = std::malloc(n); ++g_hosts; return hipSuccess; }
inline hipError_t hipHostFree(void* p) { std::free(p); --g_hosts; return hipSuccess; }
inline hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) { *e = new Event{g_device, false}; ++g_events; return hipSuccess; }
inline hipError_t hipEventDestroy(hipEvent_t e) { delete e; --g_events; return hipSuccess; }
inline hipError_t hipEventRecord(hipEvent_t e, hipStream_t s) {
  if (e->device != s->device) return hipErrorInvalidHandle;
  e->recorded = true;
  return hipSuccess;
}
inline hipError_t hipEventQuery(hipEvent_t) { return g_busy ? hipErrorNotReady : hipSuccess; }
inline hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
inline hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, hipMemcpyKind, hipStream_t) { std::memcpy(d, s, n); return hipSuccess; }
"""

PROGRAM = r"""
#include "host.h"
using namespace muon;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (%s)\n", __LINE__, #x, g_last_error.c_str()); return 1; } } while (0)
int main() {
  Stream streams[2] = {{0}, {1}};
  for (bool busy : {false, true}) {
    g_busy = busy;
    for (int round = 0; round < 200; ++round) {
      const int dev = round & 1;
      g_device = dev;
      std::vector<unsigned char> table(100 + round, static_cast<unsigned char>(round)), out(table.size());
      CHECK(g_pool.take()->upload(table, out.data(), &streams[dev]) == MUON_OK);
      CHECK(out == table);
      CHECK(g_pool.slots.size() <= kPoolMax);
    }
  }
  CHECK(g_events == static_cast<int>(g_pool.slots.size()) && g_hosts == g_events);
  Staging own;
  std::vector<unsigned char> table(64, 7), out(64);
  for (int dev : {0, 1, 1, 0}) {
    g_device = dev;
    CHECK(own.upload(table, out.data(), &streams[dev]) == MUON_OK);
  }
  own.release();
  CHECK(g_events == static_cast<int>(g_pool.slots.size()) && g_hosts == g_events);
  return 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no g++")
def test_one_thread_uploads_to_several_devices(tmp_path):
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = tmp_path / "main"
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", f"-I{tmp_path}", f"-I{ROOT}/include",
                    f"-I{ROOT}/dimuon_newton_schulz_amd/csrc", str(tmp_path / "main.cpp"), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert done.returncode == 0, done.stdout
