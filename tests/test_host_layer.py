"""The C-ABI layer on the host, without a GPU: the API's translation unit is compiled
with the CUDA runtime's calls and the kernel launchers replaced by recording
stand-ins, so that what a call asks of the device, and in which order, can be read.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_gqa_decode_gb300", "csrc")

# A device of 152 SMs.  A launch is recorded with the address of its status word, which
# is its workspace's first.
STAND_INS = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <map>
#include <string>
#include <thread>
#include <vector>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

struct Event { std::string what; const void* at; size_t bytes; cudaStream_t stream; };
static std::mutex ev_mu;
static std::condition_variable ev_cv;
static std::vector<Event> events;
static std::function<void(const char*)> before_launch;

static void record(const char* what, const void* at, size_t bytes, cudaStream_t st) {
  std::lock_guard<std::mutex> lk(ev_mu);
  events.push_back({what, at, bytes, st});
  ev_cv.notify_all();
}
static cudaError_t launched(const char* what, const void* ws, cudaStream_t st) {
  if (before_launch) before_launch(what);
  record(what, ws, 0, st);
  return cudaSuccess;
}

static cudaError_t stub_cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
static cudaError_t stub_cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152
       : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 227 * 1024 : 228 * 1024;
  return cudaSuccess;
}
static cudaError_t stub_cudaMallocAsync(void** p, size_t n, cudaStream_t st) {
  static uintptr_t next = 0x10000000;
  std::lock_guard<std::mutex> lk(ev_mu);
  *p = reinterpret_cast<void*>(next);
  next += (n + 0xffff) & ~size_t(0xffff);
  events.push_back({"malloc", *p, n, st});
  return cudaSuccess;
}
static cudaError_t stub_cudaFreeAsync(void* p, cudaStream_t st) { record("free", p, 0, st); return cudaSuccess; }
static cudaError_t stub_cudaFree(void* p) { record("free", p, 0, nullptr); return cudaSuccess; }
static cudaError_t stub_cudaDeviceSynchronize() { record("sync", nullptr, 0, nullptr); return cudaSuccess; }
static cudaError_t stub_cudaMemsetAsync(void* p, int, size_t n, cudaStream_t st) {
  record("zero", p, n, st);
  return cudaSuccess;
}
static cudaError_t stub_cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
static cudaError_t stub_cudaStreamGetId(cudaStream_t st, unsigned long long* id) {
  *id = 1000 + reinterpret_cast<uintptr_t>(st);
  return cudaSuccess;
}
static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
static cudaError_t stub_cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int,
                                             unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDevice stub_cudaGetDevice
#define cudaDeviceGetAttribute stub_cudaDeviceGetAttribute
#define cudaMallocAsync stub_cudaMallocAsync
#define cudaFreeAsync stub_cudaFreeAsync
#define cudaFree stub_cudaFree
#define cudaDeviceSynchronize stub_cudaDeviceSynchronize
#define cudaMemsetAsync stub_cudaMemsetAsync
#define cudaStreamIsCapturing stub_cudaStreamIsCapturing
#define cudaStreamGetId stub_cudaStreamGetId
#define cudaGetDriverEntryPointByVersion stub_cudaGetDriverEntryPointByVersion
#include "paged_attn_api.cu"

using namespace pagedattn;

namespace pagedattn {
#define DECODE(name)                                                                          \
  cudaError_t launch_##name(int, bool, const CUtensorMap&, const CUtensorMap&,                \
                            const DecodeParams& p, int, size_t, cudaStream_t st) {            \
    return launched(#name, p.status, st);                                                     \
  }
DECODE(decode_d64) DECODE(decode_d128) DECODE(decode_d256)
DECODE(decode_xp_d64) DECODE(decode_xp_d128) DECODE(decode_xp_d256)
DECODE(decode_multi_d64) DECODE(decode_multi_d128) DECODE(decode_multi_d256)
DECODE(decode_fp8_d128) DECODE(decode_fp8_d256)
DECODE(decode_mod_d64) DECODE(decode_mod_d128) DECODE(decode_mod_d256)
DECODE(decode_fp8_mod_d128) DECODE(decode_fp8_mod_d256)
#define TILE(name)                                                                            \
  cudaError_t launch_##name(const CUtensorMap&, const CUtensorMap&, const TileParams& p,      \
                            cudaStream_t st) {                                                \
    return launched(#name, p.status, st);                                                     \
  }
TILE(tile_d64) TILE(tile_d128) TILE(tile_d256)
cudaError_t launch_merge(const MergeParams&, cudaStream_t st) {
  return launched("merge", nullptr, st);
}
cudaError_t launch_append(const AppendParams&, int, cudaStream_t st) {
  return launched("append", nullptr, st);
}
cudaError_t launch_append_fp8(const AppendParams&, int, cudaStream_t st) {
  return launched("append_fp8", nullptr, st);
}
cudaError_t launch_append_slots(const AppendSlotsParams&, int, cudaStream_t st) {
  return launched("append_slots", nullptr, st);
}
cudaError_t launch_assign(const AssignParams&, cudaStream_t st) {
  return launched("assign", nullptr, st);
}
}  // namespace pagedattn

static int bad = 0;
#define CHECK(c) do { if (!(c)) { std::printf("%s:%d: %s\n", __func__, __LINE__, #c); ++bad; } } while (0)

// Non-null, aligned addresses that no one follows.
template <class T> static T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }
static cudaStream_t stream_of(int i) { return reinterpret_cast<cudaStream_t>(uintptr_t(i) * 64); }
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    where = tmp_path_factory.mktemp("host")

    def go(name, program):
        src, exe = where / f"{name}.cu", where / name
        src.write_text(STAND_INS + program)
        r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17",
                            "--expt-relaxed-constexpr", "-I", CSRC, "-I",
                            os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and r.stdout.strip().endswith("OK"), (r.returncode, r.stdout)

    return go


def test_workspace_sizes_of_few_rows_and_no_groups(run):
    """The size of a shared-prefix call without groups (the decode of the own tokens) is at
    least that of the decode itself; no size query divides by the number of pieces."""
    run("sizes", r"""
int main() {
  for (int D : {64, 128, 256})
    for (int G : {1, 4, 16})
      for (int n : {0, 1, 4, 31, 128, 1000})
        for (int groups : {0, 1, 3}) {
          const size_t shared = paged_attn_shared_workspace_bytes(n, groups, 2 * G, 2, D, 8, 16);
          const size_t mods = paged_attn_mods_workspace_bytes(n, 2 * G, 2, D, 8, 16);
          CHECK(mods > 0 && shared >= paged_attn_workspace_bytes(n, 2 * G, 2, D, 8, 16));
          CHECK(shared > 0);
          CHECK(paged_attn_multi_mods_workspace_bytes(n, n, 2 * G, 2, D, 8, 16) > 0);
          if (n == 0) continue;
          // the call itself takes a workspace of that size
          events.clear();
          CHECK(paged_attn_decode_shared(at<void>(16), at<void>(16), at<void>(16), at<void>(16),
                                         at<int32_t>(16), at<int32_t>(16), at<int32_t>(16), groups, 4,
                                         at<int32_t>(16), at<int32_t>(16), n, 2 * G, 2, D, 8, 16,
                                         0.1f, 0.f, nullptr, at<void>(256), shared,
                                         nullptr) == PAGED_ATTN_OK);
          CHECK(events.size() == (groups ? 3u : 1u) ||
                (n > 512 && events.size() > (groups ? 3u : 1u)));
        }
  std::printf(bad ? "FAIL\n" : "OK\n");
  return bad != 0;
}
""")


# Calls through each entry point that may use a library-owned workspace; `big`: sizes that
# need a larger one than any call before.  check_live: a launch names a buffer that is
# allocated at that place in the order of its stream.
CALLS = r"""
static int call(int kind, bool big, cudaStream_t st) {
  void* p = at<void>(256);
  const int32_t* i = at<int32_t>(256);
  float* f = at<float>(256);
  const int n = big ? 400 : 2, H = big ? 32 : 2, D = big ? 256 : 128;
  switch (kind) {
    case 0: return paged_attn_decode(p, p, p, p, i, i, n, H, 2, D, 8, 16, 0.1f, st);
    case 1: return paged_attn_append_decode(p, p, p, p, p, p, i, i, n, H, 2, D, 8, 16, 0.1f, st);
    case 2: return paged_attn_append_decode_fp8(p, p, p, p, p, f, f, p, i, i, n, H, 2, D, 8, 16, 0.1f, st);
    case 3: return paged_attn_decode_multi(p, p, p, p, i, i, i, n, 2 * n, 2, H, 2, D, 8, 16, 0.1f, st);
    case 4: return paged_attn_decode_mods(p, p, p, p, i, i, n, H, 2, D, 8, 16, 0.1f, 0.f, nullptr,
                                          0, nullptr, nullptr, nullptr, 0, st);
    case 5: return paged_attn_decode_multi_mods(p, p, p, p, i, i, i, big ? 9 : 1, big ? 60 : 3, H, 2, D,
                                                8, 16, 0.1f, 1, 0.f, nullptr, 0, nullptr, nullptr,
                                                nullptr, 0, st);
    default: return paged_attn_decode_shared(p, p, p, p, i, i, i, 1, 8, i, i, n, H, 2, D, 8, 16, 0.1f,
                                             0.f, nullptr, nullptr, 0, st);
  }
}
constexpr int kKinds = 7;

static void check_live() {
  std::map<const void*, bool> live;
  for (const Event& e : events) {
    if (e.what == "malloc") live[e.at] = true;
    else if (e.what == "free") live[e.at] = false;
    else if (e.at != nullptr && e.what != "zero")
      CHECK(live[e.at]);
  }
}
"""


def test_two_host_threads_on_one_stream(run):
    """While one thread is between taking the library's workspace and launching, another
    thread's larger call must not release that buffer ahead of the launch."""
    run("threads", CALLS + r"""
int main() {
  for (int kind = 0; kind < kKinds; ++kind) {
    std::atomic<bool> entered{false};
    std::atomic<int> launches{0};
    const size_t from = events.size();
    before_launch = [&](const char*) {
      if (launches++ > 0) return;
      entered = true;
      std::unique_lock<std::mutex> lk(ev_mu);  // as long as a release takes to come, if it may
      ev_cv.wait_for(lk, std::chrono::milliseconds(300), [&] {
        for (size_t k = from; k < events.size(); ++k)
          if (events[k].what == "free") return true;
        return false;
      });
    };
    std::thread a([&] { CHECK(call(kind, false, nullptr) == PAGED_ATTN_OK); });
    while (!entered) std::this_thread::yield();
    std::thread b([&] { CHECK(call(kind, true, nullptr) == PAGED_ATTN_OK); });
    a.join();
    b.join();
    check_live();
    before_launch = nullptr;
    // (the next kind begins with its small buffer again)
    for (auto& w : g_ws) w = OwnedWorkspace();
    for (auto& w : g_opt_ws) w = StreamWorkspaces();
  }
  std::printf(bad ? "FAIL\n" : "OK\n");
  return bad != 0;
}
""")


def test_streams_have_their_own_workspaces(run):
    """The score-option and shared-prefix calls without a workspace of the caller's: one
    per stream, kept while its stream needs it, released in its stream's order; past the
    number the library keeps, only after the device has finished."""
    run("streams", CALLS + r"""
int main() {
  std::map<cudaStream_t, const void*> of;
  for (int kind = 4; kind < kKinds; ++kind) {
    for (int round = 0; round < 2; ++round)
      for (int i = 0; i < 5; ++i) {
        const size_t from = events.size();
        CHECK(call(kind, round == 1 && i == 3, stream_of(i)) == PAGED_ATTN_OK);
        const void* ws = nullptr;
        for (size_t k = from; k < events.size(); ++k) {
          const Event& e = events[k];
          CHECK(e.stream == stream_of(i));
          if (e.what == "free") CHECK(of[stream_of(i)] == e.at);
          if (ws == nullptr && e.what != "malloc" && e.what != "zero" && e.what != "free") ws = e.at;
        }
        CHECK(ws != nullptr);
        for (auto& [st, w] : of) CHECK((st == stream_of(i)) || w != ws);
        of[stream_of(i)] = ws;
      }
  }
  check_live();
  // as many streams as come: what is taken over is idle
  for (int i = 5; i < 200; ++i) {
    const size_t from = events.size();
    CHECK(call(4, false, stream_of(i)) == PAGED_ATTN_OK);
    bool synced = false;
    for (size_t k = from; k < events.size(); ++k) {
      if (events[k].what == "sync") synced = true;
      if (events[k].what == "free") CHECK(synced);
    }
    CHECK(synced == (i >= kStreamWorkspaces));
    const size_t again = events.size();
    CHECK(call(4, false, stream_of(i)) == PAGED_ATTN_OK);
    CHECK(events.size() == again + 1);  // the launch alone
  }
  check_live();
  // a reset reaches every buffer that is kept
  const size_t from = events.size();
  CHECK(paged_attn_reset_workspace(stream_of(1)) == PAGED_ATTN_OK);
  CHECK(events.size() - from == (size_t)kStreamWorkspaces);
  std::printf(bad ? "FAIL\n" : "OK\n");
  return bad != 0;
}
""")
