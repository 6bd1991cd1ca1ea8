"""The library's memory per stream (csrc/fa_workspace.h), compiled on its own
against a fake of the CUDA calls (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include "fa_workspace.h"

static std::map<long, unsigned long long> ids;  // handle -> the stream it names now
static std::set<void*> live;
static int allocs, frees, fail_allocs, fail_frees;

struct Fake {
  using Stream = long;
  static bool id(long s, unsigned long long* out) {
    if (!ids.count(s)) return false;
    *out = ids[s];
    return true;
  }
  static bool shared(long s) { return s == 2; }
  static bool alloc(void** p, size_t n) {
    if (fail_allocs) return false;
    ++allocs;
    *p = std::malloc(n);
    live.insert(*p);
    return true;
  }
  static bool free(void* p) {
    ++frees;
    if (!live.erase(p)) { std::puts("freed twice"); std::exit(1); }
    std::free(p);
    return !fail_frees;
  }
};

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  fa::StreamWorkspaces<Fake> w;
  ids = {{0, 10}, {1, 10}, {2, 20}, {100, 30}, {200, 40}};
  // one block a stream, the same one again, whatever smaller size is asked for
  void* a = w.get(100, 1000)->ptr;
  CHECK(w.get(100, 400)->ptr == a && w.get(100, 1000)->ptr == a);
  void* b = w.get(200, 1000)->ptr;
  CHECK(a != b && allocs == 2 && frees == 0);
  // two handles of one stream
  CHECK(w.get(0, 64)->ptr == w.get(1, 64)->ptr);
  CHECK(allocs == 3);
  // one handle of a stream in each thread: each has its own, and keeps it
  void* t1 = w.get(2, 64)->ptr;
  ids[2] = 21;
  void* t2 = w.get(2, 64)->ptr;
  CHECK(t1 != t2 && frees == 0);
  ids[2] = 20;
  CHECK(w.get(2, 64)->ptr == t1);
  ids[2] = 21;
  CHECK(w.get(2, 64)->ptr == t2 && allocs == 5 && frees == 0);
  // a new stream with a destroyed one's handle: the old memory is freed first
  ids[100] = 31;
  CHECK(live.count(a) == 1);
  CHECK(w.get(100, 500) != nullptr);
  CHECK(frees == 1 && allocs == 6 && live.size() == 5);
  CHECK(w.get(200, 1000)->ptr == b);
  // with its counters
  auto* e = w.get(200, 1000);
  Fake::alloc(&e->tail_ctr, 8);
  e->tail_ctr_n = 1;
  CHECK(w.get(200, 10)->tail_ctr_n == 1);
  ids[200] = 41;
  CHECK(w.get(200, 1000)->tail_ctr == nullptr);
  CHECK(frees == 3 && live.size() == 5);
  // growth frees the smaller block; without memory the entry is empty, not lost
  w.get(200, 2000);
  CHECK(frees == 4 && live.size() == 5);
  fail_allocs = 1;
  CHECK(w.get(200, 3000) == nullptr && w.get(0, 64) != nullptr);
  ids[300] = 50;
  CHECK(w.get(300, 64) == nullptr);
  fail_allocs = 0;
  CHECK(w.get(200, 10) != nullptr && w.get(300, 64) != nullptr);
  CHECK(w.get(999, 64) == nullptr);  // no such stream
  CHECK(live.size() == 6);
  // everything goes, and comes back
  CHECK(w.release() && live.empty());
  CHECK(w.get(100, 64) != nullptr && live.size() == 1);
  fail_frees = 1;
  CHECK(!w.release() && live.empty());
  std::puts("ok");
  return 0;
}
"""


def compile_and_run(tmp_path, program):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "w.cpp", tmp_path / "w"
    src.write_text(program)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-pthread", "-I",
                    os.path.join(ROOT, "attention_forward_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_one_block_a_stream_known_by_its_id(tmp_path):
    compile_and_run(tmp_path, PROGRAM)


DEVICES = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <future>
#include "fa_workspace.h"

static std::atomic<int> frees{0};
struct Fake {
  using Stream = long;
  static bool id(long s, unsigned long long* out) { *out = 1000 + s; return true; }
  static bool shared(long) { return false; }
  static bool alloc(void** p, size_t n) { *p = std::malloc(n); return *p != nullptr; }
  static bool free(void* p) { ++frees; std::free(p); return true; }
};

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::_Exit(1); } } while (0)

int main() {
  using namespace std::chrono_literals;
  static fa::DeviceWorkspaces<Fake, 2> w;
  auto call = [](int dev) {
    return std::async(std::launch::async, [dev] {
      std::unique_lock<std::mutex> hold;
      CHECK(w.acquire(dev, 7, 100, &hold) != nullptr && hold.owns_lock());
    });
  };
  std::future<void> second;
  {
    // a call in progress on device 0: device 1 does not wait, device 0 does
    std::unique_lock<std::mutex> hold;
    CHECK(w.acquire(0, 7, 100, &hold) != nullptr && hold.owns_lock());
    CHECK(call(1).wait_for(20s) == std::future_status::ready);
    second = call(0);
    CHECK(second.wait_for(200ms) == std::future_status::timeout);
  }
  CHECK(second.wait_for(20s) == std::future_status::ready);
  // a device's memory alone is freed
  {
    auto lock = w.lock(0);
    CHECK(call(1).wait_for(20s) == std::future_status::ready);
    CHECK(w.release(0) && frees == 1);
  }
  w.forget(1);
  CHECK(call(1).wait_for(20s) == std::future_status::ready && frees == 1);
  std::puts("ok");
  return 0;
}
"""


def test_a_call_on_one_device_keeps_none_on_another_waiting(tmp_path):
    compile_and_run(tmp_path, DEVICES)
