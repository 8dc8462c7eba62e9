"""Per-device look-ups under concurrent first calls (CPU only): the host header
is compiled with ThreadSanitizer, and threads that meet at the first call of
each device must neither race nor fill a value twice.  Filling it from every
thread that arrives early, as plain data behind an atomic flag, is a race."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "lossless_draft_verify_vc_b200", "csrc")

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>
#include "vc_once.h"
struct Value { int active[4]; };
static vc::PerDevice<Value> values;
static std::atomic<int> fills{0};
struct Planted {  // the pattern that the header replaces
  std::atomic<bool> set{false};
  int active[4];
} planted[64];
int main(int argc, char** argv) {
  const bool plant = argc > 1 && !std::strcmp(argv[1], "plant");
  int bad = 0;
  for (int dev = 0; dev < 64; ++dev) {
    std::atomic<int> here{0};
    std::atomic<int> wrong{0};
    std::vector<std::thread> t;
    for (int i = 0; i < 4; ++i)
      t.emplace_back([&] {
        here.fetch_add(1);
        while (here.load() < 4) std::this_thread::yield();
        if (plant) {
          Planted& p = planted[dev];
          if (!p.set.load(std::memory_order_acquire)) {
            for (int j = 0; j < 4; ++j) p.active[j] = dev + j;
            p.set.store(true, std::memory_order_release);
          }
          return;
        }
        const Value& v = values.get(dev, [&](Value& x) {
          ++fills;
          for (int j = 0; j < 4; ++j) x.active[j] = dev + j;
        });
        for (int j = 0; j < 4; ++j) wrong += v.active[j] != dev + j;
      });
    for (auto& x : t) x.join();
    bad += wrong;
  }
  if (!plant && (bad || fills != 64)) { std::printf("bad %d fills %d\n", bad, fills.load()); return 3; }
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("once")
    (d / "p.cpp").write_text(PROGRAM)
    exe = str(d / "p")
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O1", "-g", "-pthread", "-I", CSRC, str(d / "p.cpp"), "-o", exe]
    r = subprocess.run(cmd + ["-fsanitize=thread"], capture_output=True, text=True)
    if r.returncode and "tsan" in r.stderr:
        pytest.skip("no ThreadSanitizer here")
    assert r.returncode == 0, r.stderr
    return exe


def run(exe, *args):
    env = {**os.environ, "TSAN_OPTIONS": "exitcode=66"}
    return subprocess.run([exe, *args], capture_output=True, text=True, env=env, timeout=120)


def test_concurrent_first_calls_fill_once_without_a_race(program):
    r = run(program)
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("ThreadSanitizer does not run here")
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_sanitizer_sees_the_planted_race(program):
    r = run(program, "plant")
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("ThreadSanitizer does not run here")
    assert r.returncode == 66 and "data race" in r.stderr
