"""Set-up that each device needs once, from several host threads: no data race (the
compiler's race detector), a failure is tried again, a device past the table is set up
every time.  And no entry point keeps such state in a plain static."""
import glob
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_long_context_mse_b200", "csrc")

PROGRAM = r"""
#include <atomic>
#include <cassert>
#include <thread>
#include <vector>
#include "device_once.h"
#ifdef PLAIN  // what must be found
template <int N> struct Once {
  bool done[N] = {};
  template <typename F> int run(int dev, F f) { if (done[dev]) return 0; int rc = f(); if (!rc) done[dev] = true; return rc; }
};
#else
template <int N> using Once = losa::DeviceOnce<N>;
#endif
static Once<4> once;
int main() {
  static std::atomic<int> calls[8] = {}, here{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 4; ++i)
    t.emplace_back([] {
      // all at once (relaxed: nothing here orders the threads' accesses)
      here.fetch_add(1, std::memory_order_relaxed);
      while (here.load(std::memory_order_relaxed) < 4) std::this_thread::yield();
      for (int k = 0; k < 200; ++k) assert(once.run(k % 3, [&] { calls[k % 3].fetch_add(1, std::memory_order_relaxed); return 0; }) == 0);
    });
  for (auto& x : t) x.join();
  for (int d = 0; d < 3; ++d) assert(calls[d] >= 1 && calls[d] <= 4);
#ifndef PLAIN
  assert(once.run(3, [] { return 7; }) == 7);  // a failure is not kept
  assert(once.run(3, [] { return 0; }) == 0);
  assert(once.run(3, [] { return 7; }) == 0);
  for (int d : {-1, 4, 1000}) {
    assert(once.run(d, [] { return 0; }) == 0);
    assert(once.run(d, [] { return 5; }) == 5);
  }
#endif
}
"""


def run(tmp_path, *flags):
    src, exe = tmp_path / "once.cpp", str(tmp_path / "once")
    src.write_text(PROGRAM)
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-g", *flags, "-I", CSRC, str(src), "-o", exe,
                            "-lpthread"], capture_output=True, text=True)
    if build.returncode and "tsan" in build.stderr:
        pytest.skip("no race detector in this compiler")
    assert build.returncode == 0, build.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("the race detector does not run on this kernel")
    return r


def test_device_once_has_no_race(tmp_path):
    r = run(tmp_path, "-fsanitize=thread")
    assert r.returncode == 0, r.stderr


def test_a_plain_flag_is_a_race(tmp_path):
    r = run(tmp_path, "-fsanitize=thread", "-DPLAIN")
    assert "data race" in r.stderr


def test_no_unguarded_flags_in_the_library():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path).read()
        assert not re.search(r"static\s+(bool|int)\s+\w+\s*(\[[^\]]*\])?\s*(=|;)", text), path
        # flags at file scope: only beside a mutex
        if re.search(r"^bool\s+g_\w+", text, re.M):
            assert "std::mutex" in text and "lock_guard" in text, path
