"""Parts of the library that are plain C++, compiled and run on the host."""
import os
import shutil
import subprocess
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_quantized_dequant_gb300", "csrc")


def run(tmp_path, source: str) -> str:
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(textwrap.dedent(source))
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-Wall", "-Werror", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                          timeout=60).stdout


# Two threads raise one limit at the same time: A to 100 and, between A's set and A's
# note of it, B to 64.  Naive is a limit whose look, set and note are three steps.
GROW = """
    #include <chrono>
    #include <cstdio>
    #include <future>
    #include <thread>
    #include "grow_limit.h"
    struct Naive {
      std::atomic<int> now{0};
      template <class Set> int ensure(int want, Set &&set) {
        if (now >= want) return 0;
        const int e = set(want);
        if (e == 0) now = want;
        return e;
      }
    };
    template <class Limit> int after() {
      Limit l;
      std::atomic<int> real{0};  // what the device allows
      std::promise<void> a_set, b_done;
      auto b_has = b_done.get_future();
      std::thread b([&] {
        a_set.get_future().wait();
        l.ensure(64, [&](int v) { real = v; return 0; });
        b_done.set_value();
      });
      l.ensure(100, [&](int v) {
        real = v;
        a_set.set_value();
        b_has.wait_for(std::chrono::milliseconds(300));
        return 0;
      });
      b.join();
      l.ensure(80, [&](int v) { real = v; return 0; });
      return real;
    }
    int main() {
      qz::GrowLimit l;
      int sets = 0;
      auto ok = [&](int) { return ++sets, 0; };
      auto bad = [&](int) { return ++sets, 7; };
      const int r[] = {l.ensure(5, bad), l.ensure(5, ok), l.ensure(4, ok), l.ensure(6, bad),
                       l.ensure(5, ok), l.ensure(6, ok)};
      for (int v : r) std::printf("%d ", v);
      std::printf("%d\\n%d %d\\n", sets, after<Naive>(), after<qz::GrowLimit>());
    }
"""


def test_a_limit_only_grows(tmp_path):
    one, two = run(tmp_path, GROW).splitlines()
    assert one.split() == ["7", "0", "0", "7", "0", "0", "4"]
    assert two.split() == ["64", "100"]  # the naive one allows 64 and counts on 100
