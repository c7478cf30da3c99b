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


PLAN = """
    #include <cstdio>
    #include "lora_plan.h"
    int main() {
      const long Ts[] = {1, 2, 3, 7, 16, 31, 64, 127, 128, 200, 300, 1000, 1500, 4500, 100000},
                 Ks[] = {1, 64, 512, 513, 1000, 2048, 4096, 4104, 8192, 12000, 1 << 20},
                 Ns[] = {1, 64, 136, 256, 257, 4096, 11008, 1 << 20};
      const int all[] = {1, 132, 148, 152, 160};
      for (int sms : all)
        for (long T : Ts) for (long K : Ks) for (long N : Ns)
          for (long R = 1; R <= 128; R += R < 24 ? 1 : 8) {
            const qz::LoraPlan p = qz::lora_plan(T, K, N, R, sms);
            std::printf("%d %ld %ld %ld %ld %d %d %d %d %d %d %d\\n", sms, T, K, N, R, p.Rp, p.Rk,
                        p.slices, p.k_slice, p.rows_down, p.rows_up, p.along_n);
          }
    }
"""


def test_adapter_plans_keep_to_what_the_kernels_hold(tmp_path):
    import numpy as np
    v = np.loadtxt(run(tmp_path, PLAN).splitlines(), dtype=np.int64).T
    sms, T, K, N, R, Rp, Rk, slices, k_slice, down, up, along_n = v
    assert ((Rp - R < 16) & (Rp >= R) & (Rp % 16 == 0)).all()
    assert ((Rk - R < 32) & (Rk >= R) & (Rk % 32 == 0)).all()
    # slices: at most a portable cluster, whole steps, none empty, all of K
    assert ((slices >= 1) & (slices <= 8) & (k_slice % 512 == 0)).all()
    assert ((slices * k_slice >= K) & ((slices - 1) * k_slice < K)).all()
    for rows in (down, up):
        assert ((rows >= 1) & (rows <= 32) & (rows & (rows - 1) == 0)).all()
    # 8 warps' sums: two CTAs of the down product share an SM's 227 KB (1 KB of it each reserved)
    smem = 8 * down * Rp * 4
    assert (2 * (smem + 1024) <= 227 * 1024).all()
    assert (smem <= 96 * 1024).all()
    assert ((along_n >= 1) & (along_n <= -(-N // 256))).all()
    # the sizes that the tests and real calls reach
    assert set(np.unique(down)) == set(np.unique(up)) == {1, 2, 4, 8, 16, 32}


def test_adapter_cases_reach_every_variant(tmp_path):
    """The tests' calls of many rows take the wide forms of both products: more than 8
    rows a CTA, u in registers whole (R <= 32) or in halves, aligned rows or not."""
    import layer_cases as C
    calls = "".join(f"P({sms}, {T}, {K}, {N}, {R});" for sms in (148, 152)
                    for T, _, _, R, K, N, _, _ in C.ADAPTERS)
    out = run(tmp_path, """
        #include <cstdio>
        #include "lora_plan.h"
        static void P(int sms, long T, long K, long N, long R) {
          const qz::LoraPlan p = qz::lora_plan(T, K, N, R, sms);
          std::printf("%%d %%d %%d\\n", p.rows_down, p.rows_up, p.slices);
        }
        int main() { %s }
    """ % calls)
    v = [tuple(map(int, line.split())) for line in out.splitlines()]
    n = len(C.ADAPTERS)
    for plans in (v[:n], v[n:]):
        got = [(down > 8, up, slices == 8, R <= 32, K % 8 == 0 and not off,
                N % 8 == 0 and R % 8 == 0 and not off)
               for (down, up, slices), (_, _, _, R, K, N, _, off) in zip(plans, C.ADAPTERS)]
        assert {16, 32} <= {up for _, up, *_ in got}
        assert {(up > 8, small, vb) for _, up, _, small, _, vb in got} >= {
            (True, True, True), (True, True, False), (True, False, True), (True, False, False)}
        assert {(down, va) for down, _, full, _, va, _ in got if full} >= {
            (True, True), (True, False)}
