"""Launch plans against what their kernels have room for, on the host: small
programs over the planning headers and the library's objects (no GPU)."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dequant_matmul_nf4_amd", "csrc")


def run(tmp_path, text, link=()):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is not available")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text("#include <cstdio>\n#include <initializer_list>\n#include <utility>\n" + text)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{CSRC}", str(src), *link, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]
    return r.stdout


# Every index that the walk forms into its partial sums: part p < wpr, its rows i < kmax, segment s, row c of x.
WALK = r"""
#include "gemv_plan.h"
using namespace nf4i;
int main() {
  long bad = 0, plans = 0;
  for (int mc = 1; mc <= 2; ++mc)
    for (int waves = 8; waves <= 16; waves += 8)
      for (int nseg = 1; nseg <= 16; ++nseg)
        for (int64_t cus : {16, 32, 64, 128, 256, 304})
          for (int64_t rows = 1; rows <= 300000; rows += rows < 300 || rows % 4096 == 4095 || rows % 4096 == 0 ? 1 : 4095 - rows % 4096 < 391 ? 4095 - rows % 4096 : 391) {
            const int64_t cols = int64_t(nseg) * 4096 - 64 * (rows % 7);
            const RowsPlan pl = rows_plan(rows, cols, waves, mc, cus);
            if (pl.nseg > kSegMax || pl.wpr < 1) continue;
            ++plans;
            const int64_t np = int64_t(pl.grid) * pl.wpr, kmax = (rows + np - 1) / np;
            const int64_t last = (((pl.wpr - 1) * kmax + kmax - 1) * kSegMax + pl.nseg - 1) * mc + mc - 1;
            const bool in = last < int64_t(rows_room(mc)) * kSegMax * mc;
            if (!in || !rows_plan_fits(pl, rows, cols, mc)) {
              if (bad++ < 5) printf("rows %ld cols %ld waves %d mc %d cus %ld: %ld rows, index %ld\n", long(rows), long(cols), waves, mc, long(cus), long(pl.wpr * kmax), long(last));
            }
          }
  // a plan for one row of x does not pass for two, and too wide a row for none
  const RowsPlan one = rows_plan(128256, 4096, 8, 1, 256);
  if (!rows_plan_fits(one, 128256, 4096, 1) || rows_plan_fits(one, 128256, 4096, 2)) ++bad;
  if (rows_plan_fits(rows_plan(100, 65600, 16, 1, 256), 100, 65600, 1)) ++bad;
  printf("%ld plans, %ld bad\n", plans, bad);
  return bad || plans < 100000;
}
"""


def test_walk_over_rows_has_room_for_its_sums(tmp_path):
    run(tmp_path, WALK)


def test_two_rows_of_x_over_a_tall_weight(tmp_path):
    """The sizes whose plan for one row of x overran the sums of two: a vocabulary's projection and beyond."""
    out = run(tmp_path, r"""
#include "gemv_plan.h"
using namespace nf4i;
int main() {
  int bad = 0;
  for (auto [rows, cols] : {std::pair<int64_t, int64_t>{65536, 128}, {65537, 128}, {65537, 4096}, {70000, 128}, {128256, 4096}, {151936, 8192}, {300000, 32768}}) {
    const RowsPlan pl = rows_plan(rows, cols, 8, 2, 256);
    const int64_t np = int64_t(pl.grid) * pl.wpr, here = pl.wpr * ((rows + np - 1) / np);
    printf("%ld x %ld: %ld rows of %d\n", long(rows), long(cols), long(here), rows_room(2));
    bad += here > rows_room(2);
  }
  return bad;
}
""")
    assert "128256 x 4096" in out


# Sizes of every kernel of the product, and both sides of the rules between them.
SIZES = r"""
#include <cstdint>
#include <cstddef>
namespace nf4i {
int cus = 256;
int device_cus() { return cus; }
size_t linear_workspace(int64_t m, int64_t rows, int64_t cols, int r);
size_t act_backward_workspace(int64_t m, int64_t rows);
size_t expert_balance_workspace(int64_t tokens, int experts);
size_t grad_workspace(int count);
}
using namespace nf4i;
int main() {
  long bad = 0, cases = 0;
  const auto same = [&](const char* what, long a, long b, long c, auto call) {
    cus = 256;
    const size_t want = call();
    for (int n : {16, 32, 64, 80, 128, 255, 304}) {
      cus = n;
      ++cases;
      const size_t got = call();
      if (got != want && bad++ < 5) printf("%s %ld %ld %ld: %zu bytes with 256 units, %zu with %d\n", what, a, b, c, want, got, n);
    }
  };
  for (int64_t m : {1, 2, 3, 16, 17, 32, 33, 64, 100, 128, 192, 300, 512, 513, 700, 1024, 2048, 4096, 4097, 70000})
    for (int64_t rows : {1, 16, 300, 512, 1024, 4096, 14336, 28672, 128256})
      for (int64_t cols : {64, 192, 256, 1024, 4096, 8192, 14336})
        for (int r : {0, 16})
          same("linear", m, rows, cols, [&] { return linear_workspace(m, rows, cols, r); });
  for (int64_t m : {1, 7, 333, 4096, 1 << 20})
    for (int64_t n : {1, 100, 11007, 14336}) {
      same("act_backward", m, n, 0, [&] { return act_backward_workspace(m, n); });
      same("balance", m, 1 + n % 1024, 0, [&] { return expert_balance_workspace(m, int(1 + n % 1024)); });
      same("grads", n, 0, 0, [&] { return grad_workspace(int(n)); });
    }
  printf("%ld cases, %ld bad\n", cases, bad);
  return bad != 0;
}
"""


def test_workspaces_do_not_depend_on_the_device(tmp_path):
    """A workspace is sized before the call that uses it, perhaps on another thread or for another device:
    its size must not follow the compute units of whichever device was current."""
    from dequant_matmul_nf4_amd import build
    objects = [os.path.join(build.BUILD, f + ".o") for f in build.sources() if f != "api.cpp"]
    if not all(os.path.exists(o) for o in objects):
        build.build()
    rocm = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc()))), "lib")
    run(tmp_path, SIZES, [*objects, f"-L{rocm}", f"-Wl,-rpath,{rocm}", "-lamdhip64", "-pthread"])
