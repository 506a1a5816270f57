"""The runs of rows that the norm's and the gate's workgroups take
(gemm_rwkv_amd/csrc/runs.h) cover every row once, up to the largest number of
tokens the interface admits.  They are constant expressions, in which the
compiler refuses any sum that leaves its type."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 65

PROGRAM = """
#include "runs.h"
constexpr bool covers(int tokens, int rows) {
  const int n = rq::run_count(tokens, rows);
  if (rows < 1 || n < 1) return false;
  long long next = 0;
  // the first runs, and the last ones
  for (int i = 0; i < n; i = i == 3 && n > 8 ? n - 4 : i + 1) {
    const unsigned begin = (unsigned)i * (unsigned)rows;   // as a workgroup's index times the rows
    if (begin >= (unsigned)tokens) return false;
    if (i < 4 || i > n - 4) if ((long long)begin != next) return false;
    next = rq::run_end(tokens, (int)begin, rows);
    if (next <= (long long)begin || next - begin > rows) return false;
  }
  return next == tokens;
}
constexpr int kTokens[] = {1, 2, 15, 16, 17, 768, 769, 1536, 1537, 4099, 1 << 20, (1 << 22) + 1, (1 << 30) + 7, 2143289345,
                           2147483000, %d};
constexpr int kGroups[] = {1, 2, 7, 511, 512};
constexpr bool all() {
  for (int t : kTokens) {
    if (!covers(t, rq::norm_rows(t)) || !covers(t, rq::gate_rows(t))) return false;
    for (int groups : kGroups) {
      const int rows = rq::run_rows(t, groups);
      if (!covers(t, rows) || rq::run_count(t, rows) > groups) return false;
    }
    if (rq::run_count(t, rq::norm_rows(t)) > 1 << 22 || rq::run_count(t, rq::gate_rows(t)) > 1 << 20) return false;
  }
  return true;
}
static_assert(all(), "every row once");
static_assert(rq::run_rows(0, 1) == 1 && rq::run_count(0, 1) == 0, "no rows");
"""


def test_runs_cover_every_row(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    src = tmp_path / "runs.cpp"
    src.write_text(PROGRAM % MOST)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", "-fconstexpr-ops-limit=100000000",
                        "-I" + os.path.join(ROOT, "gemm_rwkv_amd", "csrc"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
