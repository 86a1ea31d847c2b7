"""exp in 64 bits behind drawn tokens (csrc/exp64.h, compiled by the host's compiler): the polynomial and the table over
all bf16 values, against exp in 80 bits.

Bound: the polynomial is within 1.9e-14 of 2^r; its ten steps, the argument (log2(e) to 2^-57 of itself, times at most 760)
and the scaling add less than 3e-16 + 760 * 1.5 * 2^-57 < 1e-14 for far values, and below 1e-15 for those above -80."""

import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_logits_filtering_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "exp64.h"
int main() {
  using namespace tkp;
  static double table[kTable];
  for (int m = kTableLow; m <= kTableHigh; ++m) table_pair(m, table[m - kTableLow], table[kTableSign + m - kTableLow]);
  for (int b = 0; b < 0x10000; ++b) {  // every bf16 value, by the entry that it is looked up in
    int m = b & 0x7FFF;
    m = m < kTableLow ? kTableLow : (m > kTableHigh ? kTableHigh : m);
    std::printf("%a\n", table[(b & 0x8000 ? kTableSign : 0) + m - kTableLow]);
  }
  float x, ref;
  while (std::scanf("%a %a", &x, &ref) == 2) std::printf("%a\n", exp_from(x, ref));
}
"""


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx is not None, "no host C++ compiler"
    folder = tmp_path_factory.mktemp("exp")
    (folder / "exp.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(folder / "exp"), str(folder / "exp.cpp")], check=True,
                   timeout=120)
    rng = np.random.default_rng(0)
    x = np.float32(rng.uniform(-790, 80, 4000))
    ref = np.float32(rng.choice([0.0, 0.0, 80.0, -900.5], 4000))
    x[:6], ref[:6] = [0.0, -0.0, 3e-39, -70.0, -np.inf, -745.0], 0.0
    x[ref < 0] -= np.float32(900.5)
    text = "\n".join(f"{float(a).hex()} {float(b).hex()}" for a, b in zip(x, ref))
    res = subprocess.run([str(folder / "exp")], input=text, capture_output=True, text=True, timeout=60)
    assert res.returncode == 0
    got = np.array([float.fromhex(line) for line in res.stdout.splitlines()])
    return got[:0x10000], x, ref, got[0x10000:]


def test_table(results):
    table = results[0]
    with np.errstate(invalid="ignore"):  # NaN are among them
        x = (np.arange(0x10000, dtype=np.uint32) << 16).view(np.float32).astype(np.longdouble)
    near = np.isfinite(x) & (x > -128) & (x < 128)
    want = np.exp(x[near])
    assert (np.abs(table[near] - want) <= 2e-14 * want).all()
    assert table[0] == table[0x8000] == 1.0
    assert (table[(x <= -128) | (x == -np.inf)] == 0.0).all()


def test_polynomial(results):
    _, x, ref, got = results
    d = x.astype(np.longdouble) - ref
    want = np.exp(d)
    close, far = d > -80, (d <= -80) & (d > -700)
    assert (np.abs(got[close] - want[close]) <= 2e-14 * want[close]).all()
    assert (np.abs(got[far] - want[far]) <= 3e-14 * want[far]).all()
    assert (got[d < -746] == 0.0).all() and (got[d > -744] > 0.0).all()
