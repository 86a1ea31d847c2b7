"""How speculative_verify cuts its work (csrc/verify_plan.h, compiled by the host's compiler): grids that a launch takes,
and cuts that cover every row, over the sizes that the entry point allows."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_logits_filtering_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "verify_plan.h"
using namespace tkp::verify;
// In: dtype N D V draft tree greedy. Out: sequences of a launch, most threads of a grid, whether chunks and parts cover
// the row, parts, threads of the last kernel.
int main() {
  long long dtype, N, D, V, draft, tree, greedy;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &dtype, &N, &D, &V, &draft, &tree, &greedy) == 7) {
    const Plan p = plan_of(dtype, N, D, V, draft, tree);
    const int64_t n = sequences_of_launch(p, N, D, draft, greedy), held = n < N ? n : N;
    int64_t most = held * rows_groups(p, D, draft) * kT;
    auto also = [&](int64_t threads) { most = most > threads ? most : threads; };
    also(held * final_groups(p, greedy) * final_threads(p, greedy));
    if (p.steps > 0) {
      also(held * p.split.chunks * kT);
      also(held * behind_groups(N, D, p.split) * int64_t{kT});
    }
    const int64_t nv = V / (dtype == 0 ? 4 : 8);
    const int parts = p.cut.groups * (p.cut.threads / kWaveLanes);
    const bool covers = int64_t{p.split.chunks} * p.split.vecs >= nv && int64_t{parts} * p.cut.pieces * kPiece >= V;
    std::printf("%lld %lld %d %d %d\n", (long long)n, (long long)most, covers ? 1 : 0, parts, final_threads(p, greedy));
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx is not None, "no host C++ compiler"
    folder = tmp_path_factory.mktemp("plan")
    (folder / "plan.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, "-o", str(folder / "plan"), str(folder / "plan.cpp")],
                   check=True, timeout=120)

    def run(cases):
        text = "\n".join(" ".join(str(int(v)) for v in c) for c in cases)
        res = subprocess.run([str(folder / "plan")], input=text, capture_output=True, text=True, timeout=60)
        assert res.returncode == 0
        return [tuple(map(int, line.split())) for line in res.stdout.splitlines()]

    return run


def test_grids_hold_below_two_to_the_32_threads(plan):
    cases = []
    for dtype in (0, 1, 2):
        for D in (0, 1, 2, 3, 7, 39, 254, 255):
            for V in (0, 1, 4, 511, 513, 1000, 65536, 151936, 1 << 20):
                for N in (1, 2, 17, 64, 511, 513, 5000, 2 ** 20, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 2 ** 31 - 1):
                    N = min(N, (2 ** 31 - 1) // (2 * D + 1))
                    for draft, tree, greedy in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
                        cases.append((dtype, N, D, V, draft if D else 0, tree, greedy))
    many = 0
    for case, (n, most, covers, parts, threads) in zip(cases, plan(cases)):
        assert n >= 1 and most < 2 ** 32 and covers and parts <= 256, case
        many += threads == 1024 and case[2] == 0 and case[1] >= 2 ** 22
    assert many > 0  # draws from rows without drafts, by workgroups of 1024
