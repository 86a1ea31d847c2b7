"""The drafts' tree of speculative_verify on the host: which drafts are there, and which rows lie behind which
(csrc/draft_tree.h, compiled by the host's compiler), over parents of any kind."""

import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_logits_filtering_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "draft_tree.h"
int main() {
  int D, V;
  while (std::scanf("%d %d", &D, &V) == 2) {
    std::vector<int32_t> token(D), above(D);
    for (int j = 0; j < D; ++j) {
      int t, p;
      if (std::scanf("%d %d", &t, &p) != 2) return 1;
      const tkp::DraftPlace d = tkp::draft_place(j, t, p, V);
      token[j] = d.token;
      above[j] = d.node;
      std::printf("%d %d\n", d.token, d.node);
    }
    for (int node = 0; node <= D; ++node)
      for (int r = 0; r <= D; ++r) std::putchar(tkp::row_behind(r, node, token.data(), above.data()) ? '1' : '0');
    std::putchar('\n');
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx is not None, "no host C++ compiler"
    folder = tmp_path_factory.mktemp("tree")
    (folder / "tree.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-D_GLIBCXX_ASSERTIONS", "-I", CSRC, "-o", str(folder / "tree"),
                    str(folder / "tree.cpp")], check=True, timeout=120)
    return str(folder / "tree")


def parents_of(kind, D, rng):
    j = np.arange(D)
    good = np.array([rng.integers(-1, i) if i else -1 for i in range(D)], np.int64)
    any_of = rng.random(D) < 0.4
    if kind == "self":
        return np.where(any_of, j, good)
    if kind == "later":
        return np.where(any_of, j + rng.integers(1, 300, D), good)
    if kind == "huge":
        return np.where(any_of, rng.choice([1000, 2 ** 31 - 1, 255, 256], D), good)
    if kind == "negative":
        return np.where(any_of, rng.choice([-2, -257, -2 ** 31], D), good)
    if kind == "constant":  # padding
        return np.full(D, rng.integers(0, D))
    if kind == "chain":
        return j - 1
    if kind == "cycle":  # pairs that follow each other
        return np.where(any_of, j ^ 1, good)
    return good


def test_places_and_rows_behind(program):
    rng = np.random.default_rng(0)
    cases = []
    for kind in ("good", "self", "later", "huge", "negative", "constant", "chain", "cycle"):
        for D in (1, 2, 7, 40, 255):
            for _ in range(4):
                V = 50
                token = rng.integers(0, V, D)
                token[rng.random(D) < 0.1] = rng.choice([-1, V, -2 ** 31, 2 ** 31 - 1])
                cases.append((D, V, token, parents_of(kind, D, rng)))
    text = "\n".join(f"{D} {V}\n" + "\n".join(f"{t} {p}" for t, p in zip(token, parent)) for D, V, token, parent in cases)
    res = subprocess.run([program], input=text, capture_output=True, text=True, timeout=60)  # ends, whatever the parents
    assert res.returncode == 0
    lines = iter(res.stdout.splitlines())
    dead_on_the_way = 0
    for D, V, token, parent in cases:
        there = [0 <= token[j] < V and -1 <= parent[j] < j for j in range(D)]
        for j in range(D):
            want = (token[j], parent[j] + 1) if there[j] else (-1, -1)
            assert tuple(map(int, next(lines).split())) == want
        # rows at and behind each one, from the front: a draft is behind what its parent is at or behind
        behind = np.zeros((D + 1, D + 1), bool)
        for r in range(D + 1):
            behind[r, r] = r == 0 or there[r - 1]
            if r and there[r - 1]:
                behind[:, r] |= behind[:, parent[r - 1] + 1]
                dead_on_the_way += bool(parent[r - 1] >= 0 and not there[parent[r - 1]])
        got = np.array(list(next(lines))).reshape(D + 1, D + 1) == "1"
        for node in range(D + 1):
            if node == 0 or there[node - 1]:  # where paths stand
                assert (got[node] == behind[node]).all()
    assert dead_on_the_way > 100
