"""A device query that fails is asked again by the next call; one that has succeeded is not."""
import os
import shutil
import subprocess

import pytest

import top_sparse_attention_chunked_gb300 as pkg

PROGRAM = r"""
#include "kept_answers.h"
#include <cstdio>
#include <thread>
#include <vector>
int main() {
  dsa::KeptAnswers<4> kept;
  int asked = 0;
  const auto fails = [&](int* n) { ++asked; *n = 7; return false; };
  const auto works = [&](int* n) { ++asked; *n = 5; return true; };
  const auto none = [&](int* n) { ++asked; *n = 0; return true; };
  const int a = kept.get(1, fails), b = kept.get(1, fails), c = kept.get(1, works), d = kept.get(1, fails);
  const int e = kept.get(2, none), f = kept.get(2, works);   // an answer of 0 is kept too
  std::printf("%d %d %d %d %d %d %d\n", a, b, c, d, e, f, asked);
  int together = 0;
  std::vector<std::thread> all;
  for (int i = 0; i < 16; ++i)
    all.emplace_back([&] { kept.get(3, [&](int* n) { ++together; *n = 1; return true; }); });
  for (auto& t : all) t.join();
  std::printf("%d\n", together);
}
"""


def test_failed_queries_are_not_kept(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    src = tmp_path / "kept.cpp"
    src.write_text(PROGRAM)
    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    subprocess.run([gxx, "-std=c++17", "-pthread", "-I", csrc, str(src), "-o", str(tmp_path / "kept")], check=True)
    out = subprocess.run([str(tmp_path / "kept")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == [0, 0, 5, 5, 0, 0, 4, 1]
