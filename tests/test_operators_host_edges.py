"""Host arithmetic and refusals of the operators at their limits, on the CPU."""

import os
import shutil
import subprocess
import types

import pytest
import torch

import generative_recommendation_ranking_b200 as mt
from generative_recommendation_ranking_b200 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "generative_recommendation_ranking_b200", "csrc")

RUNS = r"""
#include <stdio.h>
#include <initializer_list>
#include "row_runs.h"
int main() {
  const int32_t T[] = {1, 3, 4, 5, 1917, 20011, 200003, 1 << 30, 2147481600, 2147483646, 2147483647};
  const int64_t resident[] = {1, 148, 1184, 7104, 14208};
  for (int32_t t : T)
    for (int64_t r : resident)
      for (int32_t d : {8, 64, 512, 8192})
        for (int32_t G : {1, 4, 32}) {
          const int32_t n = mtgr::bwd_teams(t, d, G, r);
          printf("%d %lld %d %d %d %d\n", t, (long long)r, d, G, n, mtgr::rows_per_team(t, n));
        }
}
"""


def test_rows_are_dealt_out_up_to_the_largest_count(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "runs.cc").write_text(RUNS)
    subprocess.run([cxx, "-std=c++17", "-fwrapv", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "runs.cc"), "-o",
                    str(tmp_path / "runs")], check=True)
    out = subprocess.run([str(tmp_path / "runs")], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        T, resident, d, G, teams, rows = map(int, line.split())
        # every row has one team, and every team a row; slots of at most 256 MB, unless one team
        assert teams >= 1 and rows >= 1 and teams * rows >= T > (teams - 1) * rows, line
        assert teams <= resident and (teams == 1 or teams * G * 5 * d * 4 <= 256 << 20), line


def test_a_given_workspace_is_checked():
    # a host tensor's device is -1: one that is asked for on the GPU is refused before its
    # address is used, and so is one with gaps, between which others' bytes lie
    whole = torch.zeros(1024, dtype=torch.uint8)
    assert ops._given_ws(None, 100, 0) == 0
    for dev, ws in ((0, whole), (-1, whole[::2]), (-1, whole.view(32, 32)[:, :16]), (-1, whole.view(32, 32).t())):
        with pytest.raises(ValueError, match="ws"):
            ops._given_ws(ws, 100, dev)
    assert ops._given_ws(whole, 1024, -1) == 1024 and ops._given_ws(whole, 1025, -1) == 0
    assert ops._given_ws(whole[512:], 100, -1) == 512 and ops._given_ws(torch.zeros(8, 8), 100, -1) == 256
    assert ops._given_ws(whole[:0], 0, -1) == 0


def test_wrappers_without_a_workspace():
    # NULL is a workspace of no bytes: what needs none goes through, what needs one is refused
    x = torch.zeros(0, 64)
    w, ws = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    try:
        mt.mtgr_linear_i8(x, w, ws, None, 0, None, 0, torch.zeros(0, 8), None, None,
                          types.SimpleNamespace(cuda_stream=None))  # no rows: nothing is launched
    except mt.MTGRError as e:
        assert e.status == mt._lib.MTGR_ERR_UNSUPPORTED  # no GPU here


def test_an_output_that_is_an_operand_is_refused():
    # other blocks still read what a block would write; addresses are never read here
    lib, (a, b, c, d) = mt.load(), (0x100000, 0x200000, 0x300000, 0x400000)
    invalid, f32 = mt._lib.MTGR_ERR_INVALID_ARG, mt.MTGR_F32
    for out in (a, b):
        assert lib.mtgr_gemm_i8(40, 64, 64, a, c, b, c, None, 0, None, 0, f32, out, None, None) == invalid
        for M in (9, 40):
            assert lib.mtgr_linear_i8(M, 64, 64, f32, a, 64, b, c, None, 0, None, 0, f32, out, d, 1 << 20, None, None) == invalid
    assert lib.mtgr_quantize_rows(40, 64, f32, a, 64, a, c, None) == invalid
