"""The operators' calls beside the ordinary ones, each against the float64 oracle or
against the same call made plainly. Tolerances: tests/test_gpu_operators.py."""

import numpy as np
import pytest
import torch

import generative_recommendation_ranking_b200 as mt
from oracle import operators as op
from test_gpu_operators import case, host, mags, near, oracle_args, upstream

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- boundary --
@pytest.mark.parametrize("d", [8, 64, 104, 128, 256])
@pytest.mark.parametrize("T", [5, 10, 21, 1003])
@pytest.mark.parametrize("gate", ["none", "linear", "silu"])
def test_boundary_backward_without_eps(T, d, gate):
    # narrow rows share a warp: a team with fewer rows than its neighbour adds nothing
    # behind them, whatever eps is
    dev, r = case(T, d, torch.float32, gate=gate)
    dh, dy = upstream(T, d)
    out = mt.boundary_backward(**dev, dh=dh, dy=dy, gate=gate, eps=0.0)
    want = op.boundary_backward(**oracle_args(r), dh=host(dh), dy=host(dy), kind=gate, eps=0.0)
    # the magnitudes are taken at the framework's eps: 1e-5 of a variance near 1
    m = mags(r, gate, host(dh), host(dy))
    for k in want:
        near(out[k], want[k], 1.001 * m[k], k)


@pytest.mark.parametrize("d", [8, 64, 104, 128, 256])
def test_boundary_forward_without_eps(d):
    dev, r = case(21, d, torch.float32)
    h, y, _ = mt.boundary_forward(**dev, y_dtype=torch.float32, eps=0.0)
    want = op.boundary_forward(**oracle_args(r), eps=0.0)
    m = mags(r, "linear")
    near(h, want[0], 1.001 * m["h"], "h")
    near(y, want[1], 1.001 * m["y"], "y")
