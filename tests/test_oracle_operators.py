"""CPU pins of the operators' oracle: the boundary's forward against its parts and
its backward against differences, the quantised rows against the definition,
the clip against closed forms."""

import numpy as np
import pytest

import oracle
from oracle import operators as op

NAMES = ("post_gamma", "post_beta", "scale", "pre_gamma", "pre_beta")


def case(T=7, d=16, G=4, seed=0, post=True, scale=True, pre=True, kind="linear"):
    rng = np.random.default_rng(seed)
    c = dict(x=rng.standard_normal((T, d)), o=rng.standard_normal((T, d)) + 0.2,
             u=rng.standard_normal((T, d)) if kind != "none" else None, gid=rng.integers(0, G, T).astype(np.int8))
    p = {n: (1.0 if n.endswith("gamma") else 0.0) + 0.3 * rng.standard_normal((G, d)) for n in NAMES}
    if not post:
        p["post_gamma"] = p["post_beta"] = None
    if not scale:
        p["scale"] = None
    if not pre:
        p["pre_gamma"] = p["pre_beta"] = None
    return c, p


def test_boundary_forward_is_made_of_its_parts():
    c, p = case()
    h, y = op.boundary_forward(**c, **p, kind="silu")
    n = oracle.group_layernorm(c["o"], c["gid"], p["post_gamma"], p["post_beta"], oracle.EPS)
    want = c["x"] + p["scale"][c["gid"]] * n * oracle.silu(c["u"])
    np.testing.assert_allclose(h, want, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(y, oracle.group_layernorm(want, c["gid"], p["pre_gamma"], p["pre_beta"], oracle.EPS),
                               rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "linear", "silu"])
@pytest.mark.parametrize("post,scale,pre", [(True, True, True), (False, True, True), (True, False, True),
                                            (True, True, False), (False, False, False)])
def test_boundary_backward_against_differences(kind, post, scale, pre):
    c, p = case(T=5, d=8, seed=3, post=post, scale=scale, pre=pre, kind=kind)
    rng = np.random.default_rng(9)
    dh = rng.standard_normal(c["x"].shape)
    dy = rng.standard_normal(c["x"].shape) if pre else None
    got = op.boundary_backward(**c, **p, dh=dh, dy=dy, kind=kind)

    def loss():
        h, y = op.boundary_forward(**c, **p, kind=kind)
        return float((h * dh).sum() + ((y * dy).sum() if pre else 0.0))

    step = 1e-6
    for name, arr, key in [("x", c["x"], "dx"), ("o", c["o"], "do"), ("u", c["u"], "du")] + [(n, p[n], n) for n in NAMES]:
        if arr is None:
            assert key not in got
            continue
        want = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + step
            up = loss()
            arr[i] = keep - step
            want[i] = (up - loss()) / (2 * step)
            arr[i] = keep
        # central differences: truncation ~ step^2, rounding ~ 1e-15 |loss| / step
        np.testing.assert_allclose(got[key], want, rtol=1e-6, atol=1e-7, err_msg=name)


def test_quantised_rows_by_hand():
    x = np.array([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0], [1e-38, -1e-38, 0, 0], [np.inf, 1, 2, 3],
                  [np.nan, 1, 2, 3], [3e38, -3e38, 1, 0]], np.float32)
    q, s = op.quantize_rows(x)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, -2]  # ties to even
    assert s[1] == np.float32(2.0 ** -100) * np.float32(1 / 127) and not q[1].any()
    assert not q[2].any() and s[2] == s[1]
    assert np.isnan(s[3]) and not q[3].any() and np.isnan(s[4]) and not q[4].any()
    assert q[5].tolist() == [127, -127, 0, 0]


def test_quantised_rows_are_the_nearest():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 64)) * 10.0 ** rng.integers(-20, 20, (50, 1))).astype(np.float32)
    q, s = op.quantize_rows(x)
    far = np.abs(q.astype(np.float64) * s.astype(np.float64)[:, None] - x)
    assert (far <= 0.5 * s.astype(np.float64)[:, None]).all() and np.abs(q.astype(int)).max(1).min() == 127


def test_gemm_i8_closed_form():
    a = np.array([[1, -2], [127, -128]], np.int8)
    b = np.array([[3, 4], [-128, 127], [0, 1]], np.int8)
    v = op.gemm_i8(a, [0.5, 2.0], b, [1.0, 0.25, 4.0], bias=[1.0, 0.0, 0.0], q_cols=0)
    np.testing.assert_array_equal(v, [[-2.5 + 1, -382 * 0.125, -4.0], [2 * -131 + 1.0, 0.5 * -32512, -1024.0]])


def test_clip_closed_form():
    grads = [np.full((3,), 4.0), np.full((2, 2), -2.0)]
    norm, out = op.grad_clip(grads, 4.0, 0.5)
    assert norm == 4.0  # 0.5 sqrt(48 + 16)
    c = 0.5 * 4.0 / (4.0 + 1e-6)
    np.testing.assert_allclose(out[0], 4.0 * c)
    norm, out = op.grad_clip(grads, 100.0, 0.5)
    np.testing.assert_array_equal(out[1], grads[1] * 0.5)
    assert op.grad_clip([np.array([np.inf])], 1.0)[1] is None
