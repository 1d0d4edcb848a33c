"""GPU parity of the block-boundary, int8 and gradient-clipping operators with the
float64 oracle.

Tolerances count roundings: a rounding is off by at most half a step, 2^-24 of the
value in fp32, 2^-8 in bf16, 2^-11 in f16. An fp32 result that is made of a chain of
at most K roundings is off by at most K 2^-24 times the same formula over
absolute values (its magnitude). The longest chains: a row's sum (8 VPL additions
in a thread, VPL <= 4, five or ten across lanes and warps), twice for a norm, and
the elementwise steps; __expf adds 2 + 1.2 |u| roundings, |u| < 8. K = 128 covers them.
"""

import numpy as np
import pytest
import torch

import generative_recommendation_ranking_b200 as mt
from oracle import operators as op
from oracle import EPS

pytestmark = pytest.mark.gpu

K32 = 128 * 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half an f16 subnormal's step
NAMES = ("post_gamma", "post_beta", "scale", "pre_gamma", "pre_beta")
GATES = ["none", "linear", "silu"]


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, mag, what):
    """got (a tensor of its type) against want, within K32 mag and one rounding to the type."""
    g = host(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    tol = K32 * mag + HALF[got.dtype] * (np.abs(want) + K32 * mag) + LEAST[got.dtype]
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(g - want) / np.maximum(tol, 1e-300), 0))), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; at {i} got {g[i]!r}, want {want[i]!r}, tol {tol[i]:.3e}")


def case(T, d, branch=torch.bfloat16, stream=torch.float32, gate="linear", post=True, scale=True, pre=True, G=4, seed=0,
         wide=True, gid=None):
    """Device tensors and the same values in float64."""
    rng = np.random.default_rng(seed + 1000 * T + d)
    t = lambda a, dt: torch.from_numpy(np.asarray(a, np.float32)).to(dt).cuda()  # noqa: E731
    gid = np.sort(rng.integers(0, G, T)) if gid is None else gid
    dev = dict(x=t(rng.standard_normal((T, d)) * 3, stream), o=t(rng.standard_normal((T, d)) + 0.1, branch), u=None,
               group_id=torch.from_numpy(np.asarray(gid).astype(np.int8)).cuda())
    if gate != "none":
        buf = t(rng.standard_normal((T, 4 * d if wide else d)) * 0.7, branch)
        dev["u"] = buf[:, -d:]
    for n in NAMES:
        on = {"post": post, "scal": scale, "pre_": pre}[n[:4]]
        dev[n] = t((1.0 if n.endswith("gamma") else 0.0) + 0.3 * rng.standard_normal((G, d)), torch.float32) if on else None
    ref = {k: host(v) for k, v in dev.items() if k != "group_id"}
    ref["gid"] = np.clip(np.asarray(gid), 0, G - 1)
    return dev, ref


def f(r, g):
    return op.gate(r["u"], g)


def mags(r, gate, dh=None, dy=None):
    """Magnitudes of the forward's and the backward's values: the formulas over absolute values."""
    A = lambda v: np.abs(v)  # noqa: E731
    row = lambda v: v.mean(1, keepdims=True)  # noqa: E731
    gid, m = r["gid"], {}

    def norm(v, mag):  # normalised rows and what an error of `mag` in v does to them
        c = v - v.mean(1, keepdims=True)
        rstd = 1 / np.sqrt((c * c).mean(1, keepdims=True) + EPS)
        hat = c * rstd
        spread = rstd * (mag + row(mag))
        return hat, rstd, A(hat) + spread + A(hat) * row(A(hat) * spread) + A(hat) * row(hat * hat)

    n = mag_n = None
    if r["post_gamma"] is not None:
        oh, rstd_o, mag_oh = norm(r["o"], A(r["o"]))
        n = oh * r["post_gamma"][gid] + r["post_beta"][gid]
        mag_n = mag_oh * A(r["post_gamma"][gid]) + A(r["post_beta"][gid])
    else:
        n, mag_n = r["o"], A(r["o"])
    fu, dfu = f(r, gate)
    s = 1.0 if r["scale"] is None else r["scale"][gid]
    mag_f = A(fu) + (A(r["u"]) if gate == "silu" else 0.0)
    m["h"] = A(r["x"]) + A(s) * mag_n * mag_f
    if r["pre_gamma"] is not None:
        h = r["x"] + s * n * fu
        hh, rstd_h, mag_hh = norm(h, m["h"])
        m["y"] = mag_hh * A(r["pre_gamma"][gid]) + A(r["pre_beta"][gid])
    if dh is None and dy is None:
        return m
    G = next((r[k].shape[0] for k in ("post_gamma", "pre_gamma", "scale") if r[k] is not None), 1)
    by = lambda v: np.stack([v[gid == g].sum(0) for g in range(G)])  # noqa: E731

    def back(mag, mag_hat, rstd):
        # the terms of the norm's backward and the relative error of its rstd
        return rstd * (mag + row(mag) + mag_hat * row(mag * mag_hat)) * 2

    H = 0.0 if dh is None else A(dh)
    if dy is not None:
        a = A(dy) * A(r["pre_gamma"][gid])
        H = H + back(a, mag_hh, rstd_h)
        m["pre_gamma"], m["pre_beta"] = by(A(dy) * mag_hh), by(A(dy))
    m["dx"] = H
    m["scale"] = by(H * mag_n * mag_f)
    dn = H * A(s) * mag_f
    m["du"] = H * A(s) * mag_n * (1.0 + A(dfu) + A(fu))
    m["do"] = dn
    if r["post_gamma"] is not None:
        m["post_gamma"], m["post_beta"] = by(dn * mag_oh), by(dn)
        m["do"] = back(dn * A(r["post_gamma"][gid]), mag_oh, rstd_o)
    return m


def oracle_args(r):
    return {k: r[k] for k in ("x", "o", "u", "gid") + NAMES}


# ------------------------------------------------------- boundary, forward --
SHAPES = [(1, 8), (3, 64), (70, 40), (37, 72), (50, 128), (5, 200), (33, 256), (9, 264), (17, 512), (4, 1000), (6, 1024), (3, 1032), (2, 2048), (2, 5000),
          (2, 8192)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("gate", GATES)
def test_boundary_forward_shapes(T, d, gate):
    dev, r = case(T, d, gate=gate)
    h, y, ys = mt.boundary_forward(**dev, gate=gate, y_dtype=torch.float32)
    want = op.boundary_forward(**oracle_args(r), kind=gate)
    m = mags(r, gate)
    assert ys is None
    near(h, want[0], m["h"], "h")
    near(y, want[1], m["y"], "y")


@pytest.mark.parametrize("branch", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("stream", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16, torch.int8])
def test_boundary_forward_types(branch, stream, y_dtype):
    dev, r = case(70, 512, branch, stream, "silu")
    h, y, ys = mt.boundary_forward(**dev, gate="silu", y_dtype=y_dtype)
    want = op.boundary_forward(**oracle_args(r), kind="silu")
    m = mags(r, "silu")
    assert h.dtype == stream and y.dtype == y_dtype
    near(h, want[0], m["h"], "h")
    if y_dtype != torch.int8:
        near(y, want[1], m["y"], "y")
        return
    # the scale is the row's largest value over 127: one more rounding; a byte is off by
    # half a step, and by the error of y itself
    near(ys, np.abs(want[1]).max(1) / 127, m["y"].max(1) / 127, "y_scale")
    s = host(ys)[:, None]
    assert (np.abs(host(y) * s - want[1]) <= s * (0.5 + 2.0 ** -16) + K32 * m["y"]).all()
    assert (host(y.abs().amax(1)) == 127).all()


@pytest.mark.parametrize("post,scale,pre", [(False, True, True), (True, False, True), (True, True, False),
                                            (False, False, False), (False, False, True)])
@pytest.mark.parametrize("gate", GATES)
def test_boundary_parts_left_out(post, scale, pre, gate):
    dev, r = case(21, 264, torch.float16, gate=gate, post=post, scale=scale, pre=pre)
    h, y, ys = mt.boundary_forward(**dev, gate=gate, y_dtype=torch.float32)
    want = op.boundary_forward(**oracle_args(r), kind=gate)
    m = mags(r, gate)
    near(h, want[0], m["h"], "h")
    assert (y is None) == (not pre) and ys is None
    if pre:
        near(y, want[1], m["y"], "y")


def test_boundary_groups_out_of_range_count_as_the_nearest():
    gid = np.array([-128, -1, 0, 3, 4, 127])
    dev, r = case(6, 64, gid=gid)
    h, y, _ = mt.boundary_forward(**dev, y_dtype=torch.float32)
    near(h, op.boundary_forward(**oracle_args(r))[0], mags(r, "linear")["h"], "h")


def test_boundary_in_place_and_rows_left_alone():
    dev, r = case(40, 512)
    n = 33  # the rows behind the last sequence stay as they were
    part = {k: (v[:n] if v is not None and v.shape[0] == 40 else v) for k, v in dev.items()}
    keep = dev["x"].clone()
    y = torch.full((40, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    h, y2, _ = mt.boundary_forward(**part, h=part["x"], y=y[:n])
    assert h.data_ptr() == dev["x"].data_ptr() and y2.data_ptr() == y.data_ptr()
    want = op.boundary_forward(**{k: (v[:n] if k in ("x", "o", "u", "gid") else v) for k, v in oracle_args(r).items()})
    near(dev["x"][:n], want[0], mags(r, "linear")["h"][:n], "h")
    assert torch.equal(dev["x"][n:], keep[n:]) and (y[n:] == 7.0).all()


@pytest.mark.parametrize("T,d", [(1, 8), (5, 64), (3, 104), (7, 256), (5, 512), (3, 1000), (2, 2048)])
def test_boundary_writes_its_rows_alone(T, d):
    dev, _ = case(T, d)
    h = torch.full((T + 40, d), 7.0, device="cuda")
    y = torch.full((T + 40, d), 77, dtype=torch.int8, device="cuda")
    ys = torch.full((T + 40,), 9.0, device="cuda")
    mt.boundary_forward(**dev, h=h[16:16 + T], y=y[16:16 + T], y_scale=ys[16:16 + T], y_dtype=torch.int8)
    for t, v in ((h, 7), (y, 77), (ys, 9)):
        assert (t[:16] == v).all() and (t[16 + T:] == v).all()
    # gradients into wide rows: what lies past d stays
    L = mt._lib
    do, du = (torch.full((T + 8, d + 24), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dx = torch.full((T + 8, d), 3.0, device="cuda")
    dh, dy = upstream(T, d)
    want = mt.boundary_backward(**dev, dh=dh, dy=dy)
    par = {n: torch.empty(4, d, device="cuda") for n in NAMES}
    p = L.MtgrBoundaryParams(d, 4, EPS, L.MTGR_GATE_LINEAR, *[dev[n].data_ptr() for n in NAMES])
    gr = L.MtgrBoundaryGrads(*[par[n].data_ptr() for n in NAMES])
    ws = torch.empty(max(256, L.mtgr_boundary_bwd_workspace_bytes(T, p)), dtype=torch.uint8, device="cuda")
    L.mtgr_boundary_bwd(p, T, dev["group_id"], dev["o"], dev["u"], dev["x"], dh, dy, do[4:4 + T], du[4:4 + T], dx[4:4 + T], gr, ws)
    assert torch.equal(do[4:4 + T, :d], want["do"]) and torch.equal(du[4:4 + T, :d], want["du"]) and torch.equal(dx[4:4 + T], want["dx"])
    assert all(torch.equal(par[n], want[n]) for n in NAMES)
    for t in (do, du, dx):
        assert (t[:4] == 3).all() and (t[4 + T:] == 3).all()
    assert (do[:, d:] == 3).all() and (du[:, d:] == 3).all()


def test_boundary_no_rows():
    dev, _ = case(0, 64)
    h, y, ys = mt.boundary_forward(**dev, y_dtype=torch.int8)
    assert h.shape == (0, 64) and y.shape == (0, 64) and ys.shape == (0,)
    out = mt.boundary_backward(**dev, dh=h, dy=h)
    assert all((out[n] == 0).all() and out[n].shape == (4, 64) for n in NAMES)


def test_boundary_nan_row_stays_in_its_row():
    dev, r = case(9, 512, branch=torch.float32)
    dev["o"][4, 100] = float("nan")
    dev["o"][6, 0] = float("inf")
    h, y, ys = mt.boundary_forward(**dev, y_dtype=torch.int8)
    ok = [i for i in range(9) if i not in (4, 6)]
    for i in (4, 6):
        assert torch.isnan(ys[i]) and (y[i] == 0).all() and torch.isnan(h[i]).any()
    want = op.boundary_forward(**oracle_args(r))
    near(h[ok], want[0][ok], mags(r, "linear")["h"][ok], "h")


def test_boundary_large_mean_keeps_its_variance():
    # the variance is taken from centred values: a mean of a thousand sigma costs its
    # own rounding (2^-24 of 1000 sigma) and no more
    dev, r = case(8, 512, branch=torch.float32)
    dev["o"] += 1000.0
    r["o"] = host(dev["o"])
    h, y, _ = mt.boundary_forward(**dev, y_dtype=torch.float32)
    near(h, op.boundary_forward(**oracle_args(r))[0], mags(r, "linear")["h"], "h")


# ------------------------------------------------------ boundary, backward --
def check_backward(dev, r, gate, dh, dy, **kw):
    out = mt.boundary_backward(**dev, dh=dh, dy=dy, gate=gate, **kw)
    want = op.boundary_backward(**oracle_args(r), dh=host(dh), dy=host(dy), kind=gate)
    m = mags(r, gate, host(dh), host(dy))
    assert set(out) == set(want)
    for k in want:
        near(out[k], want[k], m[k], k)
    return out


def upstream(T, d, stream=torch.float32, y=torch.bfloat16, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, d, generator=g).to(stream).cuda(), torch.randn(T, d, generator=g).to(y).cuda()


@pytest.mark.parametrize("T,d", SHAPES + [(300, 64), (1003, 120), (1500, 256), (700, 512)])
@pytest.mark.parametrize("gate", GATES)
def test_boundary_backward_shapes(T, d, gate):
    dev, r = case(T, d, gate=gate)
    check_backward(dev, r, gate, *upstream(T, d))


@pytest.mark.parametrize("branch", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("stream", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("y", [torch.float32, torch.bfloat16])
def test_boundary_backward_types(branch, stream, y):
    dev, r = case(60, 512, branch, stream, "silu")
    out = check_backward(dev, r, "silu", *upstream(60, 512, stream, y))
    assert out["dx"].dtype == stream and out["do"].dtype == branch and out["du"].dtype == branch


@pytest.mark.parametrize("post,scale,pre", [(False, True, True), (True, False, True), (True, True, False),
                                            (False, False, False), (False, False, True)])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("d", [56, 200, 264])
def test_boundary_backward_parts_left_out(post, scale, pre, gate, d):
    dev, r = case(21, d, gate=gate, post=post, scale=scale, pre=pre)
    dh, dy = upstream(21, d)
    check_backward(dev, r, gate, dh, dy if pre else None)
    if pre:
        check_backward(dev, r, gate, None, dy)


@pytest.mark.parametrize("d", [64, 104, 264])
@pytest.mark.parametrize("G", [1, 4, 32])
def test_boundary_backward_groups_in_any_order(G, d):
    # the group changes at nearly every row: every change adds to the team's slots
    gid = np.random.default_rng(G).integers(0, G, 400)
    dev, r = case(400, d, G=G, gid=gid)
    check_backward(dev, r, "linear", *upstream(400, d))


def test_boundary_backward_same_bits_every_time():
    dev, _ = case(5000, 512)
    dh, dy = upstream(5000, 512)
    a = mt.boundary_backward(**dev, dh=dh, dy=dy)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # what a workspace held does not matter
    b = mt.boundary_backward(**dev, dh=dh, dy=dy, ws=ws)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("d", [8, 64, 104, 128, 256, 264, 512, 1024])
@pytest.mark.parametrize("T", [1, 21, 77, 20011])
def test_boundary_backward_keeps_to_its_workspace(d, T):
    # the workspace exactly as large as asked for, in the middle of a larger buffer;
    # teams that do not fill a block write nothing
    dev, r = case(T, d)
    dh, dy = upstream(T, d)
    p = mt._lib.MtgrBoundaryParams(d, 4, EPS, mt.MTGR_GATE_LINEAR, 16, 16, 16, 16, 16)
    need = mt.mtgr_boundary_bwd_workspace_bytes(T, p)
    pad = 1 << 20
    buf = torch.full((pad + need + pad,), 0xA5, dtype=torch.uint8, device="cuda")
    mt.boundary_backward(**dev, dh=dh, dy=dy, ws=buf[pad:pad + need])
    assert (buf[:pad] == 0xA5).all() and (buf[pad + need:] == 0xA5).all()


def test_boundary_backward_f16_range_is_reported():
    dev, _ = case(8, 512, torch.float16)
    dh, dy = upstream(8, 512)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mt.boundary_backward(**dev, dh=dh, dy=dy, status=status)
    assert status.item() == 0
    mt.boundary_backward(**dev, dh=dh * 1e6, dy=dy, status=status)
    assert status.item() == mt._lib.MTGR_ERR_RANGE


def test_boundary_backward_against_differences():
    dev, r = case(6, 64, torch.float32, gate="silu")
    dh, dy = upstream(6, 64, y=torch.float32)
    out = mt.boundary_backward(**dev, dh=dh, dy=dy, gate="silu")
    rng = np.random.default_rng(3)

    def loss(shift):
        a = oracle_args(r)
        a = {k: (v if k == "gid" else v + shift.get(k, 0.0)) for k, v in a.items()}
        h, y = op.boundary_forward(**a, kind="silu")
        return float((h * host(dh)).sum() + (y * host(dy)).sum())

    for k, key in [("x", "dx"), ("o", "do"), ("u", "du")] + [(n, n) for n in NAMES]:
        e = rng.standard_normal(r[k].shape)
        slope = (loss({k: 1e-5 * e}) - loss({k: -1e-5 * e})) / 2e-5
        terms = host(out[key]) * e
        # fp32 gradients: K32 of the terms' magnitudes, some tenfold in the norms; differences: 1e-9
        assert abs(terms.sum() - slope) <= 20 * K32 * np.abs(terms).sum() + 1e-6, key


# --------------------------------------------------------------- quantise --
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (130, 256), (7, 264), (5, 512), (4, 1000), (9, 1024), (3, 2048), (2, 2056),
                                 (5, 4096), (2, 8192), (2, 8200), (1, 32768)])
def test_quantize_rows_bit_for_bit(M, K, dtype):
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K)) * 10.0 ** rng.uniform(-3, 3, (M, 1))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    q, s = mt.quantize_rows(x)
    wq, ws = op.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantize_borders_and_special_rows():
    # multiples of half a step: ties, and their neighbours in fp32
    rows = []
    for top in (127.0, 1.0, 0.37, 3e38, 1e-25):
        s = np.float32(top) / np.float32(127)
        k = np.arange(-126, 127)
        v = ((k + 0.5) * np.float64(s)).astype(np.float32)
        row = np.concatenate([[top], v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf * np.sign(top)))])
        rows.append(np.resize(row, 768).astype(np.float32))
    rows += [np.zeros(768, np.float32), np.full(768, 1e-40, np.float32), np.full(768, 2.0 ** -101, np.float32)]
    bad = np.ones((3, 768), np.float32)
    bad[0, 5], bad[1, 767], bad[2, 0] = np.inf, np.nan, -np.inf
    x = np.concatenate([np.stack(rows), bad])
    q, s = mt.quantize_rows(torch.from_numpy(x).cuda())
    wq, ws = op.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.array_equal(q.cpu().numpy(), wq)
    assert np.isnan(ws[-3:]).all()


@pytest.mark.parametrize("M,K", [(3, 8), (5, 520), (7, 2056), (9, 4104)])
def test_quantize_writes_its_rows_alone(M, K):
    q = torch.full((M + 16, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M + 16,), 3.0, device="cuda")
    mt.quantize_rows(torch.randn(M, K, device="cuda"), q[8:8 + M], s[8:8 + M])
    assert (q[:8] == 99).all() and (q[8 + M:] == 99).all() and (s[:8] == 3).all() and (s[8 + M:] == 3).all()


def test_quantize_strided_rows():
    buf = torch.randn(50, 4 * 512, device="cuda").bfloat16()
    x = buf[:, 512:1024]
    q, s = mt.quantize_rows(x)
    wq, ws = op.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


# ----------------------------------------------------------- int8 product --
EPIS = {"none": mt.MTGR_EPI_NONE, "silu": mt.MTGR_EPI_SILU, "resid": mt.MTGR_EPI_RESID}


def product_case(M, N, K, seed=0, full=False):
    rng = np.random.default_rng(seed + M + N + K)
    lo = -128 if full else -127
    a, b = (rng.integers(lo, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sb = (rng.uniform(0.5, 2.0, n).astype(np.float32) * np.float32(1 / (73 * K ** 0.25)) for n in (M, N))
    bias, resid = rng.standard_normal(N).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    return a, sa, b, sb, bias, resid


def product_mag(a, sa, b, sb, bias, resid, epi):
    # one conversion, two products, the bias, the residual: five roundings of the terms;
    # silu's steepest slope is 1.1 and e^-v adds 2 + 1.2 |v| roundings of the value
    v = np.abs(a.astype(np.int64) @ b.astype(np.int64).T) * sa[:, None].astype(np.float64) * sb
    v = v + (0 if bias is None else np.abs(bias))
    return v + (np.abs(resid) if epi == "resid" else 0) if epi != "silu" else 1.1 * v


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 2048, 512), (8, 2048, 512), (16, 520, 48), (17, 64, 128), (64, 2048, 512),
                                   (127, 200, 144), (129, 1024, 4096), (300, 96, 1024), (1000, 4096, 1024), (513, 328, 272),
                                   (5000, 2048, 512), (20001, 1000, 528), (40003, 264, 64), (9473, 512, 2048)])
@pytest.mark.parametrize("epi,out", [("none", torch.float32), ("none", torch.float16), ("silu", torch.bfloat16),
                                     ("resid", torch.float32), ("silu", torch.float32)])
def test_int8_product(M, N, K, epi, out):
    a, sa, b, sb, bias, resid = product_case(M, N, K)
    g = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bias = bias if epi != "none" else None
    q_cols = 32 if (N >= 64 and epi == "none") else 0
    got = mt.gemm_i8(g(a), g(sa), g(b), g(sb), None if bias is None else g(bias), EPIS[epi],
                     g(resid) if epi == "resid" else None, q_cols, out, status=status)
    assert status.item() == 0
    rows = np.unique(np.concatenate([np.arange(min(M, 300)), np.arange(max(0, M - 300), M), np.linspace(0, M - 1, 200).astype(int)]))
    r = a[rows].astype(np.float64) @ b.astype(np.float64).T  # exact: below 2^53
    v = r * sa[rows][:, None].astype(np.float64) * sb
    if bias is not None:
        v += bias
    if epi == "silu":
        v = v / (1 + np.exp(-v))
    elif epi == "resid":
        v += resid[rows]
    v[:, :q_cols] *= 0.5
    near(got[torch.from_numpy(rows).cuda()], v, product_mag(a[rows], sa[rows], b, sb, bias, resid[rows], epi), f"{epi} {out}")
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("M", [17, 64, 100, 128, 129, 257])
@pytest.mark.parametrize("N,K", [(8, 512), (72, 528), (512, 1040), (1024, 4096), (1160, 2064), (264, 8208)])
@pytest.mark.parametrize("epi,out", [("none", torch.float32), ("silu", torch.float16), ("silu", torch.bfloat16), ("resid", torch.float32)])
def test_int8_product_split_over_k_is_the_same(M, N, K, epi, out):
    # few tiles, k shared by a cluster: the same bits as these rows in a product of many
    rng, many = torch.Generator(device="cuda").manual_seed(M + N + K), 10000
    a, b = (torch.randint(-127, 128, (n, K), generator=rng, device="cuda", dtype=torch.int8) for n in (many, N))
    sa, sb = ((torch.rand(n, generator=rng, device="cuda") + 0.5) / (73 * K ** 0.25) for n in (many, N))
    bias, resid = (torch.randn(n, generator=rng, device="cuda") for n in ((N,), (many, N)))
    q_cols = 32 if N >= 64 else 0
    want = mt.gemm_i8(a, sa, b, sb, bias, EPIS[epi], resid if epi == "resid" else None, q_cols, out)
    buf = torch.full((M + 300, N), 7.0, dtype=out, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mt.gemm_i8(a[:M], sa[:M], b, sb, bias, EPIS[epi], resid[:M] if epi == "resid" else None, q_cols, out,
               out=buf[8:8 + M], status=status)
    assert torch.equal(buf[8:8 + M], want[:M]) and (buf[:8] == 7).all() and (buf[8 + M:] == 7).all()
    assert status.item() == 0


def test_int8_product_extreme_sums_are_exact():
    # every byte -128: the sums pass 2^30; K close to the largest
    K = 131056
    a = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((64, K), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    one = torch.ones(130, device="cuda")
    got = mt.gemm_i8(a, one, b, one[:64].clone())
    assert (got[:, 0] == float(K * 16384)).all() and (got[:, 1] == float(np.float32(-128 * 127 * K))).all()


def test_int8_product_nan_rows_and_range():
    a, sa, b, sb, _, _ = product_case(40, 64, 64)
    sa[7] = np.nan
    g = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mt.gemm_i8(g(a), g(sa), g(b), g(sb), out_dtype=torch.float16, status=status)
    assert torch.isnan(got[7]).all() and torch.isfinite(got[[i for i in range(40) if i != 7]]).all() and status.item() == 0
    got = mt.gemm_i8(g(a), g(sa * 1e7), g(b), g(sb), out_dtype=torch.float16, status=status)
    assert status.item() == mt._lib.MTGR_ERR_RANGE and got[0].abs().max() == 65504


@pytest.mark.parametrize("M", [1, 5, 16, 17, 100, 3000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_is_quantise_then_product(M, dtype):
    x = torch.randn(M, 4 * 512, device="cuda").to(dtype)[:, 512:1024]
    w, ws = mt.quantize_rows(torch.randn(328, 512, device="cuda"))
    bias = torch.randn(328, device="cuda")
    q, s = mt.quantize_rows(x)
    for epi in (mt.MTGR_EPI_NONE, mt.MTGR_EPI_SILU):
        assert torch.equal(mt.linear_i8(x, w, ws, bias=bias, epi=epi), mt.gemm_i8(q, s, w, ws, bias, epi))


@pytest.mark.parametrize("M,N,K", [(9, 520, 512), (100, 1032, 4096), (1000, 1032, 512), (2500, 2048, 512), (2500, 1032, 2048)])
def test_linear_from_inputs_that_change(M, N, K):
    # in a graph: the product launches while its rows are quantised, and reads none of them before
    w, ws = mt.quantize_rows(torch.randn(N, K, device="cuda"))
    x = torch.randn(M, K, device="cuda")
    out = torch.empty(M, N, device="cuda")
    mt.linear_i8(x, w, ws, out_dtype=torch.float32, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mt.linear_i8(x, w, ws, out_dtype=torch.float32, out=out)
    for k in range(4):
        x.copy_(torch.randn(M, K, device="cuda") * (k + 1))
        q, s = mt.quantize_rows(x)
        want = mt.gemm_i8(q, s, w, ws, out_dtype=torch.float32)
        out.zero_()
        graph.replay()
        assert torch.equal(out, want), k
        y = q.double() @ w.double().T * s.double()[:, None] * ws.double()
        mag = (q.double() @ w.double().T).abs() * s.double()[:, None] * ws.double()
        near(out, y.cpu().numpy(), mag.cpu().numpy(), "linear")


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (16, 72, 528), (17, 200, 64), (129, 520, 144), (9000, 1160, 512), (9001, 1000, 640)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
def test_product_writes_its_rows_alone(M, N, K, out):
    a, sa, b, sb, _, _ = product_case(M, N, K)
    g = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    buf = torch.full((M + 300, N), 7.0, dtype=out, device="cuda")
    mt.gemm_i8(g(a), g(sa), g(b), g(sb), out_dtype=out, out=buf[8:8 + M])
    assert (buf[:8] == 7).all() and (buf[8 + M:] == 7).all()
    assert torch.equal(buf[8:8 + M], mt.gemm_i8(g(a), g(sa), g(b), g(sb), out_dtype=out))


def test_product_no_rows_or_columns():
    w, ws = torch.zeros(64, 128, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    assert mt.linear_i8(torch.zeros(0, 128, device="cuda"), w, ws).shape == (0, 64)
    assert mt.linear_i8(torch.zeros(5, 128, device="cuda"), w[:0], ws[:0]).shape == (5, 0)


# -------------------------------------------------------------------- clip --
def clip_case(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda() for i, n in enumerate(sizes)]


def check_clip(grads, outs, max_norm, inv, s=None):
    before = [host(x) for x in grads]
    norm = (s or mt.GradientSet(grads, outs)).clip(max_norm, inv)
    want, clipped = op.grad_clip(before, max_norm, inv)
    # squares of eight in fp32 (8 roundings, all positive), the rest in fp64; halved by the root
    assert abs(norm.item() - want) <= 8 * 2.0 ** -24 * want
    for o, w in zip(grads if outs is None else outs, clipped):
        if w.size:  # the factor: the norm's error and three roundings; the product: one
            near(o, w, np.abs(w), "clipped")
    return norm


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [7, 1, 16385, 0], [100003], [16384, 32768], list(range(1, 400)),
                                   [3 * 1000003, 17]])
@pytest.mark.parametrize("dtypes", [(torch.float32,), (torch.bfloat16,), (torch.float16,),
                                    (torch.float32, torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("to", ["same", "f32", "in place"])
def test_clip(sizes, dtypes, to):
    grads = clip_case(sizes, dtypes)
    outs = None if to == "in place" else [torch.empty_like(x, dtype=x.dtype if to == "same" else torch.float32) for x in grads]
    check_clip(grads, outs, 0.5, 0.25)


def test_clip_leaves_small_norms_alone():
    grads = clip_case([1000, 33], (torch.float32, torch.bfloat16))
    keep = [x.clone() for x in grads]
    s = mt.GradientSet(grads)
    assert abs(s.clip(1e9).item() - np.sqrt(sum((host(x) ** 2).sum() for x in keep))) < 1e-3
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    s.clip(float("inf"), 0.5)
    assert all(torch.equal(a, (b.float() * 0.5).to(b.dtype)) for a, b in zip(grads, keep))
    s.clip(0.0)
    assert all((a == 0).all() for a in grads)
    s.check()


def test_clip_odd_addresses():
    flat = torch.randn(5000, device="cuda")
    half = torch.randn(5000, device="cuda").bfloat16()
    grads = [flat[1:1000], flat[1003:2000], half[1:77], half[101:2500], half[2501:2502]]
    outs = [torch.empty(x.numel() + 3, dtype=x.dtype, device="cuda")[i % 3:][:x.numel()] for i, x in enumerate(grads)]
    check_clip(grads, outs, 0.1, 1.0)
    check_clip(grads, None, 0.1, 1.0)


@pytest.mark.parametrize("shift", [0, 1, 3, 4])
@pytest.mark.parametrize("dtype,to", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float16, torch.float16)])
def test_clip_writes_its_tensors_alone(dtype, to, shift):
    sizes = [1, 7, 8, 100, 16384, 16391, 40000]
    grads, outs, buf = [], [], torch.full((sum(sizes) + 64 * len(sizes),), 5.0, dtype=to, device="cuda")
    at = 16 + shift
    inside = torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
    for i, n in enumerate(sizes):
        grads.append(torch.randn(n + 8, device="cuda").to(dtype)[i % 5:][:n])
        outs.append(buf[at:at + n])
        inside[at:at + n] = True
        at += n + 40 + i
    check_clip(grads, outs, 0.1, 1.0)
    assert (buf[~inside] == 5).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e19, 1e30])
def test_clip_sums_beyond_fp32(scale):
    check_clip(clip_case([5003, 17], (torch.float32,), scale=scale), None, 1.0, 1e-30 if scale > 1 else 1.0)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_clip_norm_not_finite_touches_nothing(bad):
    grads = clip_case([100, 200], (torch.float32,))
    grads[1][150] = bad
    outs = [torch.full_like(x, 3.0) for x in grads]
    s = mt.GradientSet(grads, outs)
    assert not torch.isfinite(s.clip(1.0)).item() and all((o == 3.0).all() for o in outs)
    with pytest.raises(mt.MTGRError):
        s.check()
    s.check()  # cleared


def test_clip_norm_alone_and_overlaps():
    grads = clip_case([300, 70000], (torch.float32, torch.bfloat16))
    keep = [x.clone() for x in grads]
    s = mt.GradientSet(grads)
    want = 2.0 * np.sqrt(sum((host(x) ** 2).sum() for x in grads))
    assert abs(s.norm(2.0).item() - want) <= 1e-5 * want and all(torch.equal(a, b) for a, b in zip(grads, keep))
    flat = torch.zeros(100, device="cuda")
    for g, o in (([flat, flat], None), ([flat[:60], flat[50:]], None), ([flat[:50]], [flat[10:60]]),
                 ([flat[:50], flat[50:]], [flat[50:], flat[:50]])):
        with pytest.raises(ValueError):
            mt.GradientSet(g, o)
    mt.GradientSet([flat, flat], [torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")])  # read twice: fine


def held_values():  # the most values of one tensor that the one-kernel form takes
    return torch.cuda.get_device_properties(0).multi_processor_count * 2 * 4 * 4096


@pytest.mark.parametrize("more", [-1, 0, 1, 5000])
@pytest.mark.parametrize("rest", [[], [0, 3, 0]])
def test_clip_at_the_border_of_the_forms(more, rest):
    sizes = [held_values() + more - sum(4096 for n in rest if n)] + rest
    for to in (torch.float32, torch.bfloat16):
        grads = clip_case(sizes, (torch.bfloat16,))
        outs = [torch.full((x.numel() + 64,), 5.0, dtype=to, device="cuda") for x in grads]
        check_clip(grads, [o[32:32 + x.numel()] for o, x in zip(outs, grads)], 0.5, 0.25)
        assert all((o[:32] == 5).all() and (o[32 + x.numel():] == 5).all() for o, x in zip(outs, grads))


def test_clip_again_and_again():
    # a set's workspace is left fit for the next call: many in a row, no wait between, then in a graph
    grads = clip_case([70001, 0, 300, 500000], (torch.float32, torch.bfloat16))
    outs = [torch.empty_like(x) for x in grads]
    s = mt.GradientSet(grads, outs)
    want = s.clip(0.5, 0.25)
    first = [o.clone() for o in outs]
    norms = [s.clip(0.5, 0.25) for _ in range(200)]
    assert all(torch.equal(n, want) for n in norms)
    assert (s.ws[:8] == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pair = [s.clip(0.5, 0.25), s.norm(0.25)]
    for _ in range(50):
        for o in outs:
            o.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(n, want) for n in pair) and all(torch.equal(a, b) for a, b in zip(outs, first))
    s.check()


def test_clips_of_two_sets_at_once():
    # each a cooperative kernel over the whole GPU: neither may keep the other from ending
    sets, streams, want = [], [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        grads = clip_case([held_values() - 8192 * (i + 1), 77], (torch.float32,), seed=i)
        sets.append(mt.GradientSet(grads, [torch.empty_like(x) for x in grads]))
        want.append(sets[i].clip(0.5))
    torch.cuda.synchronize()
    norms = [[], []]
    for _ in range(30):
        for i in range(2):
            norms[i].append(sets[i].clip(0.5, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(n, want[i]) for n in norms[i])
        sets[i].check()


# ------------------------------------------- streams, graphs, run together --
def test_on_another_stream_and_in_a_graph():
    dev, _ = case(600, 512)
    dh, dy = upstream(600, 512)
    w, ws = mt.quantize_rows(torch.randn(2048, 512, device="cuda"))

    def step(stream=None):
        h, y, ys = mt.boundary_forward(**dev, y_dtype=torch.int8, stream=stream)
        z = mt.gemm_i8(y, ys, w, ws, out_dtype=torch.float16, stream=stream)
        z2 = mt.linear_i8(h, w, ws, stream=stream)
        back = mt.boundary_backward(**dev, dh=dh, dy=dy, stream=stream)
        out = [torch.empty_like(back[n]) for n in NAMES]
        norm = mt.GradientSet([back[n] for n in NAMES], out).clip(0.1, 1.0, stream=stream)
        return [h, y, ys, z, z2, norm, back["dx"], back["do"], *out]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # captured: the plan made ahead, as a training program keeps it
    back = mt.boundary_backward(**dev, dh=dh, dy=dy)
    grads = [back[n].clone() for n in NAMES]
    outs = [torch.empty_like(x) for x in grads]
    plan = mt.GradientSet(grads, outs)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h, y, ys = mt.boundary_forward(**dev, y_dtype=torch.int8)
        z = mt.gemm_i8(y, ys, w, ws, out_dtype=torch.float16)
        z2 = mt.linear_i8(h, w, ws)
        b = mt.boundary_backward(**dev, dh=dh, dy=dy)
        norm = plan.clip(0.1, 1.0)
    for k in range(2):
        if k:  # other inputs in the same buffers
            dev["o"].copy_(dev["o"] * 0.5 + 0.25)
            want = step()
            for x, n in zip(grads, NAMES):
                x.copy_(mt.boundary_backward(**dev, dh=dh, dy=dy)[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [h, y, ys, z, z2, norm, b["dx"], b["do"], *outs]
        assert all(torch.equal(p, q) for p, q in zip(want, got)), k


def test_two_streams_at_once():
    # calls that overlap on the GPU keep apart: workspaces are each call's own
    devs = [case(3000, 512, seed=i)[0] for i in range(2)]
    ups = [upstream(3000, 512, seed=i) for i in range(2)]
    w, ws = mt.quantize_rows(torch.randn(1024, 512, device="cuda"))

    def work(i, stream):
        out = []
        for _ in range(8):
            h, y, ys = mt.boundary_forward(**devs[i], y_dtype=torch.int8, stream=stream)
            out += [h, y, ys, mt.gemm_i8(y, ys, w, ws, stream=stream), mt.linear_i8(h, w, ws, stream=stream),
                    mt.linear_i8(h[:7], w, ws, stream=stream)]
            b = mt.boundary_backward(**devs[i], dh=ups[i][0], dy=ups[i][1], stream=stream)
            out += list(b.values())
        return out

    want = [work(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [work(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_serving_block_from_boundary_to_mlp():
    """One block's products in int8, from the boundary before it to its second MLP
    product, against the same steps in float64 on the same quantised weights:
    every activation is rounded to 8 bits twice, about 1% of its size."""
    T, d, ff = 500, 512, 2048
    dev, r = case(T, d, gate="silu", seed=4)
    wn = [(np.random.default_rng(i).standard_normal(s) / np.sqrt(s[1])).astype(np.float32) for i, s in
          enumerate([(ff, d), (d, ff)])]
    (w1, s1), (w2, s2) = (mt.quantize_rows(torch.from_numpy(w).cuda()) for w in wn)
    h, y, ys = mt.boundary_forward(**dev, gate="silu", y_dtype=torch.int8)
    z = mt.gemm_i8(y, ys, w1, s1, epi=mt.MTGR_EPI_SILU, out_dtype=torch.bfloat16)
    out = mt.linear_i8(z, w2, s2, epi=mt.MTGR_EPI_RESID, resid=h)
    hr, yr = op.boundary_forward(**oracle_args(r), kind="silu")
    zr = yr @ (host(w1) * host(s1)[:, None]).T
    zr = zr / (1 + np.exp(-zr))
    branch = zr @ (host(w2) * host(s2)[:, None]).T
    err = host(out) - (hr + branch)
    # a byte's error is at most half a step of its row's largest over 127, uniform: rms
    # step / sqrt(12); both products average over independent errors (1% of the rms each)
    assert np.sqrt((err ** 2).mean()) <= 0.03 * np.sqrt((branch ** 2).mean())


def test_training_step_from_backward_to_clip():
    """The boundary's gradients and a block's, clipped as one set."""
    T, d = 700, 512
    dev, r = case(T, d)
    dh, dy = upstream(T, d)
    back = mt.boundary_backward(**dev, dh=dh * 1024, dy=(dy * 1024))
    names = list(NAMES)
    x = torch.randn(T, 256, device="cuda").bfloat16()
    dw = mt.gemm_wgrad(x, dev["o"])  # a Linear's weight gradient beside them
    grads = [back[n] for n in names] + [dw]
    want_norm, want = op.grad_clip([host(g) for g in grads], 1.0, 1.0 / 1024)
    outs = [torch.empty_like(g) for g in grads]
    s = mt.GradientSet(grads, outs)
    norm = s.clip(1.0, 1.0 / 1024)
    s.check()
    assert abs(norm.item() - want_norm) <= 1e-6 * want_norm
    for o, v in zip(outs, want):
        near(o, v, np.abs(v), "clipped")


def test_refusals_on_the_device():
    dev, _ = case(4, 64)
    with pytest.raises(ValueError):
        mt.boundary_forward(**dev, gate="tanh")
    with pytest.raises(ValueError):
        mt.boundary_forward(**dev, y_dtype=torch.float16)
    for k, v in (("o", dev["o"].float().t().contiguous().t()), ("group_id", dev["group_id"].long()),
                 ("post_gamma", dev["post_gamma"][:, ::2]), ("scale", dev["scale"].bfloat16()), ("u", None),
                 ("x", dev["x"].half()), ("post_beta", None)):
        with pytest.raises(ValueError):
            mt.boundary_forward(**{**dev, k: v})
    dh = torch.zeros_like(dev["x"])
    with pytest.raises(ValueError):
        mt.boundary_backward(**dev, dh=dh)  # no dy
    with pytest.raises(ValueError):
        mt.boundary_backward(**dev, dh=dh.bfloat16(), dy=dh)
    w, ws = torch.zeros(64, 64, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    for bad in (dict(x_scale=ws[:4]), dict(resid=x), dict(epi=mt.MTGR_EPI_RESID), dict(bias=ws[:3])):
        with pytest.raises(ValueError):
            mt.linear_i8(x, w, ws, **bad)
    with pytest.raises(ValueError):
        mt.linear_i8(x.to(torch.int8), w, ws)
    with pytest.raises(ValueError):
        mt.gemm_i8(x, ws[:4], w, ws)
    with pytest.raises(mt.MTGRError):
        mt.linear_i8(x, w, ws, q_cols=8)
    with pytest.raises(mt.MTGRError):  # rows 64 apart, 60 long: the library refuses the length
        mt.quantize_rows(torch.zeros(4, 64, device="cuda")[:, :60])
    with pytest.raises(ValueError):  # rows 60 apart
        mt.quantize_rows(torch.zeros(4, 60, device="cuda"))
