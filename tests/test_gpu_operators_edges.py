"""The operators' calls beside the ordinary ones, each against the float64 oracle or
against the same call made plainly. Tolerances: tests/test_gpu_operators.py."""

import threading
import types

import numpy as np
import pytest
import torch

import generative_recommendation_ranking_b200 as mt
from oracle import operators as op
from test_gpu_operators import (EPIS, HALF, NAMES, case, clip_case, host, mags, near, oracle_args, product_case,
                                upstream)

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


# ----------------------------------------------------------------- streams --
def stream_calls():
    """Each operator that allocates, on fixed inputs: its outputs on a stream."""
    dev, _ = case(3000, 512)
    dh, dy = upstream(3000, 512)
    w, ws = mt.quantize_rows(torch.randn(1024, 512, device="cuda"))
    x = torch.randn(3000, 512, device="cuda")
    q, s = mt.quantize_rows(x)
    plan = mt.GradientSet([torch.randn(100003, device="cuda")], [torch.empty(100003, device="cuda")])
    return {
        "forward": lambda st: mt.boundary_forward(**dev, y_dtype=torch.int8, stream=st),
        "backward": lambda st: tuple(mt.boundary_backward(**dev, dh=dh, dy=dy, stream=st).values()),
        "quantise": lambda st: mt.quantize_rows(x, stream=st),
        "product": lambda st: (mt.gemm_i8(q, s, w, ws, stream=st),),
        "linear": lambda st: (mt.linear_i8(x, w, ws, stream=st),),
        "linear, few rows": lambda st: (mt.linear_i8(x[:9], w, ws, stream=st),),
        "clip": lambda st: (plan.clip(0.5, stream=st), *plan.outs),
        "norm": lambda st: (plan.norm(stream=st),),
    }


STREAM_CALLS = ["forward", "backward", "quantise", "product", "linear", "linear, few rows", "clip", "norm"]


def outputs_alone(name, got):
    return got[:1] if name == "clip" else got  # what the call allocates


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_another_streams_buffers_are_no_dropped_ones(name):
    # a kernel of the current stream is still to write buffers that were dropped: a call on
    # another stream, which nothing orders behind it, gets none of them
    call = stream_calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = [torch.empty_like(t) for t in want for _ in range(4)]
    junk += [torch.empty(n << 20, dtype=torch.uint8, device="cuda") for n in (1, 2, 4, 8, 16, 32, 64)]  # workspaces
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for t in junk:
        t.view(torch.uint8).fill_(0x55)
    del junk, t
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_dropped_results_wait_for_their_reader(name):
    # results read on the current stream, dropped before that has run: the next call on the
    # other stream does not get their memory
    call = stream_calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    now = torch.cuda.current_stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = outputs_alone(name, list(call(side)))
    now.wait_stream(side)
    side.synchronize()
    torch.cuda._sleep(200_000_000)
    keep = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        junk = [torch.empty_like(t).view(torch.uint8).fill_(0x55) for t in keep for _ in range(4)]
    again = outputs_alone(name, call(side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, keep)) and all(torch.equal(a, b) for a, b in zip(want, again))
    del junk


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_on_a_side_stream_of_a_capture(name):
    call = stream_calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        got = call(side)
        now.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, copies))


def test_workspaces_of_another_stream_are_used_again():
    # no reader on the current stream: a workspace does not wait for what runs there
    w, ws = mt.quantize_rows(torch.randn(1024, 512, device="cuda"))
    x, out = torch.randn(30000, 512, device="cuda"), torch.empty(30000, 1024, device="cuda")
    side = torch.cuda.Stream()
    mt.linear_i8(x, w, ws, out=out, stream=side)
    torch.cuda.synchronize()
    room = torch.cuda.memory_reserved()
    torch.cuda._sleep(200_000_000)
    for _ in range(20):
        mt.linear_i8(x, w, ws, out=out, stream=side)
    assert torch.cuda.memory_reserved() == room
    torch.cuda.synchronize()


# ------------------------------------------------------------ int8 product --
@pytest.mark.parametrize("M,N,K", [(9, 72, 512), (17, 64, 512), (100, 64, 512), (100, 64, 4096), (1001, 328, 512), (9001, 2048, 512), (9001, 2048, 528)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
def test_range_is_that_of_the_rows(M, N, K, out):
    # a bias beyond f16 that every row's product brings back into it: the rows a tile has
    # behind the last, of the bias alone, say nothing
    a = torch.full((M, K), 100, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -100, dtype=torch.int8, device="cuda")
    one, bias = torch.ones(N, device="cuda"), torch.full((N,), 1e5, device="cuda")
    sa = torch.full((M,), 9e4 / (K * 1e4), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mt.gemm_i8(a, sa, b, one, bias, out_dtype=out, status=status)
    assert status.item() == 0
    # -9e4 + 1e5 with three roundings near 1e5, then one to the output's type
    assert ((got.double() - 1e4).abs() <= 3 * 1e5 * 2.0 ** -24 + 1e4 * 2.0 ** -11).all()
    sa[M - 1] = 0.0  # the last row of the output is the bias
    mt.gemm_i8(a, sa, b, one, bias, out_dtype=out, status=status)
    assert status.item() == (mt._lib.MTGR_ERR_RANGE if out == torch.float16 else 0)


def test_few_rows_from_several_threads():
    # calls of two lengths of k at once, each with its own shared memory: none is refused
    # (60,000 calls in each of four threads: some dozens were where the threads' limits mixed)
    f = mt.load().mtgr_linear_i8
    refused, outs = [], []

    def work(K):
        x = torch.randn(8, K, device="cuda")
        w = torch.ones(16, K, dtype=torch.int8, device="cuda")
        scale, out = torch.ones(16, device="cuda"), torch.empty(8, 16, device="cuda")
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        args = (8, 16, K, mt.MTGR_F32, x.data_ptr(), K, w.data_ptr(), scale.data_ptr(), None, 0, None, 0, mt.MTGR_F32,
                out.data_ptr(), None, 0, None, stream.cuda_stream)
        refused.append(sum(f(*args) != 0 for _ in range(60000)))
        stream.synchronize()
        outs.append(torch.equal(out, mt.linear_i8(x, w, scale)))

    threads = [threading.Thread(target=work, args=(K,)) for K in (2816, 6016, 2816, 6016)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == [0] * 4 and outs == [True] * 4


@pytest.mark.parametrize("N,K", [(8, 16), (72, 528), (328, 512), (2048, 512), (1024, 4096)])
@pytest.mark.parametrize("epi,out", [("none", torch.float32), ("none", torch.float16), ("silu", torch.float32),
                                     ("silu", torch.bfloat16), ("resid", torch.float32)])
def test_a_rows_bits_do_not_depend_on_the_rows_beside_it(N, K, epi, out):
    # one to sixteen rows take one form, the others tiles of one or two CTAs, or k in shares
    a, sa, b, sb, bias, resid = (torch.from_numpy(v).cuda() for v in product_case(10007, N, K))
    x = torch.randn(10007, K, device="cuda")
    q_cols = 32 if N >= 64 else 0

    def both(n):
        more = (b, sb, bias, EPIS[epi], resid[:n] if epi == "resid" else None, q_cols, out)
        return mt.gemm_i8(a[:n], sa[:n], *more), mt.linear_i8(x[:n], *more[:2], bias=more[2], epi=more[3], resid=more[4],
                                                             q_cols=more[5], out_dtype=more[6])

    want = both(10007)
    for n in (1, 2, 15, 16, 17, 129, 1000):
        for g, v in zip(both(n), want):
            assert torch.equal(g, v[:n]), n


# -------------------------------------------------------------- workspaces --
def test_given_workspaces():
    dev, _ = case(300, 256)
    dh, dy = upstream(300, 256)
    x, (w, ws) = torch.randn(300, 256, device="cuda"), mt.quantize_rows(torch.randn(64, 256, device="cuda"))
    want = mt.boundary_backward(**dev, dh=dh, dy=dy)
    calls = (lambda b: mt.boundary_backward(**dev, dh=dh, dy=dy, ws=b)["scale"], lambda b: mt.linear_i8(x, w, ws, ws=b))
    for call, ref in zip(calls, (want["scale"], mt.linear_i8(x, w, ws))):
        for bad in (torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(bad)
        for good in (None, torch.zeros(1 << 22, device="cuda"), torch.zeros(16, device="cuda")):  # the last is too small
            assert torch.equal(call(good), ref)
    with pytest.raises(ValueError):  # checked for few rows, too, which need none
        mt.linear_i8(x[:4], w, ws, ws=torch.zeros(64, dtype=torch.uint8))


def test_the_entry_points_one_by_one():
    # the binding's wrappers of the library's entry points, on the caller's buffers
    L = mt._lib
    dev, _ = case(40, 264, gate="silu")
    names = NAMES
    p = L.MtgrBoundaryParams(264, 4, 1e-5, L.MTGR_GATE_SILU, *[dev[n].data_ptr() for n in names])
    h, y, ys = torch.empty(40, 264, device="cuda"), torch.empty(40, 264, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    mt.mtgr_boundary_fwd(p, 40, dev["group_id"], dev["o"], dev["u"], dev["x"], h, y, ys)
    want = mt.boundary_forward(**dev, gate="silu", y_dtype=torch.int8)
    assert all(torch.equal(a, b) for a, b in zip((h, y, ys), want))
    # no rows: no workspace
    none = {k: (v[:0] if k in ("x", "o", "u", "group_id") else v) for k, v in dev.items()}
    grads = {n: torch.full((4, 264), 7.0, device="cuda") for n in names}
    mt.mtgr_boundary_bwd(p, 0, none["group_id"], none["o"], none["u"], none["x"], None, none["x"], none["o"], none["o"], none["x"],
                         L.MtgrBoundaryGrads(*[grads[n].data_ptr() for n in names]), None)
    assert all((g == 0).all() for g in grads.values())
    x = torch.randn(40, 272, device="cuda")
    q, s = torch.empty(40, 272, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    mt.mtgr_quantize_rows(x, q, s)
    assert all(torch.equal(a, b) for a, b in zip((q, s), mt.quantize_rows(x)))
    w, ws = mt.quantize_rows(torch.randn(72, 272, device="cuda"))
    out, status = torch.empty(40, 72, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mt.mtgr_gemm_i8(q, s, w, ws, None, mt.MTGR_EPI_SILU, None, 0, out, status)
    ref = mt.gemm_i8(q, s, w, ws, epi=mt.MTGR_EPI_SILU)
    assert torch.equal(out, ref)
    room = torch.empty(mt.mtgr_linear_i8_workspace_bytes(40, 72, 272), dtype=torch.uint8, device="cuda")
    for n, buf in ((40, room), (9, None)):  # few rows: no workspace
        out.zero_()
        mt.mtgr_linear_i8(x[:n], w, ws, None, mt.MTGR_EPI_SILU, None, 0, out[:n], buf, status)
        assert torch.equal(out[:n], ref[:n]) and (out[n:] == 0).all()
    assert status.item() == 0
    g, o, norm = torch.randn(1003, device="cuda"), torch.empty(1003, device="cuda"), torch.empty(1, device="cuda")
    table = (L.MtgrGradTensor * 1)(L.MtgrGradTensor(g.data_ptr(), o.data_ptr(), 1003, mt.MTGR_F32, mt.MTGR_F32))
    room = torch.zeros(mt.mtgr_grad_clip_workspace_bytes(table, 1), dtype=torch.uint8, device="cuda")
    mt.mtgr_grad_clip(table, 1, 0.5, 0.25, norm, room, status)
    plan = mt.GradientSet([g], [torch.empty_like(g)])
    assert torch.equal(norm, plan.clip(0.5, 0.25)) and torch.equal(o, plan.outs[0]) and status.item() == 0


# --------------------------------------------- long runs of the backward --
def check_long(T, d, order, rows, G=4, gate="linear", branch=torch.bfloat16):
    """The backward over many rows a team against the oracle, chunk by chunk of rows.

    A team's gradient sums are fp32 over its run of at most `rows` rows: as many
    roundings of partial sums, each at most 2^-24 of the terms' magnitudes added up,
    beside the 128 of a term; the teams are added up in fp64."""
    rng = np.random.default_rng(T + d)
    gid = rng.integers(0, G, T)
    if order == "sorted":
        gid = np.sort(gid)
    elif order == "users":  # runs of every group, some shorter than a team's rows, some longer
        gid = np.repeat(np.arange(T) % G, rng.integers(1, 60, T))[:T]
    dev, r = case(T, d, branch, gate=gate, G=G, gid=gid)
    dh, dy = upstream(T, d)
    out = mt.boundary_backward(**dev, dh=dh, dy=dy, gate=gate)
    names = NAMES
    want, mag = ({n: np.zeros((G, d)) for n in names} for _ in range(2))
    step = max(1, 4_000_000 // d)
    for t in range(0, T, step):
        cut = slice(t, min(T, t + step))
        part = {k: (v[cut] if k in ("x", "o", "u", "gid") and v is not None else v) for k, v in r.items()}
        a, b = host(dh[cut]), host(dy[cut])
        w = op.boundary_backward(**oracle_args(part), dh=a, dy=b, kind=gate)
        m = mags(part, gate, a, b)
        for k in w:
            if k in names:
                want[k] += w[k]
                mag[k] += m[k]
            else:
                near(out[k][cut], w[k], m[k], f"{k}, rows from {t}")
    for n in names:
        g = host(out[n])
        tol = (128 + rows) * 2.0 ** -24 * mag[n] + 2.0 ** -24 * np.abs(want[n])
        assert (np.abs(g - want[n]) <= tol).all(), (n, np.abs(g - want[n]).max())


# 17 rows a team on 148 SMs, the last team's fewer
LONG = [(120011, 64), (60013, 128), (30011, 256), (20011, 512), (10007, 1024), (5003, 2048), (2503, 4096), (2503, 8192)]


@pytest.mark.parametrize("T,d", LONG)
@pytest.mark.parametrize("order", ["sorted", "users", "any"])
def test_boundary_backward_long_runs(T, d, order):
    check_long(T, d, order, 32)


# 113, 113 and 50 rows a team
@pytest.mark.parametrize("T,d,G,gate,rows", [(200003, 256, 4, "silu", 128), (400009, 120, 4, "none", 128), (2503, 8192, 32, "linear", 64)])
def test_boundary_backward_a_hundred_rows_a_team(T, d, G, gate, rows):
    check_long(T, d, "users", rows, G, gate, torch.float16)


# ------------------------------------ in place, past 32 bits, in a capture --
@pytest.mark.parametrize("d", [8, 64, 104, 256, 512, 1024, 8192])
@pytest.mark.parametrize("stream", [torch.float32, torch.bfloat16])
def test_boundary_backward_dx_in_place_of_dh(d, stream):
    T = 1003 if d < 8192 else 301
    dev, _ = case(T, d, stream=stream)
    dh, dy = upstream(T, d, stream)
    want = mt.boundary_backward(**dev, dh=dh, dy=dy)
    p = mt._lib.MtgrBoundaryParams(d, 4, 1e-5, mt._lib.MTGR_GATE_LINEAR, *[dev[n].data_ptr() for n in NAMES])
    par = {n: torch.empty(4, d, device="cuda") for n in NAMES}
    do, du = torch.empty_like(want["do"]), torch.empty_like(want["du"])
    ws = torch.empty(mt._lib.mtgr_boundary_bwd_workspace_bytes(T, p), dtype=torch.uint8, device="cuda")
    mt._lib.mtgr_boundary_bwd(p, T, dev["group_id"], dev["o"], dev["u"], dev["x"], dh, dy, do, du, dh,
                        mt._lib.MtgrBoundaryGrads(*[par[n].data_ptr() for n in NAMES]), ws)
    assert torch.equal(dh, want["dx"]) and torch.equal(do, want["do"]) and torch.equal(du, want["du"])
    assert all(torch.equal(par[n], want[n]) for n in NAMES)


def test_boundary_past_32_bits():
    # 2^31 + values: the last rows against a call on them alone
    T, d = 4_200_000, 512
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s, t: torch.empty(*s, device="cuda", dtype=t).normal_(generator=g)  # noqa: E731
    dev = dict(x=r(T, d, t=torch.float32), o=r(T, d, t=torch.bfloat16), u=r(T, d, t=torch.bfloat16),
               group_id=torch.randint(0, 4, (T,), generator=g, device="cuda", dtype=torch.int8),
               **{n: r(4, d, t=torch.float32) for n in NAMES})
    n = 777
    last = {k: (v[-n:] if v.shape[0] == T else v) for k, v in dev.items()}
    got = mt.boundary_forward(**dev, y_dtype=torch.int8)
    want = mt.boundary_forward(**last, y_dtype=torch.int8)
    assert all(torch.equal(a[-n:], b) for a, b in zip(got, want))
    del got, want
    dh, dy = r(T, d, t=torch.float32), r(T, d, t=torch.bfloat16)
    got = mt.boundary_backward(**dev, dh=dh, dy=dy)
    want = mt.boundary_backward(**last, dh=dh[-n:], dy=dy[-n:])
    assert all(torch.equal(got[k][-n:], want[k]) for k in ("dx", "do", "du"))
    # dbeta of the norm before: dy's sums, at most 3552 rows a team in fp32
    pre = torch.stack([dy[dev["group_id"] == g].double().sum(0) for g in range(4)])
    mag = torch.stack([dy[dev["group_id"] == g].double().abs().sum(0) for g in range(4)])
    assert ((got["pre_beta"] - pre).abs() <= (4000 * 2.0 ** -24) * mag).all()


def test_quantise_and_product_past_32_bits():
    M, K, N = 4_200_000, 512, 520
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w, ws = mt.quantize_rows(torch.randn(N, K, device="cuda"))
    q, s = mt.quantize_rows(x)
    n = 777
    ql, sl = mt.quantize_rows(x[-n:])
    assert torch.equal(q[-n:], ql) and torch.equal(s[-n:], sl)
    for out, epi in ((torch.float32, "resid"), (torch.float16, "none")):
        resid = torch.empty(M, N, device="cuda").normal_(generator=g) if epi == "resid" else None
        got = mt.gemm_i8(q, s, w, ws, None, EPIS[epi], resid, 0, out)
        want = mt.gemm_i8(ql, sl, w, ws, None, EPIS[epi], None if resid is None else resid[-n:], 0, out)
        assert torch.equal(got[-n:], want)
        if resid is None:
            assert torch.equal(mt.linear_i8(x, w, ws, out_dtype=out), got)
    wide = x.view(-1)[:4 * 512 * (M // 4)].view(M // 4, 4 * 512)[:, -512:]
    assert torch.equal(mt.linear_i8(wide, w, ws)[-n:], mt.linear_i8(wide[-n:].contiguous(), w, ws))


def test_wide_weights_past_32_bits():
    # N K past 2^31
    N, K = 70_000 * 8, 4096
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.ones(N, device="cuda") * 1e-5
    for M in (5, 40):
        q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        s = torch.ones(M, device="cuda")
        got = mt.gemm_i8(q, s, w, ws)
        assert torch.equal(got[:, -800:], mt.gemm_i8(q, s, w[-800:], ws[-800:]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_past_32_bits(dtype):
    n = (1 << 31) + 12345
    g = torch.zeros(n, device="cuda", dtype=dtype)
    g[-5000:] = 3.0
    g[:3] = 4.0
    s = mt.GradientSet([g, torch.ones(7, device="cuda")])
    want = (9.0 * 5000 + 16 * 3 + 7) ** 0.5
    assert abs(s.clip(1.0).item() - want) <= 1e-6 * want
    f = 1.0 / (want + 1e-6)
    assert torch.allclose(g[-5000:].float(), torch.full((5000,), 3 * f, device="cuda"), rtol=1.01 * 2.0 ** -8)
    assert torch.allclose(g[:3].float(), torch.full((3,), 4 * f, device="cuda"), rtol=1.01 * 2.0 ** -8)
    assert (g[3:-5000] == 0).all()


def test_set_made_in_a_capture():
    grads = [torch.randn(100003, device="cuda"), torch.randn(77, device="cuda")]
    want = mt.GradientSet(grads, [torch.empty_like(x) for x in grads])
    norm = want.clip(0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    outs = [torch.empty_like(x) for x in grads]
    with torch.cuda.graph(graph):
        s = mt.GradientSet(grads, outs)
        n = s.clip(0.5)
    for _ in range(3):
        [o.zero_() for o in outs]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(outs, want.outs))
        s.check()
    assert torch.equal(s.clip(0.5), norm)


@pytest.mark.parametrize("M,N,K", [(10007, 2048, 512), (9001, 2048, 512), (20011, 1000, 512), (40003, 264, 512), (20011, 2560, 512), (10007, 2048, 384),
                                   (5003, 1000, 496), (9001, 4096, 272), (9001, 3840, 272), (40003, 72, 48), (10007, 4608, 512), (10007, 4616, 400)])
@pytest.mark.parametrize("epi,out", [("none", torch.float16), ("silu", torch.float32), ("resid", torch.float32)])
def test_weights_that_stay_in_shared_memory(M, N, K, epi, out):
    # on either side of the rule for the pairs' columns: the same bits as 1000 rows, in small tiles
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b = (torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    sa, sb = ((torch.rand(n, generator=g, device="cuda") + 0.5) / (73 * K ** 0.25) for n in (M, N))
    bias, resid = (torch.randn(s, generator=g, device="cuda") for s in ((N,), (M, N)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def product(rows):
        return mt.gemm_i8(a[rows], sa[rows], b, sb, bias, EPIS[epi], resid[rows] if epi == "resid" else None, 32, out, status=status)

    got = product(slice(0, M))
    for t in list(range(0, M, 1000)):
        rows = slice(t, min(M, t + 1000))
        assert torch.equal(got[rows], product(rows)), t
    assert status.item() == 0


# -------------------------------------------------------------------- clip --
@pytest.mark.parametrize("sizes", [[5003, 17], [16384 * 700, 40000], [300] * 200])
@pytest.mark.parametrize("dtype,to", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("scale,max_norm,inv", [(1e34, 1.0, 1.0), (1e34, 1e-3, 1.0), (1e34, 1e-20, 1.0), (1e34, 1e30, 1e-38), (1e30, 1e-18, 0.25),
                                                (3e33, 1e-40, 1.0)])
def test_clip_factors_below_the_normal_numbers(sizes, dtype, to, scale, max_norm, inv):
    # max_norm / norm of an exploded step: the clipped values are ordinary numbers though the
    # factor is not one of fp32's
    grads = clip_case(sizes, (dtype,), scale=scale)
    outs = None if dtype == to else [torch.empty_like(x, dtype=to) for x in grads]
    before = [host(x) for x in grads]
    plan = mt.GradientSet(grads, outs)
    norm = plan.clip(max_norm, inv).item()
    want, clipped = op.grad_clip(before, float(np.float32(max_norm)), float(np.float32(inv)))
    assert abs(norm - want) <= 8 * 2.0 ** -24 * want
    tiny = 2.0 ** -149  # results below the normal numbers: a step of the subnormal ones, bf16's 2^-133
    for o, w in zip(plan.outs, clipped):
        tol = 128 * 2.0 ** -24 * np.abs(w) + HALF[to] * np.abs(w) * 1.001 + (tiny if to == torch.float32 else 2.0 ** -133)
        assert (np.abs(host(o) - w) <= tol).all(), (np.abs(host(o) - w) / np.maximum(np.abs(w), 1e-300)).max()
    plan.check()


def test_a_stream_of_another_device_is_refused():
    x = torch.randn(4, 64, device="cuda")
    elsewhere = types.SimpleNamespace(cuda_stream=0x1234, device_index=torch.cuda.current_device() + 1)
    for call in (lambda: mt.quantize_rows(x, stream=elsewhere), lambda: mt.quantize_rows(x, None, None, elsewhere),
                 lambda: mt.GradientSet([x]).clip(1.0, stream=elsewhere)):
        with pytest.raises(ValueError, match="stream"):
            call()


@pytest.mark.parametrize("kind", ["default", "external", "priority"])
def test_streams_of_every_kind(kind):
    # the default stream while another is current, one made elsewhere, one of high priority
    x = torch.randn(300, 512, device="cuda")
    w, ws = mt.quantize_rows(torch.randn(64, 512, device="cuda"))
    want = mt.linear_i8(x, w, ws)
    raw = torch.cuda.Stream()
    stream = {"default": torch.cuda.default_stream(), "external": torch.cuda.ExternalStream(raw.cuda_stream),
              "priority": torch.cuda.Stream(priority=-1)}[kind]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        now = torch.cuda.current_stream()
        got = mt.linear_i8(x, w, ws, stream=stream)
        norm = mt.GradientSet([x]).norm(stream=stream)
        y = mt.gemm(x.bfloat16(), x[:64].bfloat16(), stream=stream) if kind == "default" else None
        assert torch.cuda.current_stream() == now
        with pytest.raises(ValueError):
            mt.linear_i8(x, w, ws, out_dtype=torch.int8, stream=stream)  # refused: the stream is put back
        assert torch.cuda.current_stream() == now
    torch.cuda.synchronize()
    assert torch.equal(got, want) and abs(norm.item() - x.double().norm().item()) <= 1e-5 * norm.item()
    assert y is None or y.shape == (300, 64)
