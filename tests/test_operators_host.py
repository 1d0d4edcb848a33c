"""The operators' entry points on the CPU: struct layouts, workspace sizes, and
every refusal before any device work (stand-in addresses are never read)."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import generative_recommendation_ranking_b200 as mt
from generative_recommendation_ranking_b200 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CAPACITY = _lib.MTGR_ERR_INVALID_ARG, _lib.MTGR_ERR_UNSUPPORTED, _lib.MTGR_ERR_CAPACITY
F = 0x100000  # an aligned stand-in address
F32, BF16, F16, I8 = _lib.MTGR_F32, _lib.MTGR_BF16, _lib.MTGR_F16, _lib.MTGR_I8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from generative_recommendation_ranking_b200 import build
        build.build()
    return _lib.load()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (("mtgr_boundary_params", _lib.MtgrBoundaryParams), ("mtgr_boundary_grads", _lib.MtgrBoundaryGrads),
               ("mtgr_grad_tensor", _lib.MtgrGradTensor))
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mtgr.h"', "int main(void) {"]
    for c, cls in structs:
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = dict(l.split() for l in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for c, cls in structs:
        assert int(got[c]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(cls, f).offset, f


def params(**kw):
    p = dict(d=512, G=4, eps=1e-5, gate=_lib.MTGR_GATE_LINEAR, post_gamma=F, post_beta=F, scale=F, pre_gamma=F, pre_beta=F)
    p.update(kw)
    return _lib.MtgrBoundaryParams(**p)


def fwd(lib, p=None, T=4, gid=F, od=BF16, o=F, ldo=512, u=F, ldu=2048, xd=F32, x=F, h=F, yd=BF16, y=F, ys=F):
    return lib.mtgr_boundary_fwd(ctypes.byref(p if p is not None else params()), T, gid, od, o, ldo, u, ldu, xd, x, h,
                                 yd, y, ys, None)


def test_boundary_forward_refusals(lib):
    assert lib.mtgr_boundary_fwd(None, 0, F, BF16, F, 512, F, 512, F32, F, F, BF16, F, F, None) == INVALID
    for bad in (dict(d=0), dict(d=12), dict(d=8200), dict(G=0), dict(eps=float("nan")), dict(eps=-1.0), dict(gate=3),
                dict(post_beta=None), dict(pre_gamma=None), dict(scale=F + 4)):
        assert fwd(lib, params(**bad)) == INVALID, bad
    assert fwd(lib, params(G=33)) == UNSUPPORTED
    for bad in (dict(T=-1), dict(gid=None), dict(o=None), dict(o=F + 2), dict(ldo=504), dict(ldo=515), dict(u=None),
                dict(ldu=100), dict(x=None), dict(x=F + 8), dict(h=None), dict(y=None), dict(yd=I8, ys=None)):
        assert fwd(lib, **bad) == INVALID, bad
    for bad in (dict(od=I8), dict(od=7), dict(xd=F16), dict(yd=F16), dict(yd=9)):
        assert fwd(lib, **bad) == UNSUPPORTED, bad
    # nothing to do: no rows
    assert fwd(lib, T=0, gid=None, o=None, u=None, x=None, h=None, y=None, ys=None) == _lib.MTGR_OK


def bwd(lib, p=None, T=4, gid=F, od=BF16, o=F, u=F, xd=F32, x=F, dh=F, dyd=BF16, dy=F, do=F, lddo=512, du=F, lddu=512,
        dx=F, grads=None, ws=F, ws_bytes=1 << 30):
    g = grads if grads is not None else _lib.MtgrBoundaryGrads(F, F, F, F, F)
    return lib.mtgr_boundary_bwd(ctypes.byref(p if p is not None else params()), T, gid, od, o, 512, u, 512, xd, x, dh, dyd,
                                 dy, do, lddo, du, lddu, dx, ctypes.byref(g), ws, ws_bytes, None, None)


def test_boundary_backward_refusals(lib):
    for bad in (dict(T=-1), dict(gid=None), dict(o=None), dict(u=None), dict(x=None), dict(dy=None), dict(do=None),
                dict(du=None), dict(dx=None), dict(lddo=8), dict(lddu=516), dict(dh=F + 4), dict(dx=F + 8), dict(ws=None),
                dict(grads=_lib.MtgrBoundaryGrads(F, F, None, F, F)), dict(grads=_lib.MtgrBoundaryGrads(F, F, F, None, F)),
                dict(grads=_lib.MtgrBoundaryGrads(F, None, F, F, F)), dict(grads=_lib.MtgrBoundaryGrads(F, F, F + 4, F, F)),
                dict(p=params(pre_gamma=None, pre_beta=None), dh=None)):
        assert bwd(lib, **bad) == INVALID, bad
    assert bwd(lib, ws_bytes=0) == CAPACITY
    assert bwd(lib, ws_bytes=_lib.mtgr_boundary_bwd_workspace_bytes(4, params()) - 1) == CAPACITY
    assert bwd(lib, dyd=F16) == UNSUPPORTED
    assert bwd(lib, od=I8) == UNSUPPORTED and bwd(lib, xd=F16) == UNSUPPORTED


def test_boundary_workspace(lib):
    # per team (at least four rows each): a word of groups seen, 5 G d sums
    size = lambda T, **kw: _lib.mtgr_boundary_bwd_workspace_bytes(T, params(**kw))  # noqa: E731
    assert size(1) == 256 + 4 * 5 * 512 * 4
    assert size(0) == 0 and size(-1) == 0 and size(8, d=12) == 0 and size(8, G=40) == 0
    assert size(1 << 30) <= (256 << 20) + (1 << 16) and size(1 << 30, G=32, d=8192) <= (256 << 20) + (1 << 16)


def test_quantize_refusals(lib):
    q = lambda M=4, K=64, xd=BF16, x=F, ld=64, qq=F, s=F: lib.mtgr_quantize_rows(M, K, xd, x, ld, qq, s, None)  # noqa: E731
    for bad in (dict(M=-1), dict(K=0), dict(ld=56), dict(ld=65), dict(x=None), dict(x=F + 2), dict(qq=None), dict(qq=F + 8),
                dict(s=None)):
        assert q(**bad) == INVALID, bad
    for bad in (dict(K=60), dict(K=32776, ld=32776), dict(xd=I8)):
        assert q(**bad) == UNSUPPORTED, bad
    assert q(M=0, x=None, qq=None, s=None) == _lib.MTGR_OK


def test_int8_product_refusals(lib):
    def gemm(M=8, N=64, K=64, a=F, sa=F, b=F, sb=F, bias=F, epi=0, resid=None, q_cols=0, od=BF16, out=F):
        return lib.mtgr_gemm_i8(M, N, K, a, sa, b, sb, bias, epi, resid, q_cols, od, out, None, None)

    def linear(M=100, N=64, K=64, xd=BF16, x=F, ld=64, b=F, sb=F, bias=F, epi=0, resid=None, q_cols=0, od=BF16, out=F, ws=F,
               ws_bytes=1 << 20):
        return lib.mtgr_linear_i8(M, N, K, xd, x, ld, b, sb, bias, epi, resid, q_cols, od, out, ws, ws_bytes, None, None)

    for f in (gemm, linear):
        for bad in (dict(M=-1), dict(N=-8), dict(K=0), dict(q_cols=-32), dict(q_cols=8), dict(epi=5), dict(b=None),
                    dict(sb=None), dict(out=None), dict(b=F + 8), dict(sb=F + 4), dict(bias=F + 4), dict(out=F + 8),
                    dict(epi=_lib.MTGR_EPI_RESID, od=F32), dict(epi=_lib.MTGR_EPI_RESID, resid=F),
                    dict(epi=_lib.MTGR_EPI_RESID, resid=F + 4, od=F32), dict(epi=_lib.MTGR_EPI_RESID, resid=F, od=F32)):
            assert f(**bad) == INVALID, (f.__name__, bad)
        assert f(M=(1 << 30) + 1) == UNSUPPORTED and f(N=(1 << 30) + 8) == UNSUPPORTED
        assert f(N=60) == UNSUPPORTED and f(od=I8) == UNSUPPORTED
    assert gemm(K=72) == UNSUPPORTED and linear(K=72, ld=72) == UNSUPPORTED
    assert gemm(K=131072) == UNSUPPORTED and linear(K=32784, ld=32784) == UNSUPPORTED
    assert gemm(a=None) == INVALID and gemm(sa=None) == INVALID and gemm(a=F + 4) == INVALID
    assert linear(x=None) == INVALID and linear(ld=8) == INVALID and linear(xd=I8) == UNSUPPORTED
    assert linear(ws=None) == INVALID and linear(ws_bytes=100) == CAPACITY
    size = _lib.mtgr_linear_i8_workspace_bytes
    assert size(100, 64, 48) == 4864 + 512 and size(100, 64, 4096) == 409600 + 512
    # few rows and columns are quantised within the product
    assert size(16, 16, 512) == 0 and size(17, 16, 512) > 0 and size(16, 1 << 20, 512) > 0 and size(16, 16, 32768) > 0
    assert size(-1, 8, 48) == 0 and size(5, -8, 48) == 0 and size(5, 8, 0) == 0
    assert size(1 << 20, 64, 8192) == (1 << 33) + (1 << 22)


def test_grad_clip_refusals(lib):
    def clip(*t, max_norm=1.0, inv=1.0, norm=F, ws=F, ws_bytes=1 << 20, status=F, n=None):
        arr = (_lib.MtgrGradTensor * max(1, len(t)))(*t)
        return lib.mtgr_grad_clip(arr, len(t) if n is None else n, max_norm, inv, norm, ws, ws_bytes, status, None)

    G = _lib.MtgrGradTensor
    ok = G(F, F, 100, F32, F32)
    assert clip(ok, n=-1) == INVALID
    assert lib.mtgr_grad_clip(None, 1, 1.0, 1.0, F, F, 1 << 20, F, None) == INVALID
    for t in (G(None, F, 100, F32, F32), G(F, F, -1, F32, F32), G(F, F, 1 << 39, F32, F32), G(F + 2, F, 100, F32, F32),
              G(F, F + 1, 100, BF16, BF16), G(F, F, 100, BF16, F32)):
        assert clip(t) == INVALID, (t.g, t.n)
    assert clip(G(F, F, 100, I8, I8)) == UNSUPPORTED and clip(G(F, F, 100, F32, BF16)) == UNSUPPORTED
    assert clip(ok, G(F, None, 5, F32, F32)) == INVALID  # outputs for all tensors or none
    assert clip(G(None, None, 0, F32, F32), ok, G(F, None, 5, F32, F32)) == INVALID  # empty ones aside
    assert clip(G(None, F, 0, F32, F32), G(F, None, 5, F32, F32), G(F, F, 5, F32, F32)) == INVALID
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(inv=0.0), dict(inv=float("inf")),
                dict(inv=float("nan")), dict(norm=None), dict(status=None), dict(ws=None)):
        assert clip(ok, **bad) == INVALID, bad
    assert clip(ok, ws_bytes=0) == CAPACITY
    assert _lib.mtgr_grad_clip_workspace_bytes((G * 1)(G(None, F, 5, F32, F32)), 1) == 0
    assert _lib.mtgr_grad_clip_workspace_bytes((G * 1)(ok), 1) >= 512


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64)
    gid = torch.zeros(4, dtype=torch.int8)
    for call in (lambda: mt.boundary_forward(x, x, x, gid), lambda: mt.quantize_rows(x),
                 lambda: mt.linear_i8(x, x.to(torch.int8), x[:, 0]), lambda: mt.GradientSet([x]),
                 lambda: mt.GradientSet([]), lambda: mt.GradientSet([x], [])):
        with pytest.raises(ValueError):
            call()
