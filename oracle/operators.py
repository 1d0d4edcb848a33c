"""Float64 oracle of the block-boundary, int8 and gradient-clipping operators.
TEST INFRASTRUCTURE ONLY (see the package docstring for who may import it).

Boundary between two blocks (GroupLN as in ``mtgr.group_layernorm``: fun-rec 7.3.3,
the GLN formula; gate and residual: summary page, Method, the update equations):

  n = GLN(o; post);  h = x + scale_g n f(u);  y = GLN(h; pre)

its backward by the chain rule; rows quantised to signed bytes; the product of
such rows; the global gradient norm with clipping.
"""

from __future__ import annotations

import numpy as np
from scipy.special import expit

from .mtgr import EPS

QUANT_TINY = 2.0 ** -100
CLIP_EPS = 1e-6


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def _norm(v, eps):
    c = v - v.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c * rstd, rstd


def gate(u, kind):
    """(f(u), f'(u)) of the gate ``kind``; u None for "none"."""
    if kind == "none":
        return 1.0, 0.0
    if kind == "linear":
        return u, np.ones_like(u)
    s = expit(u)
    return u * s, s * (1.0 + u * (1.0 - s))


def boundary_forward(x, o, u, gid, post_gamma=None, post_beta=None, scale=None, pre_gamma=None, pre_beta=None,
                     kind="linear", eps=EPS):
    """(h, y); y None without the pre norm."""
    x, o, u = _f64(x), _f64(o), _f64(u)
    n = o
    if post_gamma is not None:
        n = _norm(o, eps)[0] * _f64(post_gamma)[gid] + _f64(post_beta)[gid]
    h = x + (1.0 if scale is None else _f64(scale)[gid]) * n * gate(u, kind)[0]
    if pre_gamma is None:
        return h, None
    return h, _norm(h, eps)[0] * _f64(pre_gamma)[gid] + _f64(pre_beta)[gid]


def boundary_backward(x, o, u, gid, post_gamma=None, post_beta=None, scale=None, pre_gamma=None, pre_beta=None,
                      dh=None, dy=None, kind="linear", eps=EPS):
    """dict of dx, do, du and the parameters' gradients [G, d]."""
    x, o, u = _f64(x), _f64(o), _f64(u)
    G = next((np.shape(p)[0] for p in (post_gamma, pre_gamma, scale) if p is not None), 1)

    def by_group(v):
        return np.stack([v[np.asarray(gid) == g].sum(0) for g in range(G)])

    def norm_back(dv, vhat, rstd):
        return rstd * (dv - dv.mean(1, keepdims=True) - vhat * (dv * vhat).mean(1, keepdims=True))

    out = {}
    n = o
    if post_gamma is not None:
        ohat, rstd_o = _norm(o, eps)
        n = ohat * _f64(post_gamma)[gid] + _f64(post_beta)[gid]
    f, df = gate(u, kind)
    s = 1.0 if scale is None else _f64(scale)[gid]
    H = np.zeros_like(x) if dh is None else _f64(dh).copy()
    if pre_gamma is not None:
        hhat, rstd_h = _norm(x + s * n * f, eps)
        dy = _f64(dy)
        out["pre_gamma"], out["pre_beta"] = by_group(dy * hhat), by_group(dy)
        H += norm_back(dy * _f64(pre_gamma)[gid], hhat, rstd_h)
    out["dx"] = H
    if scale is not None:
        out["scale"] = by_group(H * n * f)
    dn = H * s * f
    if kind != "none":
        out["du"] = H * s * n * df
    if post_gamma is not None:
        out["post_gamma"], out["post_beta"] = by_group(dn * ohat), by_group(dn)
        out["do"] = norm_back(dn * _f64(post_gamma)[gid], ohat, rstd_o)
    else:
        out["do"] = dn
    return out


def quantize_rows(x):
    """(q int8, scale float32): the scale is an fp32 product with 1 / 127 in fp32,
    the quotient is exact."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(x).max(1) if x.shape[1] else np.zeros(len(x), np.float32)
        scale = (np.maximum(top, np.float32(QUANT_TINY)) * (np.float32(1) / np.float32(127))).astype(np.float32)
        bad = ~np.isfinite(x).all(1)
        scale[bad] = np.nan
        # longdouble has 64 bits of fraction: the quotient of two fp32 numbers is
        # told from a border k + 1/2 that it does not equal
        q = np.rint(x.astype(np.longdouble) / scale.astype(np.longdouble)[:, None])
    q = np.where(bad[:, None], 0, q)
    return q.astype(np.int8), scale


def gemm_i8(a, sa, b, sb, bias=None, epi="none", resid=None, q_cols=0):
    acc = np.asarray(a, np.int64) @ np.asarray(b, np.int64).T
    v = acc * _f64(sa)[:, None] * _f64(sb)[None, :]
    if bias is not None:
        v = v + _f64(bias)
    if epi == "silu":
        v = v * expit(v)
    elif epi == "resid":
        v = v + _f64(resid)
    v[:, :q_cols] *= 0.5
    return v


def grad_clip(grads, max_norm, inv_scale=1.0):
    """(norm, clipped gradients); a norm that is not finite gives None for them."""
    with np.errstate(over="ignore", invalid="ignore"):
        norm = inv_scale * np.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
    if not np.isfinite(norm):
        return norm, None
    c = inv_scale * min(1.0, max_norm / (norm + CLIP_EPS))
    return norm, [_f64(g) * c for g in grads]
