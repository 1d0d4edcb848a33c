"""The block-boundary, int8 and gradient-clipping operators over libmtgr.so.

Each function checks shapes, types and places of its tensors, allocates the
outputs that are not given (and the workspace), and makes one call into the C
ABI on ``stream`` (default: the device's current stream). What it allocates is
tied to ``stream``, so it may be dropped while the work still runs.
"""

from __future__ import annotations

import torch

from . import _lib
from ._lib import (MTGR_EPI_NONE, MTGR_EPI_RESID, MTGR_GATE_LINEAR, MTGR_GATE_NONE, MTGR_GATE_SILU,
                   MtgrBoundaryGrads, MtgrBoundaryParams, MtgrGradTensor)
from .api import EPS

GATES = {None: MTGR_GATE_NONE, "none": MTGR_GATE_NONE, "linear": MTGR_GATE_LINEAR,
         "silu": MTGR_GATE_SILU}
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_STREAM_TYPES = (torch.float32, torch.bfloat16)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class _On:
    """The device of a call's tensors, made the current one for the call (the
    library works on the current device), and its stream."""

    __slots__ = ("index", "guard", "stream", "other")

    def __init__(self, t: torch.Tensor, stream):
        _need(t.is_cuda, "a device tensor is needed")
        self.index = t.device.index
        self.guard = None if self.index == torch.cuda.current_device() else torch.cuda.device(self.index)
        current = torch.cuda.current_stream(self.index)
        self.stream = current if stream is None else stream
        self.other = stream is not None and stream != current

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)

    def empty(self, shape, dtype) -> torch.Tensor:
        t = torch.empty(shape, dtype=dtype, device=self.index)
        if self.other:
            t.record_stream(self.stream)
        return t

    def bytes(self, n: int) -> torch.Tensor:
        return self.empty(max(int(n), 256), torch.uint8)

    def given(self, name, t, shape, dtypes, rows=False) -> None:
        """Checks one tensor; ``rows``: rows may be further apart than their length."""
        if t.shape != shape or t.dtype not in dtypes or t.device.index != self.index or not t.is_cuda:
            raise ValueError(f"{name}: {tuple(shape)} of {' / '.join(map(str, dtypes))} on cuda:{self.index} "
                             f"is needed, got {tuple(t.shape)} of {t.dtype} on {t.device}")
        if rows:
            if t.shape[0] and (t.stride(1) != 1 and t.shape[1] > 1 or t.shape[0] > 1 and
                               (t.stride(0) < t.shape[1] or t.stride(0) % 8)):
                raise ValueError(f"{name}: rows of consecutive values, a multiple of 8 apart, are needed")
        elif not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous tensor is needed")


_F32 = (torch.float32,)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """``t`` with a row stride that the library accepts: that of a single row means nothing."""
    if t.shape[0] <= 1 and (t.stride(0) < t.shape[1] or t.stride(0) % 8):
        return t.as_strided(t.shape, (t.shape[1], 1))
    return t


def _boundary(on, x, o, u, group_id, post_gamma, post_beta, scale, pre_gamma, pre_beta, eps, gate):
    """Checks what the forward and the backward share; returns the parameters and u."""
    _need(gate in GATES, f"gate {gate!r}: one of none, linear, silu")
    _need(x.dim() == 2, "x: [T, d] is needed")
    shape = x.shape
    T, d = shape
    on.given("x", x, shape, _STREAM_TYPES)
    on.given("o", o, shape, _FLOATS, rows=True)
    on.given("group_id", group_id, (T,), (torch.int8,))
    code = GATES[gate]
    if code == MTGR_GATE_NONE:
        u = None
    else:
        _need(u is not None, "u is needed with a gate")
        on.given("u", u, shape, (o.dtype,), rows=True)
        u = _rows(u)
    _need((post_gamma is None) == (post_beta is None), "post_gamma and post_beta come together")
    _need((pre_gamma is None) == (pre_beta is None), "pre_gamma and pre_beta come together")
    G = next((p.shape[0] for p in (post_gamma, pre_gamma, scale) if p is not None), 1)
    ptr = [None] * 5
    for i, (name, p) in enumerate((("post_gamma", post_gamma), ("post_beta", post_beta), ("scale", scale),
                                   ("pre_gamma", pre_gamma), ("pre_beta", pre_beta))):
        if p is not None:
            on.given(name, p, (G, d), _F32)
            ptr[i] = p.data_ptr()
    return MtgrBoundaryParams(d, G, eps, code, *ptr), _rows(o), u


def boundary_forward(x, o, u, group_id, post_gamma=None, post_beta=None, scale=None, pre_gamma=None,
                     pre_beta=None, *, gate="linear", y_dtype=torch.bfloat16, eps: float = EPS, h=None,
                     y=None, y_scale=None, stream=None):
    """The boundary between two blocks (mtgr_boundary_fwd): the branch output ``o``
    [T, d] normalised by group (post_gamma, post_beta), gated by ``u``, scaled and
    added to the residual stream ``x`` [T, d], and the next block's GroupLN
    (pre_gamma, pre_beta) of the sum:

        h = x + scale_g GLN(o) f(u),    y = GLN(h)

    Parameters are float32 [G, d]; each norm and the scale may be None. ``gate``:
    "none" (u None), "linear" (f(u) = u) or "silu". ``o`` and ``u`` share a type
    and may be columns of wider rows. ``y_dtype``: float32, bfloat16 or int8 (rows
    with a scale, for gemm_i8). Returns (h, y, y_scale); y is None without the
    pre norm, y_scale but for int8. ``h`` may be given as ``x``: in place.
    """
    with _On(x, stream) as on:
        p, o, u = _boundary(on, x, o, u, group_id, post_gamma, post_beta, scale, pre_gamma, pre_beta, eps, gate)
        T, d = x.shape
        if h is None:
            h = on.empty(x.shape, x.dtype)
        else:
            on.given("h", h, x.shape, (x.dtype,))
        if pre_gamma is None:
            y = y_scale = None
        else:
            _need(y_dtype in (torch.float32, torch.bfloat16, torch.int8),
                  f"y_dtype {y_dtype}: float32, bfloat16 or int8")
            if y is None:
                y = on.empty(x.shape, y_dtype)
            else:
                on.given("y", y, x.shape, (y_dtype,))
            if y_dtype != torch.int8:
                y_scale = None
            elif y_scale is None:
                y_scale = on.empty((T,), torch.float32)
            else:
                on.given("y_scale", y_scale, (T,), _F32)
        _lib.mtgr_boundary_fwd(p, T, group_id, o, u, x, h, y, y_scale, on.stream)
    return h, y, y_scale


def boundary_backward(x, o, u, group_id, post_gamma=None, post_beta=None, scale=None, pre_gamma=None,
                      pre_beta=None, dh=None, dy=None, *, gate="linear", eps: float = EPS, ws=None,
                      status=None, stream=None) -> dict:
    """Gradients of boundary_forward (mtgr_boundary_bwd) from ``dh`` = dL/dh
    through the stream (None: 0; [T, d] of x's type) and ``dy`` = dL/dy ([T, d],
    float32 or bfloat16; None without the pre norm). Returns a dict: ``dx``,
    ``do``, ``du`` (with a gate) in the types of x, o, u, and the float32
    gradients of the parameters that were given, under their names.
    """
    with _On(x, stream) as on:
        p, o, u = _boundary(on, x, o, u, group_id, post_gamma, post_beta, scale, pre_gamma, pre_beta, eps, gate)
        T, d = x.shape
        if dh is not None:
            on.given("dh", dh, x.shape, (x.dtype,))
        if pre_gamma is not None:
            _need(dy is not None, "dy is needed with the pre norm")
            on.given("dy", dy, x.shape, _STREAM_TYPES)
        else:
            _need(dh is not None and dy is None, "without the pre norm dh is needed, and no dy")
        out = dict(dx=on.empty(x.shape, x.dtype), do=on.empty(x.shape, o.dtype))
        if u is not None:
            out["du"] = on.empty(x.shape, o.dtype)
        # one allocation for the parameters' gradients
        names = [n for n, t in (("post_gamma", post_gamma), ("post_beta", post_beta), ("scale", scale),
                                ("pre_gamma", pre_gamma), ("pre_beta", pre_beta)) if t is not None]
        flat = on.empty((len(names), p.G, d), torch.float32)
        out.update(zip(names, flat.unbind(0)))
        g = MtgrBoundaryGrads(*[out[n].data_ptr() if n in out else None
                                for n in ("post_gamma", "post_beta", "scale", "pre_gamma", "pre_beta")])
        need = _lib.mtgr_boundary_bwd_workspace_bytes(T, p)
        if ws is None or ws.numel() < need:
            ws = on.bytes(need)
        _lib.mtgr_boundary_bwd(p, T, group_id, o, u, x, dh, dy, out["do"], out.get("du"), out["dx"], g, ws,
                               status, on.stream)
    return out


def quantize_rows(x, q=None, scale=None, stream=None):
    """Rows of ``x`` [M, K] (float32, bfloat16, float16) to signed bytes with a
    float32 scale each (mtgr_quantize_rows): returns (q [M, K] int8, scale [M]).
    A weight's rows give the scales of its output channels."""
    with _On(x, stream) as on:
        _need(x.dim() == 2, "x: [M, K] is needed")
        on.given("x", x, x.shape, _FLOATS, rows=True)
        if q is None:
            q = on.empty(x.shape, torch.int8)
        else:
            on.given("q", q, x.shape, (torch.int8,))
        if scale is None:
            scale = on.empty(x.shape[:1], torch.float32)
        else:
            on.given("scale", scale, x.shape[:1], _F32)
        _lib.mtgr_quantize_rows(_rows(x), q, scale, on.stream)
    return q, scale


def linear_i8(x, w, w_scale, x_scale=None, bias=None, epi: int = MTGR_EPI_NONE, resid=None, q_cols: int = 0,
              out_dtype=torch.float32, out=None, ws=None, status=None, stream=None) -> torch.Tensor:
    """Linear layer with int8 weights ``w`` [N, K] and a scale per output channel
    ``w_scale`` [N]: out = epi(x w^T + bias) [M, N]. ``x`` [M, K] is float32,
    bfloat16 or float16, quantised by row on the way (mtgr_linear_i8), or int8
    with its rows' scales ``x_scale`` [M] (mtgr_gemm_i8). Epilogues, ``resid``
    [M, N] float32 and ``q_cols`` as in gemm. ``status``: a device int32 word
    (zeroed by the caller) for errors the device finds: an f16 value out of
    range, a wait that ran out; without it they go unseen."""
    with _On(x, stream) as on:
        _need(x.dim() == 2 and w.dim() == 2, "x: [M, K] and w: [N, K] are needed")
        M, K = x.shape
        N = w.shape[0]
        on.given("w", w, (N, K), (torch.int8,))
        on.given("w_scale", w_scale, (N,), _F32)
        if bias is not None:
            on.given("bias", bias, (N,), _F32)
        if epi == MTGR_EPI_RESID:
            _need(resid is not None, "resid is needed with MTGR_EPI_RESID")
            on.given("resid", resid, (M, N), _F32)
        else:
            _need(resid is None, "resid goes with MTGR_EPI_RESID")
        if out is None:
            out = on.empty((M, N), out_dtype)
        else:
            on.given("out", out, (M, N), (out_dtype,))
        if x.dtype == torch.int8:
            on.given("x", x, (M, K), (torch.int8,))
            _need(x_scale is not None, "x_scale is needed with int8 rows")
            on.given("x_scale", x_scale, (M,), _F32)
            _lib.mtgr_gemm_i8(x, x_scale, w, w_scale, bias, epi, resid, q_cols, out, status, on.stream)
            return out
        _need(x_scale is None, "x_scale goes with int8 rows")
        on.given("x", x, (M, K), _FLOATS, rows=True)
        need = _lib.mtgr_linear_i8_workspace_bytes(M, K)
        if ws is None or ws.numel() < need:
            ws = on.bytes(need)
        _lib.mtgr_linear_i8(_rows(x), w, w_scale, bias, epi, resid, q_cols, out, ws, status, on.stream)
    return out


def gemm_i8(a, a_scale, b, b_scale, bias=None, epi: int = MTGR_EPI_NONE, resid=None, q_cols: int = 0,
            out_dtype=torch.float32, out=None, status=None, stream=None) -> torch.Tensor:
    """out = epi(a_scale b_scale a b^T + bias) of int8 ``a`` [M, K] and ``b`` [N, K]
    with a scale per row of each (mtgr_gemm_i8)."""
    _need(a.dtype == torch.int8, "a: int8 rows are needed")
    return linear_i8(a, b, b_scale, a_scale, bias, epi, resid, q_cols, out_dtype, out, None, status, stream)


class GradientSet:
    """A set of gradient tensors whose global norm is clipped in one call
    (mtgr_grad_clip), kept by a training program from step to step.

    ``grads``: device tensors (float32, bfloat16, float16), e.g. what
    hstu_block_backward and boundary_backward return; contiguous, of any size.
    ``outs``: where the clipped values go, tensor by tensor (the gradient's
    type or float32); None: in place. The tensors' memory is read at every
    call, so a step writes new gradients into the same buffers.
    """

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        _need(len(self.grads) == len(self.outs), "one output per gradient is needed")
        _need(len(self.grads) > 0, "at least one gradient is needed")
        self.device = self.grads[0].device
        spans = []
        n = len(self.grads)
        self.c = (MtgrGradTensor * n)()
        with _On(self.grads[0], None) as on:
            for i, (g, o) in enumerate(zip(self.grads, self.outs)):
                on.given(f"grads[{i}]", g, g.shape, _FLOATS)
                on.given(f"outs[{i}]", o, g.shape, (g.dtype, torch.float32))
                self.c[i] = MtgrGradTensor(g.data_ptr(), o.data_ptr(), g.numel(), _lib.dtype_code(g.dtype),
                                           _lib.dtype_code(o.dtype))
                if g.numel():
                    spans.append((o.data_ptr(), o.data_ptr() + o.numel() * o.element_size(), i, 1))
                    if o.data_ptr() != g.data_ptr() or o.dtype != g.dtype:
                        spans.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), i, 0))
            # no two outputs may share memory, nor an output and another gradient
            spans.sort()
            end_out = end_any = 0
            for lo, hi, i, is_out in spans:
                _need(lo >= (end_any if is_out else end_out), f"tensor {i} shares memory with another one")
                end_any = max(end_any, hi)
                if is_out:
                    end_out = max(end_out, hi)
            # the norm alone
            self.c_norm = (MtgrGradTensor * n)(*[MtgrGradTensor(c.g, None, c.n, c.dtype, c.dtype) for c in self.c])
            self.ws_bytes = _lib.mtgr_grad_clip_workspace_bytes(self.c, n)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _run(self, table, max_norm, inv_scale, norm, status, stream):
        with _On(self.grads[0], stream) as on:
            if norm is None:
                norm = on.empty((1,), torch.float32)
            else:
                on.given("norm", norm, (1,), _F32)
            _lib.mtgr_grad_clip(table, len(self.grads), max_norm, inv_scale, norm, on.bytes(self.ws_bytes),
                                self.status if status is None else status, on.stream)
        return norm

    def clip(self, max_norm: float, inv_scale: float = 1.0, norm=None, status=None, stream=None) -> torch.Tensor:
        """Clips to ``max_norm`` after taking the loss scale out (``inv_scale`` = 1 /
        loss scale). Returns the norm before clipping ([1] float32 on the
        device). A norm that is not finite leaves the outputs as they were and
        MTGR_ERR_RANGE in ``status`` (default: the set's own word, see check)."""
        return self._run(self.c, max_norm, inv_scale, norm, status, stream)

    def norm(self, inv_scale: float = 1.0, norm=None, status=None, stream=None) -> torch.Tensor:
        """The norm alone; nothing is written but it."""
        return self._run(self.c_norm, float("inf"), inv_scale, norm, status, stream)

    def check(self) -> None:
        """Synchronise and raise if a call on this set met a norm that is not
        finite; the word is then cleared for the next step."""
        torch.cuda.synchronize(self.device)
        st = int(self.status.item())
        if st != 0:
            self.status.zero_()
            raise _lib.MTGRError("device status", st)
