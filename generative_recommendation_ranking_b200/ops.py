"""The block-boundary, int8 and gradient-clipping operators over libmtgr.so.

Each function checks shapes, types and places of its tensors, allocates the
outputs that are not given (and the workspace), and makes one call into the C
ABI on ``stream`` (default: the device's current stream). What it allocates is
``stream``'s own memory, so nothing that still runs on another stream uses it, and
it may be dropped while the work runs on ``stream`` or its results are read on the
current stream. The order between the two streams is the caller's: inputs ready for
``stream`` before the call and kept until it has run, results read behind it. Outputs
and workspaces that are given overlap no input, but where a docstring says so.
"""

from __future__ import annotations

import functools
import inspect
from ctypes import byref as _byref

import torch

from . import _lib
from ._lib import (MTGR_EPI_NONE, MTGR_EPI_RESID, MTGR_GATE_LINEAR, MTGR_GATE_NONE, MTGR_GATE_SILU,
                   MtgrBoundaryGrads, MtgrBoundaryParams, MtgrGradTensor)
from .api import EPS

GATES = {None: MTGR_GATE_NONE, "none": MTGR_GATE_NONE, "linear": MTGR_GATE_LINEAR,
         "silu": MTGR_GATE_SILU}
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_STREAM_TYPES = (torch.float32, torch.bfloat16)


_device_now = torch._C._cuda_getDevice
_stream_now = torch._C._cuda_getCurrentRawStream
_set_stream = torch._C._cuda_setStream  # torch.cuda.stream takes about 10 us a use, this 1
_DENSE = torch.contiguous_format


def _in_its_place(fn):
    """Runs ``fn`` with its first tensor's device as the current one (the library works
    on the current device), and its argument ``stream`` as the current stream: what it
    allocates is then that stream's memory (the caller's may be a buffer that was dropped
    while work there still runs). Its results are kept from being handed out again before
    the caller's stream, where their reader is, has got past their release."""

    names = list(inspect.signature(fn).parameters)
    first, at = names[0], names.index("stream")

    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else kwargs.get(first)
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{first}: a device tensor is needed")
        dev = t.get_device()
        if dev != _device_now():
            with torch.cuda.device(dev):
                return call(*args, **kwargs)
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None or stream.cuda_stream == _stream_now(dev):
            return fn(*args, **kwargs)
        if stream.device_index != dev:
            raise ValueError(f"stream: one of cuda:{dev} is needed, got {stream}")
        now = torch.cuda.current_stream(dev)
        _set_stream(stream_id=stream.stream_id, device_index=dev, device_type=stream.device_type)
        try:
            out = fn(*args, **kwargs)
        finally:
            _set_stream(stream_id=now.stream_id, device_index=dev, device_type=now.device_type)
        for v in (out,) if isinstance(out, torch.Tensor) else out.values() if isinstance(out, dict) else out:
            if v is not None:
                v.record_stream(now)
        return out

    return call


def _new(like, shape=None, dtype=None) -> torch.Tensor:
    """A buffer beside ``like``, of its shape and type unless given, on the current
    stream. (An existing tensor's allocation is called twice as fast as torch.empty.)"""
    if shape is None:
        return torch.empty_like(like, memory_format=_DENSE) if dtype is None else \
            torch.empty_like(like, dtype=dtype, memory_format=_DENSE)
    return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)


def _given(name: str, t, shape, dtype, dev: int) -> None:
    if not (t.shape == shape and t.dtype == dtype and t.get_device() == dev and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {tuple(shape)} of {dtype} on cuda:{dev} is needed, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}, strides {t.stride()}")


def _given_ws(ws, need: int, dev: int) -> int:
    """Bytes of a workspace that the caller gave; 0 if it is too small, or none."""
    if ws is None:
        return 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: contiguous memory on cuda:{dev} is needed, got {tuple(ws.shape)} of {ws.dtype} on "
                         f"{ws.device}, strides {ws.stride()}")
    room = ws.numel() * ws.element_size()
    return room if room >= need else 0


def _given_rows(name: str, t, shape, dtypes, dev: int) -> int:
    """Checks a tensor whose rows may be further apart than their length; returns
    how far (that of a single row means nothing)."""
    if t.shape == shape and t.dtype in dtypes and t.get_device() == dev:
        ld, one = t.stride()
        rows, n = shape
        if rows <= 1:
            ld = n
        if (one == 1 or n <= 1 or rows == 0) and ld >= n and ld % 8 == 0:
            return ld
    raise ValueError(f"{name}: {tuple(shape)} of {' / '.join(map(str, dtypes))} on cuda:{dev}, rows of consecutive "
                     f"values a multiple of 8 apart, is needed, got {tuple(t.shape)} of {t.dtype} on {t.device}, "
                     f"strides {t.stride()}")


_PARAMS = ("post_gamma", "post_beta", "scale", "pre_gamma", "pre_beta")
_CODE = {torch.float32: _lib.MTGR_F32, torch.bfloat16: _lib.MTGR_BF16, torch.float16: _lib.MTGR_F16,
         torch.int8: _lib.MTGR_I8}


def _boundary(x, o, u, group_id, values, eps, gate, dev):
    """Checks what the forward and the backward share: (parameters, row strides of o and u)."""
    if gate not in GATES:
        raise ValueError(f"gate {gate!r}: one of none, linear, silu")
    if x.dim() != 2 or x.dtype not in _STREAM_TYPES or not x.is_contiguous():
        raise ValueError(f"x: a contiguous [T, d] of float32 or bfloat16 is needed, got {tuple(x.shape)} of {x.dtype}")
    shape = x.shape
    T, d = shape
    ld_o = _given_rows("o", o, shape, _FLOATS, dev)
    _given("group_id", group_id, shape[:1], torch.int8, dev)
    code = GATES[gate]
    ld_u = 0
    if code != MTGR_GATE_NONE:
        if u is None:
            raise ValueError("u is needed with a gate")
        ld_u = _given_rows("u", u, shape, (o.dtype,), dev)
    if (values[0] is None) != (values[1] is None) or (values[3] is None) != (values[4] is None):
        raise ValueError("a norm's gamma and beta come together")
    G = 1
    for p in values:
        if p is not None:
            G = p.shape[0]
            break
    ptr = []
    for name, p in zip(_PARAMS, values):
        if p is None:
            ptr.append(None)
        else:
            _given(name, p, (G, d), torch.float32, dev)
            ptr.append(p.data_ptr())
    return MtgrBoundaryParams(d, G, eps, code, *ptr), ld_o, ld_u


@_in_its_place
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
    dev = x.get_device()
    raw = _stream_now(dev)
    p, ld_o, ld_u = _boundary(x, o, u, group_id, (post_gamma, post_beta, scale, pre_gamma, pre_beta), eps, gate, dev)
    shape = x.shape
    if h is None:
        h = _new(x)
    else:
        _given("h", h, shape, x.dtype, dev)
    if pre_gamma is None:
        y = y_scale = None
    else:
        if y_dtype not in (torch.float32, torch.bfloat16, torch.int8):
            raise ValueError(f"y_dtype {y_dtype}: float32, bfloat16 or int8")
        if y is None:
            y = _new(x, dtype=y_dtype)
        else:
            _given("y", y, shape, y_dtype, dev)
        if y_dtype != torch.int8:
            y_scale = None
        elif y_scale is None:
            y_scale = _new(pre_gamma, shape[0])
        else:
            _given("y_scale", y_scale, shape[:1], torch.float32, dev)
    _lib.check("mtgr_boundary_fwd", _lib.load().mtgr_boundary_fwd(
        _byref(p), shape[0], group_id.data_ptr(), _CODE[o.dtype], o.data_ptr(), ld_o, u.data_ptr() if ld_u else None,
        ld_u, _CODE[x.dtype], x.data_ptr(), h.data_ptr(), 0 if y is None else _CODE[y_dtype],
        None if y is None else y.data_ptr(), None if y_scale is None else y_scale.data_ptr(), raw))
    return h, y, y_scale


@_in_its_place
def boundary_backward(x, o, u, group_id, post_gamma=None, post_beta=None, scale=None, pre_gamma=None,
                      pre_beta=None, dh=None, dy=None, *, gate="linear", eps: float = EPS, ws=None,
                      status=None, stream=None) -> dict:
    """Gradients of boundary_forward (mtgr_boundary_bwd) from ``dh`` = dL/dh
    through the stream (None: 0; [T, d] of x's type) and ``dy`` = dL/dy ([T, d],
    float32 or bfloat16; None without the pre norm). Returns a dict: ``dx``,
    ``do``, ``du`` (with a gate) in the types of x, o, u, and the float32
    gradients of the parameters that were given, under their names. ``status``: a
    device int32 word (zeroed by the caller) that tells of f16 gradients out of range.
    """
    dev = x.get_device()
    raw = _stream_now(dev)
    values = (post_gamma, post_beta, scale, pre_gamma, pre_beta)
    p, ld_o, ld_u = _boundary(x, o, u, group_id, values, eps, gate, dev)
    shape = x.shape
    T, d = shape
    if dh is not None:
        _given("dh", dh, shape, x.dtype, dev)
    if pre_gamma is not None:
        if dy is None or dy.dtype not in _STREAM_TYPES:
            raise ValueError("dy of float32 or bfloat16 is needed with the pre norm")
        _given("dy", dy, shape, dy.dtype, dev)
    elif dh is None or dy is not None:
        raise ValueError("without the pre norm dh is needed, and no dy")
    if status is not None:
        _given("status", status, (1,), torch.int32, dev)
    dx, do = _new(x), _new(o)
    out = dict(dx=dx, do=do)
    du = None
    if ld_u:
        du = out["du"] = _new(o)
    # one allocation for the parameters' gradients
    names = [n for n, v in zip(_PARAMS, values) if v is not None]
    ptr = [None] * 5
    if names:
        flat = _new(next(v for v in values if v is not None), (len(names), p.G, d))
        out.update(zip(names, flat.unbind(0)))
        base, k = flat.data_ptr(), 0
        for i, v in enumerate(values):
            if v is not None:
                ptr[i] = base + 4 * k * p.G * d
                k += 1
    need = _lib.load().mtgr_boundary_bwd_workspace_bytes(T, _byref(p))
    room = _given_ws(ws, need, dev)
    if room == 0:
        room = max(need, 256)
        ws = _new(group_id, room)
    _lib.check("mtgr_boundary_bwd", _lib.load().mtgr_boundary_bwd(
        _byref(p), T, group_id.data_ptr(), _CODE[o.dtype], o.data_ptr(), ld_o, u.data_ptr() if ld_u else None, ld_u,
        _CODE[x.dtype], x.data_ptr(), None if dh is None else dh.data_ptr(), 0 if dy is None else _CODE[dy.dtype],
        None if dy is None else dy.data_ptr(), do.data_ptr(), d, None if du is None else du.data_ptr(), d,
        dx.data_ptr(), _byref(MtgrBoundaryGrads(*ptr)), ws.data_ptr(), room,
        None if status is None else status.data_ptr(), raw))
    return out


@_in_its_place
def quantize_rows(x, q=None, scale=None, stream=None):
    """Rows of ``x`` [M, K] (float32, bfloat16, float16) to signed bytes with a
    float32 scale each (mtgr_quantize_rows): returns (q [M, K] int8, scale [M]).
    A weight's rows give the scales of its output channels."""
    dev = x.get_device()
    raw = _stream_now(dev)
    if x.dim() != 2:
        raise ValueError("x: [M, K] is needed")
    shape = x.shape
    ld = _given_rows("x", x, shape, _FLOATS, dev)
    if q is None:
        q = _new(x, dtype=torch.int8)
    else:
        _given("q", q, shape, torch.int8, dev)
    if scale is None:
        scale = _new(x, shape[0], torch.float32)
    else:
        _given("scale", scale, shape[:1], torch.float32, dev)
    _lib.check("mtgr_quantize_rows", _lib.load().mtgr_quantize_rows(
        shape[0], shape[1], _CODE[x.dtype], x.data_ptr(), ld, q.data_ptr(), scale.data_ptr(), raw))
    return q, scale


@_in_its_place
def linear_i8(x, w, w_scale, x_scale=None, bias=None, epi: int = MTGR_EPI_NONE, resid=None, q_cols: int = 0,
              out_dtype=torch.float32, out=None, ws=None, status=None, stream=None) -> torch.Tensor:
    """Linear layer with int8 weights ``w`` [N, K] and a scale per output channel
    ``w_scale`` [N]: out = epi(x w^T + bias) [M, N]. ``x`` [M, K] is float32,
    bfloat16 or float16, quantised by row on the way (mtgr_linear_i8), or int8
    with its rows' scales ``x_scale`` [M] (mtgr_gemm_i8). Epilogues, ``resid``
    [M, N] float32 and ``q_cols`` as in gemm. ``status``: a device int32 word
    (zeroed by the caller) for errors the device finds: an f16 value out of
    range, a wait that ran out; without it they go unseen."""
    dev = x.get_device()
    raw = _stream_now(dev)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x: [M, K] and w: [N, K] are needed")
    M, K = x.shape
    N = w.shape[0]
    _given("w", w, (N, K), torch.int8, dev)
    _given("w_scale", w_scale, (N,), torch.float32, dev)
    if bias is not None:
        _given("bias", bias, (N,), torch.float32, dev)
    if resid is not None:
        _given("resid", resid, (M, N), torch.float32, dev)
    if (resid is not None) != (epi == MTGR_EPI_RESID):
        raise ValueError("resid and MTGR_EPI_RESID come together")
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype {out_dtype}: float32, bfloat16 or float16")
    if out is None:
        out = _new(w_scale, (M, N)) if out_dtype == torch.float32 else _new(w_scale, (M, N), out_dtype)
    else:
        _given("out", out, (M, N), out_dtype, dev)
    if status is not None:
        _given("status", status, (1,), torch.int32, dev)
    tail = (w.data_ptr(), w_scale.data_ptr(), None if bias is None else bias.data_ptr(), epi,
            None if resid is None else resid.data_ptr(), q_cols, _CODE[out_dtype], out.data_ptr())
    st = None if status is None else status.data_ptr()
    if x.dtype == torch.int8:
        _given("x", x, (M, K), torch.int8, dev)
        if x_scale is None:
            raise ValueError("x_scale is needed with int8 rows")
        _given("x_scale", x_scale, (M,), torch.float32, dev)
        _lib.check("mtgr_gemm_i8", _lib.load().mtgr_gemm_i8(M, N, K, x.data_ptr(), x_scale.data_ptr(), *tail, st, raw))
        return out
    if x_scale is not None:
        raise ValueError("x_scale goes with int8 rows")
    ld = _given_rows("x", x, (M, K), _FLOATS, dev)
    need = _lib.load().mtgr_linear_i8_workspace_bytes(M, N, K)
    room, p = _given_ws(ws, need, dev), None
    if need > 0:
        if room == 0:
            ws, room = _new(w, need), need
        p = ws.data_ptr()
    _lib.check("mtgr_linear_i8", _lib.load().mtgr_linear_i8(M, N, K, _CODE[x.dtype], x.data_ptr(), ld, *tail, p, room, st,
                                                            raw))
    return out


def gemm_i8(a, a_scale, b, b_scale, bias=None, epi: int = MTGR_EPI_NONE, resid=None, q_cols: int = 0,
            out_dtype=torch.float32, out=None, status=None, stream=None) -> torch.Tensor:
    """out = epi(a_scale b_scale a b^T + bias) of int8 ``a`` [M, K] and ``b`` [N, K]
    with a scale per row of each (mtgr_gemm_i8)."""
    if a.dtype != torch.int8:
        raise ValueError("a: int8 rows are needed")
    return linear_i8(a, b, b_scale, a_scale, bias, epi, resid, q_cols, out_dtype, out, None, status, stream)


class GradientSet:
    """A set of gradient tensors whose global norm is clipped in one call
    (mtgr_grad_clip), kept by a training program from step to step.

    ``grads``: device tensors (float32, bfloat16, float16), e.g. what
    hstu_block_backward and boundary_backward return; contiguous, of any size.
    ``outs``: where the clipped values go, tensor by tensor (the gradient's
    type or float32); None: in place. The tensors' memory is read at every
    call, so a step writes new gradients into the same buffers. The set's
    workspaces and status word are its own: clips of one set are ordered by
    the caller, two sets may run at once. A norm may run beside a clip of the same
    set if the clip writes other buffers (in place it would read what the clip
    writes). A set made while a graph is captured is zeroed by that graph: it
    is not used before the graph has run.
    """

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.grads) != len(self.outs) or not self.grads:
            raise ValueError("at least one gradient, and one output per gradient, are needed")
        if not self.grads[0].is_cuda:
            raise ValueError("device tensors are needed")
        self.device = self.grads[0].device
        dev, n = self.device.index, len(self.grads)
        spans = []
        self.c = (MtgrGradTensor * n)()
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.dtype not in _FLOATS or o.dtype not in (g.dtype, torch.float32):
                raise ValueError(f"tensor {i}: {g.dtype} to {o.dtype}: a float type to itself or to float32")
            _given(f"grads[{i}]", g, g.shape, g.dtype, dev)
            _given(f"outs[{i}]", o, g.shape, o.dtype, dev)
            self.c[i] = MtgrGradTensor(g.data_ptr(), o.data_ptr(), g.numel(), _CODE[g.dtype], _CODE[o.dtype])
            if g.numel():
                spans.append((o.data_ptr(), o.data_ptr() + o.numel() * o.element_size(), i, 1))
                if o.data_ptr() != g.data_ptr() or o.dtype != g.dtype:
                    spans.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), i, 0))
        # no two outputs may share memory, nor an output and another gradient
        spans.sort()
        end_out = end_any = 0
        for lo, hi, i, is_out in spans:
            if lo < (end_any if is_out else end_out):
                raise ValueError(f"tensor {i} shares memory with another one")
            end_any = max(end_any, hi)
            if is_out:
                end_out = max(end_out, hi)
        # the norm alone
        self.c_norm = (MtgrGradTensor * n)(*[MtgrGradTensor(c.g, None, c.n, c.dtype, c.dtype) for c in self.c])
        with torch.cuda.device(self.device):
            # one for each of the two calls
            size = _lib.mtgr_grad_clip_workspace_bytes(self.c, n)
            self.ws, self.ws_norm = (torch.zeros(size, dtype=torch.uint8, device=self.device) for _ in range(2))
            self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()  # zeros before a clip on any stream

    def clip(self, max_norm: float, inv_scale: float = 1.0, norm=None, status=None, stream=None) -> torch.Tensor:
        """Clips to ``max_norm`` after taking the loss scale out (``inv_scale`` = 1 /
        loss scale). Returns the norm before clipping ([1] float32 on the
        device). A norm that is not finite leaves the outputs as they were and
        MTGR_ERR_RANGE in ``status`` (default: the set's own word, see check)."""
        return _clip(self.ws, self, self.c, max_norm, inv_scale, norm, status, stream)

    def norm(self, inv_scale: float = 1.0, norm=None, status=None, stream=None) -> torch.Tensor:
        """The norm alone; nothing is written but it."""
        return _clip(self.ws_norm, self, self.c_norm, float("inf"), inv_scale, norm, status, stream)

    def check(self) -> None:
        """Synchronise and raise if a call on this set met a norm that is not
        finite, or ran into the limit of its waits; the word is then cleared
        for the next step."""
        torch.cuda.synchronize(self.device)
        st = int(self.status.item())
        if st != 0:
            self.status.zero_()
            raise _lib.MTGRError("device status", st)


@_in_its_place
def _clip(ws, grads, table, max_norm, inv_scale, norm, status, stream):
    dev = ws.get_device()
    raw = _stream_now(dev)
    if norm is None:
        norm = _new(ws, 1, torch.float32)
    else:
        _given("norm", norm, (1,), torch.float32, dev)
    if status is None:
        status = grads.status
    else:
        _given("status", status, (1,), torch.int32, dev)
    if stream is not None:
        ws.record_stream(stream)
        grads.status.record_stream(stream)
    _lib.check("mtgr_grad_clip", _lib.load().mtgr_grad_clip(
        table, len(table), max_norm, inv_scale, norm.data_ptr(), ws.data_ptr(), ws.numel(), status.data_ptr(), raw))
    return norm
