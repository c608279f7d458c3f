"""Dense operators around a paged MoE layer (binding of libpe's pe_rms_norm,
pe_linear, pe_gated_ffn and their backward calls; include/pe.h states what
each computes).

Tensors are torch CUDA tensors of one device: bf16 or fp16 (``linear`` also
takes E4M3 with scales).  Matrices are [rows, features]; activations that are
read may have any row pitch that is a multiple of 16 bytes, everything else is
contiguous.  Calls are asynchronous on the current stream, or on ``stream``;
then results and workspaces belong to that stream.  Invalid arguments raise
PEError.  There is no autograd: ``save=True`` returns what the backward call
needs.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import PE_ERR_INVALID, PEError, lib

GROUP = 128  # features that share one scale of an 8-bit row

_ACT = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}
_ELEM = {torch.bfloat16: 0, torch.float16: 1}
_F32 = 2
_E4M3 = torch.float8_e4m3fn


class RmsNorm(NamedTuple):
    """What ``rms_norm`` returns; None for what was not asked for."""

    y: torch.Tensor | None
    sum: torch.Tensor  # x + residual (x itself without one)
    codes: torch.Tensor | None  # E4M3; y = codes * scale of its 128 features
    scale: torch.Tensor | None  # fp32 [rows, ceil(hidden / 128)]
    rstd: torch.Tensor | None  # fp32 [rows]


def _bad(msg: str):
    raise PEError(PE_ERR_INVALID, msg)


def _fail(st: int):
    raise PEError(st, lib().pe_last_error(None).decode())


def _elem(dt, who: str) -> int:
    e = _ELEM.get(dt)
    if e is None:
        _bad(f"{who}: {dt} is neither bf16 nor fp16")
    return e


def _act(act: str) -> int:
    a = _ACT.get(act)
    if a is None:
        _bad(f"unknown activation {act!r}; one of {', '.join(_ACT)}")
    return a


def _rows(t, shape, dtype, dev: int, name: str):
    """(pointer, row pitch) of a matrix with unit column stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _bad(f"{name}: want {dtype} {list(shape)} on cuda:{dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    ld, unit = t.stride()
    if unit != 1 and shape[0] and shape[1] > 1:
        _bad(f"{name}: columns must be contiguous")
    # the pitch of a single row is never used: a view of one row may state any
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1])


def _whole(t, shape, dtype, dev: int, name: str) -> int:
    """Pointer of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name}: want contiguous {dtype} {list(shape)} on cuda:{dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


try:  # the raw handle, without a Stream object around it
    _current_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
except AttributeError:  # CPU-only builds

    def _current_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream

    _current_device = torch.cuda.current_device


def _matrix(t, name: str):
    """(shape, device) of a CUDA matrix."""
    shape, dev = t.shape, t.get_device()
    if len(shape) != 2 or dev < 0:
        _bad(f"{name}: want a CUDA matrix [rows, features], got {list(shape)} on {t.device}")
    return shape, dev


def _elsewhere(call, dev: int, stream, *args, **kw):
    """The call with `dev` current, on ``stream``: its allocations belong there too."""
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args, **kw)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):  # makes the stream's device current
        if _current_device() != dev:
            _bad(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        return call(*args, **kw)


_empty = torch.empty
_empty_like = torch.empty_like


def error_word() -> int:
    """The device's error word: 0, or PE_DEVERR_TIMEOUT after a wait inside a
    kernel gave up.  Synchronises the device."""
    w = ctypes.c_uint32()
    st = lib().pe_dense_error(ctypes.byref(w))
    if st:
        _fail(st)
    return int(w.value)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, *, y: bool = True, quant: bool = False, save: bool = False,
             stream=None) -> RmsNorm:
    """RMS norm of x + residual, over each row.

    ``quant`` adds y as E4M3 codes with a scale per 128 features (what
    ``linear`` takes); ``y=False`` then leaves the 16-bit form out.  ``save``
    adds rstd for ``rms_norm_backward``."""
    shape, dev = _matrix(x, "x")
    if stream is not None or _current_device() != dev:
        return _elsewhere(rms_norm, dev, stream, x, weight, residual, eps, y=y, quant=quant, save=save)
    rows, hidden = shape
    dt = x.dtype
    elem = _elem(dt, "x")
    xp, xs = _rows(x, shape, dt, dev, "x")
    wp = _whole(weight, (hidden,), dt, dev, "weight")
    out = total = codes = scale = rstd = rp = yp = tp = cp = sp = sdp = None
    rs = 0
    if y:
        out = _empty(shape, dtype=dt, device=x.device)
        yp = out.data_ptr()
    if residual is None:
        total = x
    else:
        rp, rs = _rows(residual, shape, dt, dev, "residual")
        total = _empty(shape, dtype=dt, device=x.device)
        tp = total.data_ptr()
    if quant:
        codes = _empty(shape, dtype=_E4M3, device=x.device)
        scale = _empty((rows, -(-hidden // GROUP)), dtype=torch.float32, device=x.device)
        cp, sp = codes.data_ptr(), scale.data_ptr()
    if save:
        rstd = _empty(rows, dtype=torch.float32, device=x.device)
        sdp = rstd.data_ptr()
    st = lib().pe_rms_norm(xp, xs, rp, rs, wp, eps, yp, tp, cp, sp, sdp, rows, hidden, elem, _current_stream(dev))
    if st:
        _fail(st)
    return RmsNorm(out, total, codes, scale, rstd)


def rms_norm_backward(dy, sum, weight, rstd, dsum=None, *, stream=None):
    """(dx, dweight) of ``rms_norm``; dx is the residual's gradient too.
    ``dsum``: the gradient that reaches the sum by the residual stream."""
    shape, dev = _matrix(sum, "sum")
    if stream is not None or _current_device() != dev:
        return _elsewhere(rms_norm_backward, dev, stream, dy, sum, weight, rstd, dsum)
    rows, hidden = shape
    dt, L = sum.dtype, lib()
    elem = _elem(dt, "sum")
    sp, ss = _rows(sum, shape, dt, dev, "sum")
    yp, ys = _rows(dy, shape, dt, dev, "dy")
    dp, ds = (None, 0) if dsum is None else _rows(dsum, shape, dt, dev, "dsum")
    wp = _whole(weight, (hidden,), dt, dev, "weight")
    rp = _whole(rstd, (rows,), torch.float32, dev, "rstd")
    dx = _empty(shape, dtype=dt, device=sum.device)
    dw = _empty_like(weight)
    n = L.pe_rms_norm_backward_workspace(rows, hidden)
    ws = _empty(n, dtype=torch.uint8, device=sum.device)
    st = L.pe_rms_norm_backward(yp, ys, dp, ds, sp, ss, wp, rp, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), n, rows, hidden,
                                elem, _current_stream(dev))
    if st:
        _fail(st)
    return dx, dw


def linear(x, weight, bias=None, act: str = "none", residual=None, *, x_scale=None, w_scale=None, out_dtype=None,
           save: bool = False, stream=None):
    """act(x weight^T + bias) + residual; weight [out, in].

    E4M3 x and weight come with ``x_scale`` [rows, ceil(in/128)] and
    ``w_scale`` [ceil(out/128), ceil(in/128)]; the result's type is then that of
    residual or bias, or ``out_dtype``, or bf16.  ``out_dtype=torch.float32``
    leaves the result unrounded (router logits).  ``save`` returns (out, z),
    z = x weight^T + bias for ``linear_backward`` (None for act "none")."""
    shape, dev = _matrix(x, "x")
    if stream is not None or _current_device() != dev:
        return _elsewhere(linear, dev, stream, x, weight, bias, act, residual, x_scale=x_scale, w_scale=w_scale,
                          out_dtype=out_dtype, save=save)
    rows, k = shape
    a, dt = _act(act), x.dtype
    n = weight.shape[0]
    wp = _whole(weight, (n, k), dt, dev, "weight")
    xp, xs = _rows(x, shape, dt, dev, "x")
    xsp = wsp = bp = rp = zp = z = None
    rs = 0
    if dt is _E4M3:
        if x_scale is None or w_scale is None:
            _bad("E4M3 x and weight need x_scale and w_scale")
        kg = -(-k // GROUP)
        xsp = _whole(x_scale, (rows, kg), torch.float32, dev, "x_scale")
        wsp = _whole(w_scale, (-(-n // GROUP), kg), torch.float32, dev, "w_scale")
        dt = residual.dtype if residual is not None else bias.dtype if bias is not None else out_dtype
        if dt is None or dt is torch.float32:
            dt = torch.bfloat16
    elif x_scale is not None or w_scale is not None:
        _bad("scales go with E4M3 x and weight")
    elem = out_elem = _elem(dt, "x")
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype is not dt:
        if out_dtype is not torch.float32:
            _bad(f"out_dtype: want {dt} or torch.float32, got {out_dtype}")
        out_elem = _F32
    if bias is not None:
        bp = _whole(bias, (n,), dt, dev, "bias")
    if residual is not None:
        rp, rs = _rows(residual, (rows, n), dt, dev, "residual")
    out = _empty((rows, n), dtype=out_dtype, device=x.device)
    if save and a:
        z = _empty((rows, n), dtype=dt, device=x.device)
        zp = z.data_ptr()
    st = lib().pe_linear(xp, xs, xsp, wp, wsp, bp, rp, rs, out.data_ptr(), out_elem, zp, a, rows, k, n, elem,
                         _current_stream(dev))
    if st:
        _fail(st)
    return (out, z) if save else out


def linear_backward(dy, x, weight, z=None, act: str = "none", *, bias: bool = False, stream=None):
    """(dx, dweight, dbias) of ``linear``; dbias is None unless ``bias``.  The
    residual's gradient is dy itself."""
    shape, dev = _matrix(x, "x")
    if stream is not None or _current_device() != dev:
        return _elsewhere(linear_backward, dev, stream, dy, x, weight, z, act, bias=bias)
    rows, k = shape
    a, dt, L = _act(act), x.dtype, lib()
    elem = _elem(dt, "x")
    n = weight.shape[0]
    xp, xs = _rows(x, shape, dt, dev, "x")
    yp, ys = _rows(dy, (rows, n), dt, dev, "dy")
    wp = _whole(weight, (n, k), dt, dev, "weight")
    if a and z is None:
        _bad(f"act {act!r} needs the z that linear(save=True) returned")
    zp = _whole(z, (rows, n), dt, dev, "z") if a else None
    dx = _empty(shape, dtype=dt, device=x.device)
    dw = _empty_like(weight)
    db = _empty(n, dtype=dt, device=x.device) if bias else None
    ws_n = L.pe_linear_backward_workspace(rows, n, a)
    ws = _empty(ws_n, dtype=torch.uint8, device=x.device)
    st = L.pe_linear_backward(yp, ys, xp, xs, wp, zp, a, dx.data_ptr(), dw.data_ptr(), db.data_ptr() if bias else None,
                              ws.data_ptr(), ws_n, rows, k, n, elem, _current_stream(dev))
    if st:
        _fail(st)
    return dx, dw, db


def gated_ffn(x, w13, w2, act: str = "silu", residual=None, *, save: bool = False, stream=None):
    """(act(x gate^T) * (x up^T)) w2^T + residual; w13 [2 I, H] holds the gate
    rows, then the up rows, w2 is [H, I].  ``save`` returns (out, gu) with the
    [rows, 2 I] gate and up products for ``gated_ffn_backward``."""
    shape, dev = _matrix(x, "x")
    if stream is not None or _current_device() != dev:
        return _elsewhere(gated_ffn, dev, stream, x, w13, w2, act, residual, save=save)
    rows, h = shape
    a, dt, L = _act(act), x.dtype, lib()
    elem = _elem(dt, "x")
    i = w2.shape[-1]
    xp, xs = _rows(x, shape, dt, dev, "x")
    w13p = _whole(w13, (2 * i, h), dt, dev, "w13")
    w2p = _whole(w2, (h, i), dt, dev, "w2")
    rp, rs = (None, 0) if residual is None else _rows(residual, shape, dt, dev, "residual")
    out = _empty(shape, dtype=dt, device=x.device)
    gu = _empty((rows, 2 * i), dtype=dt, device=x.device) if save else None
    n = L.pe_gated_ffn_workspace(rows, i)
    ws = _empty(n, dtype=torch.uint8, device=x.device)
    st = L.pe_gated_ffn(xp, xs, w13p, w2p, rp, rs, out.data_ptr(), gu.data_ptr() if save else None, a, ws.data_ptr(), n, rows,
                        h, i, elem, _current_stream(dev))
    if st:
        _fail(st)
    return (out, gu) if save else out


def gated_ffn_backward(dy, x, w13, w2, gu, act: str = "silu", *, stream=None):
    """(dx, dw13, dw2) of ``gated_ffn``.  The residual's gradient is dy itself."""
    shape, dev = _matrix(x, "x")
    if stream is not None or _current_device() != dev:
        return _elsewhere(gated_ffn_backward, dev, stream, dy, x, w13, w2, gu, act)
    rows, h = shape
    a, dt, L = _act(act), x.dtype, lib()
    elem = _elem(dt, "x")
    i = w2.shape[-1]
    xp, xs = _rows(x, shape, dt, dev, "x")
    yp, ys = _rows(dy, shape, dt, dev, "dy")
    w13p = _whole(w13, (2 * i, h), dt, dev, "w13")
    w2p = _whole(w2, (h, i), dt, dev, "w2")
    gp = _whole(gu, (rows, 2 * i), dt, dev, "gu")
    dx, dw13, dw2 = _empty(shape, dtype=dt, device=x.device), _empty_like(w13), _empty_like(w2)
    n = L.pe_gated_ffn_backward_workspace(rows, i)
    ws = _empty(n, dtype=torch.uint8, device=x.device)
    st = L.pe_gated_ffn_backward(yp, ys, xp, xs, w13p, w2p, gp, a, dx.data_ptr(), dw13.data_ptr(), dw2.data_ptr(),
                                 ws.data_ptr(), n, rows, h, i, elem, _current_stream(dev))
    if st:
        _fail(st)
    return dx, dw13, dw2
