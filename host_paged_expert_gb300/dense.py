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
from contextlib import nullcontext
from typing import NamedTuple

import torch

from ._lib import PE_ERR_INVALID, PE_OK, PEError, lib

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


def _check(st: int) -> None:
    if st != PE_OK:
        raise PEError(st, lib().pe_last_error(None).decode())


def _elem(t, who: str) -> int:
    e = _ELEM.get(t.dtype)
    if e is None:
        _bad(f"{who}: {t.dtype} is neither bf16 nor fp16")
    return e


def _act(act: str) -> int:
    a = _ACT.get(act)
    if a is None:
        _bad(f"unknown activation {act!r}; one of {', '.join(_ACT)}")
    return a


def _rows(t, rows: int, cols: int, dtype, dev: int, name: str):
    """(pointer, row pitch) of a [rows, cols] matrix with unit column stride."""
    if t.dtype != dtype or t.shape != (rows, cols) or t.get_device() != dev:
        _bad(f"{name}: want {dtype} [{rows}, {cols}] on cuda:{dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    ld, unit = t.stride()
    if unit != 1 and rows and cols > 1:
        _bad(f"{name}: columns must be contiguous")
    # the pitch of a single row is never used: a view of one row may state any
    return t.data_ptr(), (ld if rows > 1 else cols)


def _whole(t, shape: tuple, dtype, dev: int, name: str) -> int:
    """Pointer of a contiguous tensor."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name}: want contiguous {dtype} {list(shape)} on cuda:{dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _matrix(t, name: str):
    if t.dim() != 2 or not t.is_cuda:
        _bad(f"{name}: want a CUDA matrix [rows, features], got {list(t.shape)} on {t.device}")
    return t.shape[0], t.shape[1], t.get_device()


try:  # the raw handle, without a Stream object around it
    _current_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
except AttributeError:  # pragma: no cover - CPU-only builds

    def _current_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream

    _current_device = torch.cuda.current_device


_HERE = nullcontext()


def _on(dev: int, stream):
    """Context in which allocations and launches go to ``stream`` of ``dev``."""
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        return torch.cuda.stream(stream)
    return _HERE if _current_device() == dev else torch.cuda.device(dev)


def error_word() -> int:
    """The device's error word: 0, or PE_DEVERR_TIMEOUT after a wait inside a
    kernel gave up.  Synchronises the device."""
    w = ctypes.c_uint32()
    _check(lib().pe_dense_error(ctypes.byref(w)))
    return int(w.value)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, *, y: bool = True, quant: bool = False, save: bool = False,
             stream=None) -> RmsNorm:
    """RMS norm of x + residual, over each row.

    ``quant`` adds y as E4M3 codes with a scale per 128 features (what
    ``linear`` takes); ``y=False`` then leaves the 16-bit form out.  ``save``
    adds rstd for ``rms_norm_backward``."""
    rows, hidden, dev = _matrix(x, "x")
    elem, dt = _elem(x, "x"), x.dtype
    xp, xs = _rows(x, rows, hidden, dt, dev, "x")
    wp = _whole(weight, (hidden,), dt, dev, "weight")
    rp, rs = (None, 0) if residual is None else _rows(residual, rows, hidden, dt, dev, "residual")
    with _on(dev, stream):
        out = x.new_empty((rows, hidden)) if y else None
        total = x if residual is None else x.new_empty((rows, hidden))
        codes = x.new_empty((rows, hidden), dtype=_E4M3) if quant else None
        scale = x.new_empty((rows, -(-hidden // GROUP)), dtype=torch.float32) if quant else None
        rstd = x.new_empty(rows, dtype=torch.float32) if save else None
        _check(lib().pe_rms_norm(xp, xs, rp, rs, wp, eps, out.data_ptr() if y else None,
                                 None if residual is None else total.data_ptr(), codes.data_ptr() if quant else None,
                                 scale.data_ptr() if quant else None, rstd.data_ptr() if save else None, rows, hidden,
                                 elem, _current_stream(dev)))
    return RmsNorm(out, total, codes, scale, rstd)


def rms_norm_backward(dy, sum, weight, rstd, dsum=None, *, stream=None):
    """(dx, dweight) of ``rms_norm``; dx is the residual's gradient too.
    ``dsum``: the gradient that reaches the sum by the residual stream."""
    rows, hidden, dev = _matrix(sum, "sum")
    elem, dt, L = _elem(sum, "sum"), sum.dtype, lib()
    sp, ss = _rows(sum, rows, hidden, dt, dev, "sum")
    yp, ys = _rows(dy, rows, hidden, dt, dev, "dy")
    dp, ds = (None, 0) if dsum is None else _rows(dsum, rows, hidden, dt, dev, "dsum")
    wp = _whole(weight, (hidden,), dt, dev, "weight")
    rp = _whole(rstd, (rows,), torch.float32, dev, "rstd")
    with _on(dev, stream):
        dx, dw = sum.new_empty((rows, hidden)), sum.new_empty(hidden)
        n = L.pe_rms_norm_backward_workspace(rows, hidden)
        ws = sum.new_empty(n, dtype=torch.uint8)
        _check(L.pe_rms_norm_backward(yp, ys, dp, ds, sp, ss, wp, rp, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), n,
                                      rows, hidden, elem, _current_stream(dev)))
    return dx, dw


def linear(x, weight, bias=None, act: str = "none", residual=None, *, x_scale=None, w_scale=None, out_dtype=None,
           save: bool = False, stream=None):
    """act(x weight^T + bias) + residual; weight [out, in].

    E4M3 x and weight come with ``x_scale`` [rows, ceil(in/128)] and
    ``w_scale`` [ceil(out/128), ceil(in/128)]; the result's type is then that of
    residual or bias, or ``out_dtype``, or bf16.  ``out_dtype=torch.float32``
    leaves the result unrounded (router logits).  ``save`` returns (out, z),
    z = x weight^T + bias for ``linear_backward`` (None for act "none")."""
    rows, k, dev = _matrix(x, "x")
    a, dt = _act(act), x.dtype
    n = weight.shape[0]
    wp = _whole(weight, (n, k), dt, dev, "weight")
    xp, xs = _rows(x, rows, k, dt, dev, "x")
    xsp = wsp = None
    if dt == _E4M3:
        if x_scale is None or w_scale is None:
            _bad("E4M3 x and weight need x_scale and w_scale")
        kg = -(-k // GROUP)
        xsp = _whole(x_scale, (rows, kg), torch.float32, dev, "x_scale")
        wsp = _whole(w_scale, (-(-n // GROUP), kg), torch.float32, dev, "w_scale")
        dt = residual.dtype if residual is not None else bias.dtype if bias is not None else out_dtype
        if dt is None or dt == torch.float32:
            dt = torch.bfloat16
    elif x_scale is not None or w_scale is not None:
        _bad("scales go with E4M3 x and weight")
    elem = _ELEM.get(dt)
    if elem is None:
        _bad(f"x: {dt} is neither bf16, fp16 nor E4M3")
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype != dt and out_dtype != torch.float32:
        _bad(f"out_dtype: want {dt} or torch.float32, got {out_dtype}")
    bp = None if bias is None else _whole(bias, (n,), dt, dev, "bias")
    rp, rs = (None, 0) if residual is None else _rows(residual, rows, n, dt, dev, "residual")
    with _on(dev, stream):
        out = x.new_empty((rows, n), dtype=out_dtype)
        z = x.new_empty((rows, n), dtype=dt) if save and a else None
        _check(lib().pe_linear(xp, xs, xsp, wp, wsp, bp, rp, rs, out.data_ptr(), elem if out_dtype == dt else _F32,
                               None if z is None else z.data_ptr(), a, rows, k, n, elem, _current_stream(dev)))
    return (out, z) if save else out


def linear_backward(dy, x, weight, z=None, act: str = "none", *, bias: bool = False, stream=None):
    """(dx, dweight, dbias) of ``linear``; dbias is None unless ``bias``.  The
    residual's gradient is dy itself."""
    rows, k, dev = _matrix(x, "x")
    a, elem, dt, L = _act(act), _elem(x, "x"), x.dtype, lib()
    n = weight.shape[0]
    xp, xs = _rows(x, rows, k, dt, dev, "x")
    yp, ys = _rows(dy, rows, n, dt, dev, "dy")
    wp = _whole(weight, (n, k), dt, dev, "weight")
    if a and z is None:
        _bad(f"act {act!r} needs the z that linear(save=True) returned")
    zp = _whole(z, (rows, n), dt, dev, "z") if a else None
    with _on(dev, stream):
        dx, dw = x.new_empty((rows, k)), x.new_empty((n, k))
        db = x.new_empty(n) if bias else None
        ws_n = L.pe_linear_backward_workspace(rows, n, a)
        ws = x.new_empty(ws_n, dtype=torch.uint8)
        _check(L.pe_linear_backward(yp, ys, xp, xs, wp, zp, a, dx.data_ptr(), dw.data_ptr(),
                                    db.data_ptr() if bias else None, ws.data_ptr(), ws_n, rows, k, n, elem,
                                    _current_stream(dev)))
    return dx, dw, db


def gated_ffn(x, w13, w2, act: str = "silu", residual=None, *, save: bool = False, stream=None):
    """(act(x gate^T) * (x up^T)) w2^T + residual; w13 [2 I, H] holds the gate
    rows, then the up rows, w2 is [H, I].  ``save`` returns (out, gu) with the
    [rows, 2 I] gate and up products for ``gated_ffn_backward``."""
    rows, h, dev = _matrix(x, "x")
    a, elem, dt, L = _act(act), _elem(x, "x"), x.dtype, lib()
    i = w2.shape[-1]
    xp, xs = _rows(x, rows, h, dt, dev, "x")
    w13p = _whole(w13, (2 * i, h), dt, dev, "w13")
    w2p = _whole(w2, (h, i), dt, dev, "w2")
    rp, rs = (None, 0) if residual is None else _rows(residual, rows, h, dt, dev, "residual")
    with _on(dev, stream):
        out = x.new_empty((rows, h))
        gu = x.new_empty((rows, 2 * i)) if save else None
        n = L.pe_gated_ffn_workspace(rows, i)
        ws = x.new_empty(n, dtype=torch.uint8)
        _check(L.pe_gated_ffn(xp, xs, w13p, w2p, rp, rs, out.data_ptr(), gu.data_ptr() if save else None, a,
                              ws.data_ptr(), n, rows, h, i, elem, _current_stream(dev)))
    return (out, gu) if save else out


def gated_ffn_backward(dy, x, w13, w2, gu, act: str = "silu", *, stream=None):
    """(dx, dw13, dw2) of ``gated_ffn``.  The residual's gradient is dy itself."""
    rows, h, dev = _matrix(x, "x")
    a, elem, dt, L = _act(act), _elem(x, "x"), x.dtype, lib()
    i = w2.shape[-1]
    xp, xs = _rows(x, rows, h, dt, dev, "x")
    yp, ys = _rows(dy, rows, h, dt, dev, "dy")
    w13p = _whole(w13, (2 * i, h), dt, dev, "w13")
    w2p = _whole(w2, (h, i), dt, dev, "w2")
    gp = _whole(gu, (rows, 2 * i), dt, dev, "gu")
    with _on(dev, stream):
        dx, dw13, dw2 = x.new_empty((rows, h)), x.new_empty((2 * i, h)), x.new_empty((h, i))
        n = L.pe_gated_ffn_backward_workspace(rows, i)
        ws = x.new_empty(n, dtype=torch.uint8)
        _check(L.pe_gated_ffn_backward(yp, ys, xp, xs, w13p, w2p, gp, a, dx.data_ptr(), dw13.data_ptr(), dw2.data_ptr(),
                                       ws.data_ptr(), n, rows, h, i, elem, _current_stream(dev)))
    return dx, dw13, dw2
