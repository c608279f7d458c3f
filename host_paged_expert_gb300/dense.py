"""Dense operators around a paged MoE layer (binding of libpe's pe_rms_norm,
pe_linear, pe_gated_ffn and their backward calls; include/pe.h states what
each computes).

Tensors are torch CUDA tensors of one device: bf16 or fp16 (``linear`` also
takes E4M3 with scales).  Matrices are [rows, features]; activations that are
read may have any row pitch that is a multiple of 16 bytes, everything else is
contiguous.  Calls are asynchronous on the current stream, or on ``stream``;
then results and workspaces belong to that stream, which has to wait for what
made the arguments, and the arguments may be freed as soon as the call returns.
Invalid arguments raise
PEError.  There is no autograd: ``save=True`` returns what the backward call
needs, and a tensor that requires gradients is refused unless gradients are
off (``torch.no_grad()``, or inside a ``torch.autograd.Function``).
"""

from __future__ import annotations

import ctypes
import importlib
import os
from typing import NamedTuple

import torch

from ._lib import PEError, lib

GROUP = 128  # features that share one scale of an 8-bit row
_ACT = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


class RmsNorm(NamedTuple):
    """What ``rms_norm`` returns; None for what was not asked for."""

    y: torch.Tensor | None
    sum: torch.Tensor  # x + residual (x itself without one)
    codes: torch.Tensor | None  # E4M3; y = codes * scale of its 128 features
    scale: torch.Tensor | None  # fp32 [rows, ceil(hidden / 128)]
    rstd: torch.Tensor | None  # fp32 [rows]


def _raise(status: int, msg: str):
    raise PEError(status, msg)


def _elsewhere(call, dev: int, stream, args):
    """The call with `dev` current, on ``stream``: its allocations belong there too."""
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args, None)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream.device.index != dev:
        _raise(1, f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    with torch.cuda.stream(stream):  # makes the stream's device current
        out = call(*args, None)
    for a in args:  # their memory stays theirs until the stream is past the call
        if isinstance(a, torch.Tensor):
            a.record_stream(stream)
    return out


_native = None


def _c():
    """The binding (csrc/py_dense.cpp), built in-tree next to libpe.so."""
    global _native
    if _native is None:
        lib()  # raises if libpe is not built
        try:
            m = importlib.import_module("._dense", __package__)
        except ImportError as e:
            raise RuntimeError(f"_dense.so is not built ({os.path.dirname(__file__)}); "
                               "run host_paged_expert_gb300.build.build()") from e
        m.setup(_ACT, _raise, _elsewhere, RmsNorm)
        _native = m
    return _native


def error_word() -> int:
    """The device's error word: 0, or PE_DEVERR_TIMEOUT after a wait inside a
    kernel gave up.  Synchronises the device."""
    w = ctypes.c_uint32()
    st = lib().pe_dense_error(ctypes.byref(w))
    if st:
        _raise(st, lib().pe_last_error(None).decode())
    return int(w.value)


def selftest_waits(poll_limit: int = 1 << 12) -> list[int]:
    """Error words of the twelve runs of pe_selftest_dense_waits (each must
    read PE_DEVERR_TIMEOUT).  Synchronises the device."""
    scratch = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    out = (ctypes.c_uint32 * 12)()
    st = lib().pe_selftest_dense_waits(poll_limit, scratch.data_ptr(), scratch.numel(), out)
    if st:
        _raise(st, lib().pe_last_error(None).decode())
    return list(out)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, *, y: bool = True, quant: bool = False, save: bool = False,
             stream=None) -> RmsNorm:
    """RMS norm of x + residual, over each row.

    ``quant`` adds y as E4M3 codes with a scale per 128 features (what
    ``linear`` takes); ``y=False`` then leaves the 16-bit form out.  ``save``
    adds rstd for ``rms_norm_backward``."""
    return (_native or _c()).rms_norm(x, weight, residual, eps, y, quant, save, stream)


def rms_norm_backward(dy, sum, weight, rstd, dsum=None, *, stream=None):
    """(dx, dweight) of ``rms_norm``; dx is the residual's gradient too.
    ``dsum``: the gradient that reaches the sum by the residual stream."""
    return (_native or _c()).rms_norm_backward(dy, sum, weight, rstd, dsum, stream)


def linear(x, weight, bias=None, act: str = "none", residual=None, *, x_scale=None, w_scale=None, out_dtype=None,
           save: bool = False, stream=None):
    """act(x weight^T + bias) + residual; weight [out, in].

    E4M3 x and weight come with ``x_scale`` [rows, ceil(in/128)] and
    ``w_scale`` [ceil(out/128), ceil(in/128)]; the result's type is then that of
    residual or bias, or ``out_dtype``, or bf16.  ``out_dtype=torch.float32``
    leaves the result unrounded (router logits).  ``save`` returns (out, z),
    z = x weight^T + bias for ``linear_backward`` (None for act "none")."""
    return (_native or _c()).linear(x, weight, bias, act, residual, x_scale, w_scale, out_dtype, save, stream)


def linear_backward(dy, x, weight, z=None, act: str = "none", *, bias: bool = False, stream=None):
    """(dx, dweight, dbias) of ``linear``; dbias is None unless ``bias``.  The
    residual's gradient is dy itself."""
    return (_native or _c()).linear_backward(dy, x, weight, z, act, bias, stream)


def gated_ffn(x, w13, w2, act: str = "silu", residual=None, *, save: bool = False, stream=None):
    """(act(x gate^T) * (x up^T)) w2^T + residual; w13 [2 I, H] holds the gate
    rows, then the up rows, w2 is [H, I].  ``save`` returns (out, gu) with the
    [rows, 2 I] gate and up products for ``gated_ffn_backward``."""
    return (_native or _c()).gated_ffn(x, w13, w2, act, residual, save, stream)


def gated_ffn_backward(dy, x, w13, w2, gu, act: str = "silu", *, stream=None):
    """(dx, dw13, dw2) of ``gated_ffn``.  The residual's gradient is dy itself."""
    return (_native or _c()).gated_ffn_backward(dy, x, w13, w2, gu, act, stream)
