"""Dense operators around a paged MoE layer, and those of a layer whose experts
are resident (binding of libpe's pe_rms_norm, pe_linear, pe_gated_ffn, pe_route,
pe_grouped_linear and their like; include/pe.h states what each computes).

Tensors are torch CUDA tensors of one device: bf16 or fp16 (``linear`` also
takes E4M3 with scales, ``linear_w4`` 4-bit weights); router logits and weights
are fp32, indices int32.  Matrices are [rows, features]; activations that are
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

from ._lib import PE_INT4_GPTQ, PE_MXFP4, PE_NVFP4, PEError, lib

GROUP = 128  # features that share one scale of an 8-bit row
_ACT = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}
_FORMAT = {"int4": PE_INT4_GPTQ, "mxfp4": PE_MXFP4, "nvfp4": PE_NVFP4}


class RmsNorm(NamedTuple):
    """What ``rms_norm`` returns; None for what was not asked for."""

    y: torch.Tensor | None
    sum: torch.Tensor  # x + residual (x itself without one)
    codes: torch.Tensor | None  # E4M3; y = codes * scale of its 128 features
    scale: torch.Tensor | None  # fp32 [rows, ceil(hidden / 128)]
    rstd: torch.Tensor | None  # fp32 [rows]


class Routing(NamedTuple):
    """What ``route`` returns.  A row is one entry (token, i), rows sorted by
    expert and by token within an expert."""

    ids: torch.Tensor  # int32 [tokens, top_k], in falling order of the logits
    weights: torch.Tensor  # fp32 [tokens, top_k], softmax over the chosen
    offsets: torch.Tensor  # int32 [experts + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1
    place: torch.Tensor  # int32 [tokens, top_k], the row of each entry


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
        m.setup(_ACT, _raise, _elsewhere, RmsNorm, Routing, _FORMAT)
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


def _selftest(call, poll_limit: int, scratch_bytes: int) -> list[int]:
    scratch = torch.empty(scratch_bytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    out = (ctypes.c_uint32 * 12)()
    st = call(poll_limit, scratch.data_ptr(), scratch.numel(), out)
    if st:
        _raise(st, lib().pe_last_error(None).decode())
    return list(out)


def selftest_waits(poll_limit: int = 1 << 12) -> list[int]:
    """Error words of the twelve runs of pe_selftest_dense_waits (each must
    read PE_DEVERR_TIMEOUT).  Synchronises the device."""
    return _selftest(lib().pe_selftest_dense_waits, poll_limit, 1 << 20)


def selftest_expert_waits(poll_limit: int = 1 << 12) -> list[int]:
    """The same of pe_selftest_experts_waits."""
    return _selftest(lib().pe_selftest_experts_waits, poll_limit, 4 << 20)


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


def linear_w4(x, codes, scales, fmt: str, bias=None, act: str = "none", residual=None, *, tensor_scale=None, out_dtype=None,
              stream=None):
    """act(x W^T + bias) + residual with W [out, in] in 4 bits, in the layout of
    an expert row (``formats.gptq_int4_to_row`` repacks a GPTQ checkpoint).

    ``codes`` uint8 [out, in / 2], input 2j in the low nibble of byte j; ``fmt``
    and ``scales``: "int4", (code - 8) times fp16 [out, ceil(in / 128)]; "mxfp4",
    E2M1 times E8M0 [out, in / 32] (uint8 or float8_e8m0fnu); "nvfp4", E2M1 times
    E4M3 [out, in / 16] (uint8 or float8_e4m3fn) times ``tensor_scale`` fp32 [1].
    ``out_dtype=torch.float32`` leaves the result unrounded.  Up to 128 rows no
    weight is rounded; above, int4's are rounded to x's type, and with fp16 MXFP4's
    and int4's have to lie in its range.  All but ``tensor_scale`` start at 16-byte
    boundaries."""
    return (_native or _c()).linear_w4(x, codes, scales, fmt, bias, act, residual, tensor_scale, out_dtype, stream)


def route(logits, top_k: int, *, stream=None) -> Routing:
    """Each token's ``top_k`` experts by logit (ties to the lower expert, NaN as
    -inf, as the paged layer routes) and each entry's row; logits fp32
    [tokens, experts]."""
    return (_native or _c()).route(logits, top_k, stream)


def route_backward(dweights, weights, ids, experts: int, *, stream=None):
    """The gradient of ``route``'s logits, fp32 [tokens, experts], from that of its weights."""
    return (_native or _c()).route_backward(dweights, weights, ids, experts, stream)


def expand_rows(x, place, rows: int | None = None, *, stream=None):
    """x[t] at every row place[t, i] of [rows, features] (as many rows as entries
    by default).  Entries with a place outside [0, rows) are left out, and rows
    that no entry names hold anything; no two entries may name the same row.
    Its gradient is ``combine_rows(dy, place)``."""
    return (_native or _c()).expand_rows(x, place, rows, stream)


def combine_rows(y, place, weights=None, residual=None, *, stream=None):
    """sum_i weights[t, i] y[place[t, i]] + residual[t] (weights fp32; ones without)."""
    return (_native or _c()).combine_rows(y, place, weights, residual, stream)


def combine_rows_backward(dout, y, place, weights, *, stream=None):
    """(dy, dweights) of ``combine_rows``.  Rows of dy that no entry names hold
    anything; no two entries may name the same row.  The residual's gradient is
    dout itself."""
    return (_native or _c()).combine_rows_backward(dout, y, place, weights, stream)


def grouped_linear(x, weight, offsets, *, stream=None):
    """x[r] weight[g]^T for rows offsets[g] <= r < offsets[g + 1]; weight [groups,
    out, in], offsets int32 [groups + 1], not decreasing.  Rows in no group hold
    anything."""
    return (_native or _c()).grouped_linear(x, weight, offsets, stream)


def grouped_linear_backward(dy, x, weight, offsets, *, stream=None):
    """(dx, dweight) of ``grouped_linear``; an empty group's dweight is zero."""
    return (_native or _c()).grouped_linear_backward(dy, x, weight, offsets, stream)


def grouped_ffn(x, w13, w2, offsets, act: str = "silu", *, save: bool = False, stream=None):
    """``gated_ffn`` of each group's rows with its own weights: w13 [groups, 2 I, H],
    w2 [groups, H, I].  ``save`` returns (out, gu) with the fp32 [rows, 2 I] gate and
    up products for ``grouped_ffn_backward``."""
    return (_native or _c()).grouped_ffn(x, w13, w2, offsets, act, save, stream)


def grouped_ffn_backward(dy, x, w13, w2, gu, offsets, act: str = "silu", *, stream=None):
    """(dx, dw13, dw2) of ``grouped_ffn``."""
    return (_native or _c()).grouped_ffn_backward(dy, x, w13, w2, gu, offsets, act, stream)
