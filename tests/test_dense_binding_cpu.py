"""The native binding of the dense operators without a GPU: it says what is
wrong with an argument before it asks where the tensors are, so CPU tensors
bring out each of its refusals, and a call with nothing wrong is refused for
its device alone."""

import os

import pytest
import torch

from host_paged_expert_gb300 import _lib, dense

BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(os.path.join(os.path.dirname(_lib.LIB_PATH), "_dense.so"))):
        from host_paged_expert_gb300 import build

        build.build()


def t(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


X, X0, N, W, W13, W2 = t(4, 64), t(0, 64), t(64), t(24, 64), t(32, 64), t(64, 16)
SC = dict(x_scale=t(4, 1, dt=F32), w_scale=t(1, 1, dt=F32))


@pytest.mark.parametrize("call,says", [
    (lambda: dense.rms_norm(t(4, 64, dt=F32), t(64, dt=F32)), "neither bf16 nor fp16"),
    (lambda: dense.rms_norm(t(2, 2, 64), N), "want a matrix"),
    (lambda: dense.rms_norm(t(64, 4).t(), N), "columns must be contiguous"),
    (lambda: dense.rms_norm(X, N[:32]), "weight: want contiguous BFloat16 [64]"),
    (lambda: dense.rms_norm(X, N.half()), "weight: want contiguous BFloat16 [64], got Half"),
    (lambda: dense.rms_norm(X, t(128)[::2]), "weight: want contiguous"),
    (lambda: dense.rms_norm(X, N, X[:3]), "residual: want BFloat16 [4, 64]"),
    (lambda: dense.rms_norm_backward(X, X, N, t(3, dt=F32)), "rstd: want contiguous Float [4]"),
    (lambda: dense.rms_norm_backward(X[:, :32], X, N, t(4, dt=F32)), "dy: want"),
    (lambda: dense.rms_norm_backward(X, X, N, t(4, dt=F32), X[1:]), "dsum: want"),
    (lambda: dense.linear(X, W.t()), "weight: want"),
    (lambda: dense.linear(X, N), "weight: want"),
    (lambda: dense.linear(X, t(64, 24).t()), "weight: want"),
    (lambda: dense.linear(X, W.half()), "weight: want"),
    (lambda: dense.linear(X, W, act="tanh"), "unknown activation 'tanh'"),
    (lambda: dense.linear(X, W, bias=N), "bias: want contiguous BFloat16 [24]"),
    (lambda: dense.linear(X, W, residual=X), "residual: want BFloat16 [4, 24]"),
    (lambda: dense.linear(X, W, out_dtype=HF), "out_dtype"),
    (lambda: dense.linear(X, W, **SC), "scales go with E4M3"),
    (lambda: dense.linear(X.to(F8), W.to(F8)), "need x_scale and w_scale"),
    (lambda: dense.linear(X.to(F8), W.to(F8), x_scale=t(4, 2, dt=F32), w_scale=SC["w_scale"]), "x_scale: want"),
    (lambda: dense.linear(X.to(F8), W.to(F8), residual=t(4, 24, dt=F32), **SC), "neither bf16 nor fp16"),
    (lambda: dense.linear(t(1, 8).expand(1 << 32, 8), t(4, 8)), "too large"),
    (lambda: dense.linear_backward(t(4, 24), X, W, act="silu"), "needs the z"),
    (lambda: dense.linear_backward(t(4, 24), X, W, t(4, 23), "silu"), "z: want"),
    (lambda: dense.linear_backward(t(4, 23), X, W), "dy: want"),
    (lambda: dense.gated_ffn(X, t(31, 64), W2), "w13: want contiguous BFloat16 [32, 64]"),
    (lambda: dense.gated_ffn(X, W13, W2[:, :8]), "w13: want contiguous BFloat16 [16, 64]"),
    (lambda: dense.gated_ffn(X, W13, N), "w13: want"),
    (lambda: dense.gated_ffn(X, W13, t(16, 64).t()), "w2: want"),
    (lambda: dense.gated_ffn_backward(X, X, W13, W2, t(4, 16)), "gu: want"),
    # nothing else is wrong with these
    (lambda: dense.rms_norm(X, N, X, quant=True, save=True), "want CUDA tensors"),
    (lambda: dense.rms_norm(t(4, 128)[:, :64], N), "want CUDA tensors"),
    (lambda: dense.rms_norm_backward(X, X, N, t(4, dt=F32), X), "want CUDA tensors"),
    (lambda: dense.linear(X, W, t(24), "silu", t(4, 24), out_dtype=F32, save=True), "want CUDA tensors"),
    (lambda: dense.linear(X.to(F8), W.to(F8), t(24, dt=HF), **SC), "want CUDA tensors"),
    (lambda: dense.linear(X0, W), "want CUDA tensors"),
    (lambda: dense.linear_backward(t(4, 24), X, W, t(4, 24), "silu", bias=True), "want CUDA tensors"),
    (lambda: dense.gated_ffn(X, W13, W2, "gelu", X, save=True), "want CUDA tensors"),
    (lambda: dense.gated_ffn_backward(X, X, W13, W2, t(4, 32)), "want CUDA tensors"),
])
def test_refuses(call, says):
    with pytest.raises(_lib.PEError) as e:
        call()
    assert says in str(e.value)
    assert e.value.status in (_lib.PE_ERR_INVALID, _lib.PE_ERR_RANGE)


def test_refuses_what_is_no_tensor():
    with pytest.raises(TypeError):
        dense.linear(1, 2)
    with pytest.raises(TypeError):
        dense.rms_norm(X, [1.0] * 64)
    with pytest.raises(TypeError):
        dense.linear(X, W, out_dtype="float32")
    with pytest.raises(TypeError):
        dense.rms_norm(X, N, eps="small")
    for _ in range(2000):  # the error paths hold on to nothing
        with pytest.raises(_lib.PEError):
            dense.linear(X, W, bias=N)
