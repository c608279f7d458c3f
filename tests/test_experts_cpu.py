"""What the operators of resident experts and of 4-bit products refuse, and
their workspaces, without a GPU (as test_dense_binding_cpu, which see)."""

import os

import pytest

torch = pytest.importorskip("torch")

from host_paged_expert_gb300 import _lib, dense  # noqa: E402

BF, HF, F32, I32, U8, F8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def L():
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(os.path.join(os.path.dirname(_lib.LIB_PATH), "_dense.so"))):
        from host_paged_expert_gb300 import build

        build.build()
    return _lib.lib()


def t(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


X, LG, IDS, W = t(4, 64), t(4, 16, dt=F32), t(4, 2, dt=I32), t(4, 2, dt=F32)
GW, OFF, W13, W2, GU = t(3, 24, 64), t(4, dt=I32), t(3, 32, 64), t(3, 64, 16), t(4, 32, dt=F32)
C, S4, SM, SN, TS = t(24, 32, dt=U8), t(24, 1, dt=HF), t(24, 2, dt=U8), t(24, 4, dt=F8), t(1, dt=F32)


@pytest.mark.parametrize("call,says", [
    (lambda: dense.route(X, 2), "logits: want Float"),
    (lambda: dense.route(LG[0], 2), "want a matrix"),
    (lambda: dense.route(LG, 0), "top_k: 0 of 16"),
    (lambda: dense.route(LG, 17), "top_k: 17 of 16"),
    (lambda: dense.route(LG.t(), 2), "columns must be contiguous"),
    (lambda: dense.route_backward(W[:3], W, IDS, 16), "dweights: want"),
    (lambda: dense.route_backward(W, W, IDS.long(), 16), "ids: want contiguous Int"),
    (lambda: dense.route_backward(W, W, IDS, 1), "experts: 1 for a choice of 2"),
    (lambda: dense.route_backward(W, W, IDS, 1 << 40), "too large"),
    (lambda: dense.expand_rows(X, IDS[:3]), "place: want"),
    (lambda: dense.expand_rows(X, IDS.long()), "place: want contiguous Int"),
    (lambda: dense.expand_rows(X, IDS, -1), "rows: -1"),
    (lambda: dense.expand_rows(X, IDS[:, :0]), "no entries"),
    (lambda: dense.expand_rows(X.float(), IDS), "neither bf16 nor fp16"),
    (lambda: dense.combine_rows(X, IDS, W[:, :1]), "weights: want"),
    (lambda: dense.combine_rows(X, IDS, W.half()), "weights: want contiguous Float"),
    (lambda: dense.combine_rows(X, IDS, W, X[:3]), "residual: want"),
    (lambda: dense.combine_rows(X, t(4, 4, dt=I32)[:, ::2]), "place: want contiguous"),
    (lambda: dense.combine_rows_backward(X[:3], X, IDS, W), "dout: want"),
    (lambda: dense.grouped_linear(X, GW[0], OFF), "weight: want contiguous BFloat16"),
    (lambda: dense.grouped_linear(X, GW.half(), OFF), "weight: want"),
    (lambda: dense.grouped_linear(X, GW[:, ::2], OFF), "not contiguous"),
    (lambda: dense.grouped_linear(X, t(3, 24, 56), OFF), "weight: want contiguous BFloat16 [3, 24, 64]"),
    (lambda: dense.grouped_linear(X, GW, OFF[:3]), "offsets: want contiguous Int [4]"),
    (lambda: dense.grouped_linear(X, GW, OFF.long()), "offsets: want"),
    (lambda: dense.grouped_linear(X, GW[:0], OFF), "no groups"),
    (lambda: dense.grouped_linear_backward(t(4, 23), X, GW, OFF), "dy: want"),
    (lambda: dense.grouped_ffn(X, t(3, 30, 64), W2, OFF), "w13: want"),
    (lambda: dense.grouped_ffn(X, W13, t(3, 56, 16), OFF), "w2: want"),
    (lambda: dense.grouped_ffn(X, W13[:2], W2, OFF), "w13: want"),
    (lambda: dense.grouped_ffn(X, W13, W2, OFF, "tanh"), "unknown activation"),
    (lambda: dense.grouped_ffn_backward(X, X, W13, W2, t(4, 32), OFF), "gu: want"),
    (lambda: dense.linear_w4(X, C, S4, "int8"), "unknown format 'int8'"),
    (lambda: dense.linear_w4(t(4, 48), t(24, 24, dt=U8), S4, "int4"), "multiple of 32"),
    (lambda: dense.linear_w4(X, C[:, :16], S4, "int4"), "codes: want contiguous Byte [24, 32]"),
    (lambda: dense.linear_w4(X, C, S4.float(), "int4"), "scales: want contiguous Half [24, 1]"),
    (lambda: dense.linear_w4(X, C, SM, "int4"), "scales: want contiguous Half [24, 1]"),
    (lambda: dense.linear_w4(X, C, SM[:, :1], "mxfp4"), "scales: want"),
    (lambda: dense.linear_w4(X, C, SN, "mxfp4"), "scales: want"),
    (lambda: dense.linear_w4(X, C, SN, "nvfp4"), "nvfp4 with tensor_scale"),
    (lambda: dense.linear_w4(X, C, S4, "int4", tensor_scale=TS), "tensor_scale goes with nvfp4"),
    (lambda: dense.linear_w4(X, C, SN, "nvfp4", tensor_scale=t(2, dt=F32)), "tensor_scale: want"),
    (lambda: dense.linear_w4(X, C, S4, "int4", t(24, dt=HF)), "bias: want"),
    (lambda: dense.linear_w4(X, C, S4, "int4", residual=X), "residual: want"),
    (lambda: dense.linear_w4(X, C, S4, "int4", out_dtype=HF), "out_dtype"),
    # nothing else is wrong with these
    (lambda: dense.route(LG, 2), "want CUDA tensors"),
    (lambda: dense.route(t(4, 20, dt=F32)[:, :16], 2), "want CUDA tensors"),
    (lambda: dense.route_backward(W, W, IDS, 16), "want CUDA tensors"),
    (lambda: dense.expand_rows(X, IDS), "want CUDA tensors"),
    (lambda: dense.expand_rows(X, IDS, 3), "want CUDA tensors"),
    (lambda: dense.combine_rows(X, IDS, W, X), "want CUDA tensors"),
    (lambda: dense.combine_rows_backward(X, t(8, 64), IDS, W), "want CUDA tensors"),
    (lambda: dense.grouped_linear(X, GW, OFF), "want CUDA tensors"),
    (lambda: dense.grouped_linear_backward(t(4, 24), X, GW, OFF), "want CUDA tensors"),
    (lambda: dense.grouped_ffn(X, W13, W2, OFF, save=True), "want CUDA tensors"),
    (lambda: dense.grouped_ffn_backward(X, X, W13, W2, GU, OFF), "want CUDA tensors"),
    (lambda: dense.linear_w4(X, C, S4, "int4", t(24), "silu", t(4, 24), out_dtype=F32), "want CUDA tensors"),
    (lambda: dense.linear_w4(X, C, SM, "mxfp4"), "want CUDA tensors"),
    (lambda: dense.linear_w4(X, C, SN, "nvfp4", tensor_scale=TS), "want CUDA tensors"),
])
def test_refuses(call, says):
    with pytest.raises(_lib.PEError) as e:
        call()
    assert says in str(e.value)
    assert e.value.status in (_lib.PE_ERR_INVALID, _lib.PE_ERR_RANGE)


@pytest.mark.parametrize("call", [
    lambda g: dense.route(g(LG), 2), lambda g: dense.route_backward(g(W), W, IDS, 16), lambda g: dense.expand_rows(g(X), IDS),
    lambda g: dense.combine_rows(X, IDS, g(W)), lambda g: dense.combine_rows_backward(X, g(t(8, 64)), IDS, W),
    lambda g: dense.grouped_linear(X, g(GW), OFF), lambda g: dense.grouped_linear_backward(g(t(4, 24)), X, GW, OFF),
    lambda g: dense.grouped_ffn(X, W13, g(W2), OFF), lambda g: dense.grouped_ffn_backward(X, X, W13, W2, g(GU), OFF),
    lambda g: dense.linear_w4(g(X), C, S4, "int4"),
])
def test_gradients_are_not_dropped_without_a_word(call):
    grad = lambda a: a.clone().requires_grad_()  # noqa: E731
    with pytest.raises(_lib.PEError, match="requires grad"):
        call(grad)
    with torch.no_grad(), pytest.raises(_lib.PEError, match="want CUDA tensors"):
        call(grad)


# ---- the C calls: an aligned address that no refused call uses

A, N = 1 << 20, None
MOST = (1 << 31) - (1 << 16)
GOOD = {  # name: arguments at 4 tokens or rows (40 for pe_route, which then needs a workspace)
    "pe_route": (A, 16, A, A, A, A, A, 1 << 40, 40, 2, 16, N),
    "pe_route_backward": (A, A, A, A, 4, 2, 16, N),
    "pe_expand_rows": (A, 64, A, A, 4, 2, 8, 64, 0, N),
    "pe_combine_rows": (A, 64, A, A, A, 64, A, 4, 2, 8, 64, 0, N),
    "pe_combine_rows_backward": (A, 64, A, 64, A, A, A, A, 4, 2, 8, 64, 0, N),
    "pe_grouped_linear": (A, 64, A, A, A, 4, 3, 64, 24, 0, N),
    "pe_grouped_linear_backward": (A, 24, A, 64, A, A, A, A, 4, 3, 64, 24, 0, N),
    "pe_grouped_ffn": (A, 64, A, A, A, A, A, 1, A, 1 << 40, 4, 3, 64, 16, 0, N),
    "pe_grouped_ffn_backward": (A, 64, A, 64, A, A, A, A, 1, A, A, A, A, 1 << 40, 4, 3, 64, 16, 0, N),
    "pe_linear_four_bit": (A, 64, A, A, A, 4, A, A, 24, A, 0, 1, A, 1 << 40, 4, 64, 24, 0, N),
}
INVALID, RANGE = _lib.PE_ERR_INVALID, _lib.PE_ERR_RANGE


@pytest.mark.parametrize("name,at,value,status", [
    # NULL where something is read or written
    *[("pe_route", i, N, INVALID) for i in (0, 2, 3, 4, 5, 6)], *[("pe_route_backward", i, N, INVALID) for i in range(4)],
    *[("pe_expand_rows", i, N, INVALID) for i in (0, 2, 3)], *[("pe_combine_rows", i, N, INVALID) for i in (0, 2, 6)],
    *[("pe_combine_rows_backward", i, N, INVALID) for i in (0, 2, 4, 5, 6)], *[("pe_grouped_linear", i, N, INVALID) for i in (0, 2, 3, 4)],
    *[("pe_grouped_linear_backward", i, N, INVALID) for i in (0, 2, 4, 5)], *[("pe_grouped_ffn", i, N, INVALID) for i in (0, 2, 3, 4, 5, 8)],
    *[("pe_grouped_ffn_backward", i, N, INVALID) for i in (0, 2, 4, 5, 6, 7, 12)],
    *[("pe_linear_four_bit", i, N, INVALID) for i in (0, 2, 3, 4, 9)],
    # misaligned
    ("pe_route", 0, A + 2, INVALID), ("pe_route", 5, A + 1, INVALID), ("pe_route", 6, A + 4, INVALID), ("pe_route_backward", 3, A + 4, INVALID),
    ("pe_expand_rows", 0, A + 2, INVALID), ("pe_expand_rows", 2, A + 2, INVALID), ("pe_combine_rows", 3, A + 1, INVALID), ("pe_combine_rows", 4, A + 8, INVALID),
    ("pe_combine_rows_backward", 7, A + 2, INVALID), ("pe_grouped_linear", 3, A + 2, INVALID), ("pe_grouped_linear", 4, A + 8, INVALID),
    ("pe_grouped_linear_backward", 7, A + 2, INVALID), ("pe_grouped_ffn", 6, A + 8, INVALID), ("pe_grouped_ffn_backward", 10, A + 8, INVALID),
    ("pe_linear_four_bit", 2, A + 8, INVALID), ("pe_linear_four_bit", 3, A + 2, INVALID), ("pe_linear_four_bit", 4, A + 2, INVALID),
    # pitches
    ("pe_route", 1, 15, INVALID), ("pe_expand_rows", 1, 60, INVALID), ("pe_expand_rows", 1, 68, INVALID), ("pe_combine_rows", 1, 60, INVALID),
    ("pe_combine_rows", 5, 60, INVALID), ("pe_combine_rows_backward", 3, 60, INVALID), ("pe_grouped_linear", 1, 60, INVALID),
    ("pe_grouped_linear_backward", 1, 20, INVALID), ("pe_grouped_ffn", 1, 60, INVALID), ("pe_linear_four_bit", 1, 60, INVALID),
    ("pe_linear_four_bit", 8, 20, INVALID),
    # sizes
    ("pe_route", 9, 17, INVALID), ("pe_route", 9, 0, INVALID), ("pe_route", 10, 1025, RANGE), ("pe_route", 8, MOST + 1, RANGE), ("pe_route", 8, -1, INVALID),
    ("pe_route_backward", 6, 1025, RANGE), ("pe_expand_rows", 5, 0, INVALID), ("pe_expand_rows", 7, 60, INVALID), ("pe_expand_rows", 6, -1, INVALID),
    ("pe_expand_rows", 5, 1 << 30, RANGE), ("pe_combine_rows", 9, MOST + 1, RANGE), ("pe_combine_rows", 10, (1 << 24) + 8, RANGE),
    ("pe_grouped_linear", 5, MOST + 1, RANGE), ("pe_grouped_linear", 6, 0, INVALID), ("pe_grouped_linear", 6, 1025, RANGE), ("pe_grouped_linear", 7, 60, INVALID),
    ("pe_grouped_linear", 8, 20, INVALID), ("pe_grouped_linear_backward", 8, MOST + 1, RANGE), ("pe_grouped_ffn", 10, -1, INVALID), ("pe_grouped_ffn", 13, 20, INVALID),
    ("pe_grouped_ffn_backward", 14, MOST + 1, RANGE), ("pe_linear_four_bit", 14, MOST + 1, RANGE), ("pe_linear_four_bit", 15, 48, INVALID),
    ("pe_linear_four_bit", 15, 0, INVALID), ("pe_linear_four_bit", 16, 0, INVALID), ("pe_linear_four_bit", 16, (1 << 24) + 1, RANGE),
    # types, activations, formats
    ("pe_expand_rows", 8, 2, INVALID), ("pe_combine_rows", 11, 2, INVALID), ("pe_grouped_linear", 9, 2, INVALID), ("pe_grouped_ffn", 7, 5, INVALID),
    ("pe_grouped_ffn_backward", 8, -1, INVALID), ("pe_linear_four_bit", 17, 2, INVALID), ("pe_linear_four_bit", 10, 1, INVALID), ("pe_linear_four_bit", 11, 9, INVALID),
    ("pe_linear_four_bit", 5, 0, _lib.PE_ERR_UNSUPPORTED_DTYPE), ("pe_linear_four_bit", 5, 1, _lib.PE_ERR_UNSUPPORTED_DTYPE),
    # workspaces
    ("pe_route", 7, 0, INVALID), ("pe_grouped_ffn", 9, 100, INVALID), ("pe_grouped_ffn_backward", 13, 100, INVALID),
])
def test_c_calls_refuse(L, name, at, value, status):
    a = list(GOOD[name])
    a[at] = value
    assert getattr(L, name)(*a) == status
    assert L.pe_last_error(None).decode().startswith(name)


def test_workspaces(L):
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert L.pe_linear_four_bit_workspace(128, 4096, 2048) == 0
    assert L.pe_linear_four_bit_workspace(129, 4096, 2048) == up(2 * 4096 * 2048)
    assert L.pe_grouped_ffn_workspace(100, 40) == up(2 * 100 * 40)
    assert L.pe_grouped_ffn_backward_workspace(100, 40) == up(4 * 100 * 40) + up(2 * 100 * 40)
    # never more chunks of tokens than a launch has blocks for
    assert L.pe_route_workspace(32, 128) == 0  # one block
    for tokens in (33, 64, 5000, 1 << 20, 1 << 30):
        assert 0 < L.pe_route_workspace(tokens, 128) <= up(152 * 128 * 4)
    assert L.pe_route_workspace(0, 128) == L.pe_grouped_ffn_workspace(0, 8) == 0


def test_selftest_of_the_waits_refuses(L):
    import ctypes

    out = (ctypes.c_uint32 * 12)()
    call = L.pe_selftest_experts_waits
    assert [call(0, A, 4 << 20, out), call(9, None, 4 << 20, out), call(9, A, (4 << 20) - 1, out), call(9, A + 16, 4 << 20, out),
            call(9, A, 4 << 20, None)] == [INVALID] * 5
