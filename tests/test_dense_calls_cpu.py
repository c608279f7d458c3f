"""What the dense operators' calls promise and refuse, the parts that need no
GPU."""

import os

import pytest

from host_paged_expert_gb300 import _lib


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from host_paged_expert_gb300 import build

        build.build()
    return _lib.lib()


def up(n, of):
    return -(-n // of) * of


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 65, 1021, 7826, 1 << 20])
@pytest.mark.parametrize("out", [1, 8, 9, 64, 88, 1536, 1 << 20])
@pytest.mark.parametrize("act", [0, 1, 4])
def test_linear_backward_workspace_goes_by_the_sizes(L, rows, out, act):
    """dz where it is not dy, and a row of sums for every 32 rows begun."""
    dz = up(2 * rows * up(out, 8), 256) if act or out % 8 else 0
    assert L.pe_linear_backward_workspace(rows, out, act) == dz + up(4 * -(-rows // 32) * out, 256)


def test_linear_backward_workspace_of_nothing(L):
    assert L.pe_linear_backward_workspace(0, 64, 1) == L.pe_linear_backward_workspace(4, 0, 1) == 0
    assert L.pe_linear_backward_workspace(4, 64, 5) == 0


# ---- rows past what the kernels' 32-bit counters hold

A = 1 << 20  # an aligned address that no refused call uses
MOST = (1 << 31) - (1 << 16)
N = None
CALLS = {  # at `rows` rows of 64 features, 32 outputs
    "pe_rms_norm": lambda r: (A, 64, A, 64, A, 1e-6, A, A, A, A, A, r, 64, 0, N),
    "pe_rms_norm_backward": lambda r: (A, 64, A, 64, A, 64, A, A, A, A, A, 1 << 60, r, 64, 0, N),
    "pe_linear": lambda r: (A, 64, N, A, N, A, A, 32, A, 0, A, 1, r, 64, 32, 0, N),
    "pe_linear_backward": lambda r: (A, 32, A, 64, A, A, 1, A, A, A, A, 1 << 60, r, 64, 32, 0, N),
    "pe_gated_ffn": lambda r: (A, 64, A, A, A, 64, A, A, 1, A, 1 << 60, r, 64, 32, 0, N),
    "pe_gated_ffn_backward": lambda r: (A, 64, A, 64, A, A, A, 1, A, A, A, A, 1 << 60, r, 64, 32, 0, N),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("rows", [MOST + 1, (1 << 31) - 4863, (1 << 31) - 1])
def test_too_many_rows(L, name, rows):
    assert getattr(L, name)(*CALLS[name](rows)) == _lib.PE_ERR_RANGE
    assert b"PE_MAX_ROWS" in L.pe_last_error(None)


def test_too_many_rows_from_python():
    torch = pytest.importorskip("torch")
    from host_paged_expert_gb300 import dense

    row = torch.zeros(1, 64, dtype=torch.bfloat16)
    x, w, w13, w2 = row.expand(MOST + 1, 64), row.expand(24, 64).contiguous(), row.expand(32, 64).contiguous(), torch.zeros(64, 16, dtype=row.dtype)
    for call in (lambda: dense.rms_norm(x, row[0]), lambda: dense.linear(x, w), lambda: dense.gated_ffn(x, w13, w2)):
        with pytest.raises(_lib.PEError, match="too large") as e:
            call()
        assert e.value.status == _lib.PE_ERR_RANGE
    with pytest.raises(_lib.PEError, match="want CUDA tensors"):  # the most rows are not refused
        dense.linear(row.expand(MOST, 64), w)


# ---- pointers to what is read or written one element at a time


@pytest.mark.parametrize("name,at,off", [
    ("pe_rms_norm", 9, 2), ("pe_rms_norm", 10, 1), ("pe_rms_norm", 10, 2), ("pe_rms_norm_backward", 7, 2),
    ("pe_rms_norm_backward", 9, 1), ("pe_linear_backward", 9, 1),
])
def test_misaligned_elements(L, name, at, off):
    a = list(CALLS[name](2))
    a[at] += off
    assert getattr(L, name)(*a) == _lib.PE_ERR_INVALID
    assert b"byte aligned" in L.pe_last_error(None)


@pytest.mark.parametrize("off", [(2, 0), (0, 1)])
def test_misaligned_scales(L, off):
    a = list(CALLS["pe_linear"](2))
    a[2], a[4] = A + off[0], A + off[1]
    assert L.pe_linear(*a) == _lib.PE_ERR_INVALID
    assert b"scales must be 4-byte aligned" in L.pe_last_error(None)


# ---- tensors that require gradients


def _grad_calls():
    import torch

    from host_paged_expert_gb300 import dense as D

    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    x, n, w, w13, w2, rs, y = t(4, 64), t(64), t(24, 64), t(32, 64), t(64, 16), t(4, dt=torch.float32), t(4, 24)
    return {
        "rms_norm": (D.rms_norm, (x, n, x)),
        "rms_norm_backward": (D.rms_norm_backward, (x, x, n, rs, x)),
        "linear": (D.linear, (x, w, t(24), "none", y)),
        "linear_backward": (D.linear_backward, (y, x, w, y, "silu")),
        "gated_ffn": (D.gated_ffn, (x, w13, w2, "silu", x)),
        "gated_ffn_backward": (D.gated_ffn_backward, (x, x, w13, w2, t(4, 32))),
    }


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_backward", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward"])
def test_gradients_are_not_dropped_without_a_word(name):
    torch = pytest.importorskip("torch")
    fn, args = _grad_calls()[name]
    for i, a in enumerate(args):
        if not isinstance(a, torch.Tensor):
            continue
        these = list(args)
        these[i] = a.clone().requires_grad_()
        with pytest.raises(_lib.PEError, match="requires grad") as e:
            fn(*these)
        assert e.value.status == _lib.PE_ERR_INVALID
        with torch.no_grad(), pytest.raises(_lib.PEError, match="want CUDA tensors"):
            fn(*these)


def test_inside_an_autograd_function():
    torch = pytest.importorskip("torch")
    from host_paged_expert_gb300 import dense

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            return dense.linear(x, w)

    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(24, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(_lib.PEError, match="want CUDA tensors"):  # nothing else is wrong with it
        Linear.apply(x, w)


# ---- another stream


def test_arguments_outlive_the_call_on_another_stream(monkeypatch):
    """The allocator hears of the stream that a call's tensors are used on."""
    import contextlib

    torch = pytest.importorskip("torch")
    from host_paged_expert_gb300 import dense

    seen = []

    class T(torch.Tensor):
        def record_stream(self, stream):
            seen.append((self.data_ptr(), stream))

    class Stream:
        device = torch.device("cuda:0")

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    x, w = torch.zeros(4, 64).as_subclass(T), torch.zeros(24, 64).as_subclass(T)
    s = Stream()
    assert dense._elsewhere(lambda *a: a, 0, s, (x, w, None, "none", None)) == (x, w, None, "none", None, None)
    assert seen == [(x.data_ptr(), s), (w.data_ptr(), s)]


def test_selftest_of_the_waits_refuses(L):
    import ctypes

    out = (ctypes.c_uint32 * 12)()
    call = L.pe_selftest_dense_waits
    assert [call(0, A, 1 << 20, out), call(9, None, 1 << 20, out), call(9, A, (1 << 20) - 1, out), call(9, A + 16, 1 << 20, out),
            call(9, A, 1 << 20, None)] == [_lib.PE_ERR_INVALID] * 5
