"""The native binding of the dense operators without a GPU: stand-ins for
torch's tensors and allocator go through its checks, its results and its
refusals (calls with no rows return before they touch a device)."""

import importlib
import os

import pytest
import torch

from host_paged_expert_gb300 import _lib, dense

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Fake:
    """What the binding reads of a tensor."""

    def __init__(self, shape, dtype, dev=0, stride=None):
        self.shape, self.dtype, self.device, self._dev = tuple(shape), dtype, "cuda:0", dev
        row = [1]
        for d in reversed(shape[1:]):
            row.insert(0, row[0] * d)
        self._stride = tuple(stride or row)

    def stride(self):
        return self._stride

    def get_device(self):
        return self._dev

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def m():
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(os.path.join(os.path.dirname(_lib.LIB_PATH), "_dense.so"))):
        from host_paged_expert_gb300 import build

        build.build()
    _lib.lib()
    mod = importlib.import_module("host_paged_expert_gb300._dense")
    mod.setup(lambda *shape, dtype, device: Fake(shape, dtype), lambda dev: 0, lambda: 0, BF, torch.float16, F32, F8, torch.uint8,
              dense._ACT, dense._raise, dense._elsewhere, dense.RmsNorm)
    yield mod
    dense._native = None  # the next real call sets the binding up again


X, W = Fake((0, 64), BF), Fake((64,), BF)


def test_results(m):
    r = m.rms_norm(X, W, None, 1e-6, True, True, True, None)
    assert r.sum is X and r.y.shape == (0, 64) and r.codes.dtype == F8 and r.scale.shape == (0, 1) and r.rstd.shape == (0,)
    r = m.rms_norm(X, W, X, 1e-6, False, False, False, None)
    assert r.sum is not X and r.sum.shape == (0, 64) and r.y is None and r.codes is None and r.rstd is None
    w, b = Fake((24, 64), BF), Fake((24,), BF)
    y, z = m.linear(X, w, b, "silu", Fake((0, 24), BF), None, None, None, True, None)
    assert y.shape == z.shape == (0, 24) and y.dtype == BF
    y, z = m.linear(X, w, None, "none", None, None, None, F32, True, None)
    assert z is None and y.dtype == F32
    sc = (Fake((0, 1), F32), Fake((1, 1), F32))
    assert m.linear(Fake((0, 64), F8), Fake((24, 64), F8), None, "none", None, *sc, None, False, None).dtype == BF
    assert m.linear(Fake((0, 64), F8), Fake((24, 64), F8), None, "none", Fake((0, 24), torch.float16), *sc, None, False,
                    None).dtype == torch.float16
    w13, w2 = Fake((32, 64), BF), Fake((64, 16), BF)
    y, gu = m.gated_ffn(X, w13, w2, "silu", None, True, None)
    assert y.shape == (0, 64) and gu.shape == (0, 32)
    assert m.gated_ffn(X, w13, w2, "silu", X, False, None).shape == (0, 64)


def test_refusals(m):
    x4, w = Fake((4, 64), BF), Fake((24, 64), BF)
    w13, w2 = Fake((32, 64), BF), Fake((64, 16), BF)
    none = (None, "none", None, None, None, None, False, None)
    for call in (
        lambda: m.rms_norm(X, Fake((32,), BF), None, 1e-6, True, False, False, None),
        lambda: m.rms_norm(X, W, Fake((1, 64), BF), 1e-6, True, False, False, None),
        lambda: m.rms_norm(Fake((4, 64), BF, stride=(1, 4)), W, None, 1e-6, True, False, False, None),
        lambda: m.rms_norm(Fake((4, 64), F32), Fake((64,), F32), None, 1e-6, True, False, False, None),
        lambda: m.linear(X, w, None, "tanh", None, None, None, None, False, None),
        lambda: m.linear(X, W, *none),
        lambda: m.linear(x4, Fake((24, 64), BF, stride=(1, 24)), *none),
        lambda: m.linear(Fake((4, 60), BF), Fake((24, 60), BF), *none),
        lambda: m.linear(Fake((4, 64), BF, dev=-1), w, *none),
        lambda: m.linear(x4, Fake((24, 64), BF, dev=1), *none),
        lambda: m.linear(Fake((4, 64), F8), Fake((24, 64), F8), *none),
        lambda: m.linear(Fake((1 << 31, 64), BF), w, *none),
        lambda: m.linear_backward(Fake((4, 24), BF), x4, w, None, "silu", False, None),
        lambda: m.gated_ffn(X, Fake((31, 64), BF), w2, "silu", None, False, None),
        lambda: m.gated_ffn(X, w13, W, "silu", None, False, None),
        lambda: m.gated_ffn_backward(x4, x4, w13, w2, Fake((4, 16), BF), "silu", None),
        lambda: m.rms_norm_backward(x4, x4, W, Fake((3,), F32), None, None),
    ):
        with pytest.raises(_lib.PEError):
            call()
    with pytest.raises(AttributeError):
        m.linear(1, 2, *none)
    with pytest.raises(TypeError):
        m.linear(1, 2)
