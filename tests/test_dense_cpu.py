"""Dense operators, the parts that need no GPU: the 64-bit forms' gradients
against differences, and what the C calls refuse before they touch a device."""

import ctypes
import os

import pytest
import torch

import dense_ref as R
from host_paged_expert_gb300 import _lib

ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]
F64 = torch.float64
R.U[F64], R.TINY[F64] = 0.0, 0.0


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=F64) * scale


def differences(f, p, h=1e-6):
    """Gradient of the number f() in p by central differences."""
    out = torch.zeros_like(p)
    for i in range(p.numel()):
        at = p.view(-1)[i].item()
        p.view(-1)[i] = at + h
        up = f()
        p.view(-1)[i] = at - h
        down = f()
        p.view(-1)[i] = at
        out.view(-1)[i] = (up - down) / (2 * h)
    return out


def near(a, b):
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), (a - b).abs().max()


@pytest.mark.parametrize("act", ACTS)
def test_activation_slopes_match_differences(act):
    z = torch.linspace(-6, 6, 241, dtype=F64) + 1e-3
    h = 1e-6
    near((R.phi(act, z + h)[0] - R.phi(act, z - h)[0]) / (2 * h), R.phi(act, z)[1])


def test_norm_gradient_matches_differences():
    x, res, w, dy, ds = rand(3, 16), rand(3, 16, seed=1), rand(16, seed=2), rand(3, 16, seed=3), rand(3, 16, seed=4)

    def loss():
        o = R.rms_norm(x, w, res, 1e-3, F64)
        return (o["raw"].v * dy).sum().item() + (o["sum"].v * ds).sum().item()

    o = R.rms_norm(x, w, res, 1e-3, F64)
    got = R.rms_norm_backward(dy, o["sum"].v, w, o["rstd"].v, ds, F64)
    near(got["dx"].v, differences(loss, x))
    near(got["dx"].v, differences(loss, res))
    near(got["dw"].v, differences(loss, w))


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_matches_differences(act):
    x, w, b, dy = rand(4, 8), rand(5, 8, seed=1), rand(5, seed=2), rand(4, 5, seed=3)

    def fwd():
        z = x @ w.t() + b
        return z, R.phi(act, z)[0]

    z = fwd()[0].clone()
    got = R.linear_backward(dy, x, w, None if act == "none" else z, act, F64)
    loss = lambda: (fwd()[1] * dy).sum().item()  # noqa: E731
    near(got["dx"].v, differences(loss, x))
    near(got["dw"].v, differences(loss, w))
    near(got["db"].v, differences(loss, b))


@pytest.mark.parametrize("act", ACTS)
def test_ffn_gradient_matches_differences(act):
    x, w13, w2, dy = rand(3, 8), rand(10, 8, seed=1), rand(8, 5, seed=2), rand(3, 8, seed=3)
    o = R.gated_ffn(x, w13, w2, act, None, F64)
    got = R.gated_ffn_backward(dy, x, w13, w2, o["gu"].v, act, F64)
    loss = lambda: (R.gated_ffn(x, w13, w2, act, None, F64)["y"].v * dy).sum().item()  # noqa: E731
    near(got["dx"].v, differences(loss, x))
    near(got["dw13"].v, differences(loss, w13))
    near(got["dw2"].v, differences(loss, w2))


# ---- refusals: every one is decided on the host, so the pointers are never used

A = 1 << 20  # an aligned address
INV, RANGE = _lib.PE_ERR_INVALID, _lib.PE_ERR_RANGE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from host_paged_expert_gb300 import build

        build.build()
    return _lib.lib()


def call(L, name, args, **change):
    a = dict(args, **change)
    st = getattr(L, name)(*a.values())
    if st:
        assert L.pe_last_error(None).decode().startswith(name), L.pe_last_error(None)
    return st


NORM = dict(x=A, x_stride=64, residual=A, residual_stride=64, weight=A, eps=1e-6, y=A, sum=A, codes=A, scales=A, rstd=A, rows=2,
            hidden=64, elem=0, stream=None)
NORM_BWD = dict(dy=A, dy_stride=64, dsum=A, dsum_stride=64, sum=A, sum_stride=64, weight=A, rstd=A, dx=A, dweight=A,
                workspace=A, workspace_bytes=1 << 30, rows=2, hidden=64, elem=0, stream=None)
LINEAR = dict(x=A, x_stride=64, x_scale=None, weight=A, w_scale=None, bias=A, residual=A, residual_stride=32, out=A, out_elem=0,
              keep=A, act=1, rows=2, in_features=64, out_features=32, elem=0, stream=None)
LINEAR_BWD = dict(dy=A, dy_stride=32, x=A, x_stride=64, weight=A, keep=A, act=1, dx=A, dweight=A, dbias=A, workspace=A,
                  workspace_bytes=1 << 30, rows=2, in_features=64, out_features=32, elem=0, stream=None)
FFN = dict(x=A, x_stride=64, w13=A, w2=A, residual=A, residual_stride=64, out=A, keep=A, act=1, workspace=A,
           workspace_bytes=1 << 30, rows=2, hidden=64, intermediate=32, elem=0, stream=None)
FFN_BWD = dict(dy=A, dy_stride=64, x=A, x_stride=64, w13=A, w2=A, keep=A, act=1, dx=A, dw13=A, dw2=A, workspace=A,
               workspace_bytes=1 << 30, rows=2, hidden=64, intermediate=32, elem=0, stream=None)


@pytest.mark.parametrize("name,args,change,status", [
    ("pe_rms_norm", NORM, dict(hidden=60), INV),
    ("pe_rms_norm", NORM, dict(hidden=0), INV),
    ("pe_rms_norm", NORM, dict(hidden=32776, x_stride=32776, residual_stride=32776), RANGE),
    ("pe_rms_norm", NORM, dict(rows=-1), INV),
    ("pe_rms_norm", NORM, dict(elem=2), INV),
    ("pe_rms_norm", NORM, dict(x=None), INV),
    ("pe_rms_norm", NORM, dict(x=A + 8), INV),
    ("pe_rms_norm", NORM, dict(x_stride=56), INV),
    ("pe_rms_norm", NORM, dict(residual_stride=68), INV),
    ("pe_rms_norm", NORM, dict(scales=None), INV),
    ("pe_rms_norm_backward", NORM_BWD, dict(workspace_bytes=8), INV),
    ("pe_rms_norm_backward", NORM_BWD, dict(rstd=None), INV),
    ("pe_rms_norm_backward", NORM_BWD, dict(dweight=None), INV),
    ("pe_rms_norm_backward", NORM_BWD, dict(dsum_stride=8), INV),
    ("pe_linear", LINEAR, dict(act=7), INV),
    ("pe_linear", LINEAR, dict(elem=2), INV),
    ("pe_linear", LINEAR, dict(out_elem=1), INV),
    ("pe_linear", LINEAR, dict(in_features=60, x_stride=64), INV),
    ("pe_linear", LINEAR, dict(x_scale=A), INV),
    ("pe_linear", LINEAR, dict(x_scale=A, w_scale=A, in_features=72, x_stride=80), INV),
    ("pe_linear", LINEAR, dict(x_stride=68), INV),
    ("pe_linear", LINEAR, dict(out_features=0), INV),
    ("pe_linear", LINEAR, dict(out_features=33, residual_stride=40), INV),
    ("pe_linear", LINEAR, dict(out_features=1 << 25, residual_stride=1 << 25), RANGE),
    ("pe_linear", LINEAR, dict(weight=A + 2), INV),
    ("pe_linear_backward", LINEAR_BWD, dict(keep=None), INV),
    ("pe_linear_backward", LINEAR_BWD, dict(workspace_bytes=100), INV),
    ("pe_linear_backward", LINEAR_BWD, dict(x=None), INV),
    ("pe_linear_backward", LINEAR_BWD, dict(dy_stride=36), INV),
    ("pe_linear_backward", LINEAR_BWD, dict(out_features=31, dy_stride=32), INV),
    ("pe_gated_ffn", FFN, dict(intermediate=20), INV),
    ("pe_gated_ffn", FFN, dict(workspace_bytes=127), INV),
    ("pe_gated_ffn", FFN, dict(workspace=None), INV),
    ("pe_gated_ffn", FFN, dict(act=-1), INV),
    ("pe_gated_ffn", FFN, dict(residual_stride=60), INV),
    ("pe_gated_ffn_backward", FFN_BWD, dict(keep=None), INV),
    ("pe_gated_ffn_backward", FFN_BWD, dict(workspace_bytes=255), INV),
    ("pe_gated_ffn_backward", FFN_BWD, dict(hidden=4), INV),
    ("pe_gated_ffn_backward", FFN_BWD, dict(dy=A + 4), INV),
])
def test_refuses(L, name, args, change, status):
    assert call(L, name, args, **change) == status


@pytest.mark.parametrize("name,args", [("pe_rms_norm", NORM), ("pe_linear", LINEAR), ("pe_gated_ffn", FFN)])
def test_zero_rows_are_a_no_op(L, name, args):
    assert call(L, name, args, rows=0) == _lib.PE_OK


def test_workspaces(L):
    assert L.pe_gated_ffn_workspace(3, 40) == 256
    assert L.pe_gated_ffn_backward_workspace(3, 40) == 512 + 256
    assert L.pe_gated_ffn_workspace(0, 40) == 0
    assert L.pe_rms_norm_backward_workspace(1, 64) == 256
    assert L.pe_linear_backward_workspace(65, 64, 0) == 768  # three chunks of column sums, no dz
    assert L.pe_linear_backward_workspace(1, 9, 0) > 0
    big = L.pe_gated_ffn_backward_workspace(1 << 20, 1 << 14)
    assert big == 6 * (1 << 34)  # past 32 bits
    assert L.pe_dense_error(ctypes.POINTER(ctypes.c_uint32)()) == INV
