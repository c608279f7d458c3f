"""Weights of linear products in 4 bits at the ends of their types' ranges, on
the GPU (tests/experts_ref.py holds the values in 64 bits)."""

import pytest

torch = pytest.importorskip("torch")

import dense_ref as R  # noqa: E402
import experts_ref as X  # noqa: E402
from test_gpu_experts import BF, F32, FMTS, HF, D, ints, rand, weights  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 8, 16, 17, 64, 96, 128])
def test_every_mxfp4_scale_with_fp16(D, rows):  # noqa: F811
    """Rows of the identity pick single weights out of groups whose scales lie
    as far apart as E8M0 goes: each is what fp32 holds of it, and a scale beyond
    fp16 meets inputs of zero without a word."""
    k, n = 160, 41
    codes, s = ints(0, 256, (n, k // 2)), ints(0, 255, (n, k // 32), seed=1)
    s[:8] = torch.arange(136, 144, device="cuda")[:, None]  # about where fp16 ends
    s[8:16] = torch.arange(100, 108, device="cuda")[:, None]  # and begins
    want = X.values(codes, s, "mxfp4").t().float()  # the nearest, infinity past the largest
    eye = torch.eye(k, device="cuda", dtype=HF)
    for a in range(0, k, rows):
        a = min(a, k - rows)
        assert torch.equal(D.linear_w4(eye[a : a + rows], codes, s, "mxfp4", out_dtype=F32), want[a : a + rows])


@pytest.mark.parametrize("rows,k,n", [(3, 224, 40), (16, 1056, 72), (40, 1056, 72), (128, 352, 200)])
def test_large_and_small_mxfp4_scales_with_fp16(D, rows, k, n):  # noqa: F811
    for lo, hi in ((141, 160), (80, 104)):
        codes, s = ints(0, 256, (n, k // 2)), ints(lo, hi, (n, k // 32), seed=lo)
        x = rand(rows, k, dt=HF)
        y = D.linear_w4(x, codes, s, "mxfp4", out_dtype=F32)
        R.check(y, X.linear_w4(x, X.values(codes, s, "mxfp4"), None, "none", None, HF, F32, False), "y")


def test_nan_scales_with_fp16(D):  # noqa: F811
    k, n = 160, 24
    for fmt in FMTS:
        c, s, ts = weights(fmt, n, k)
        s = s.clone()
        if fmt == "int4":
            s[5, 1] = float("nan")
        else:
            s.view(torch.uint8)[5, 4] = 255 if fmt == "mxfp4" else 127
        for rows in (3, 16, 40, 150):
            y = D.linear_w4(rand(rows, k, dt=HF), c, s, fmt, tensor_scale=ts)
            assert y[:, 5].isnan().all() and torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all()


def test_mxfp4_weights_unpacked_to_fp16(D):  # noqa: F811
    """Above 128 rows weights are what fp16 holds of code times scale."""
    k, n = 160, 48
    codes, e = ints(0, 256, (n, k // 2)), ints(100, 141, (n, k // 32), seed=1)
    small = codes & 0xBB  # magnitudes up to 1.5
    codes[:12], e[:12] = small[:12], 142
    codes[12:24], e[12:24] = small[12:24] & 0x99, 143  # and to 0.5
    want = X.values(codes, e, "mxfp4").half().t().float()
    assert torch.isfinite(want).all()
    assert torch.equal(D.linear_w4(torch.eye(k, device="cuda", dtype=HF), codes, e, "mxfp4", out_dtype=F32), want)


@pytest.mark.parametrize("rows", [128, 129, 300, 1024])
@pytest.mark.parametrize("k,n", [(1056, 200), (96, 77), (512, 2048)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_tensor_scales_of_any_size(D, rows, k, n, dt):  # noqa: F811
    """They multiply sums: no weight is rounded, at any number of rows."""
    codes, s, _ = weights("nvfp4", n, k)
    x, b, res = rand(rows, k, dt=dt), rand(n, seed=2, dt=dt), rand(rows, n, seed=3, dt=dt)
    for scale in (2.0**-20, 0.0123, 2.0**18):
        ts = torch.full((1,), scale, device="cuda")
        w = X.values(codes, s, "nvfp4", ts)
        y = D.linear_w4(x, codes, s, "nvfp4", tensor_scale=ts, out_dtype=F32)
        R.check(y, X.linear_w4(x, w, None, "none", None, dt, F32, False), f"y at {scale}")
    ts = torch.full((1,), 0.0123, device="cuda")
    w = X.values(codes, s, "nvfp4", ts)
    for act in ("none", "silu"):
        y = D.linear_w4(x, codes, s, "nvfp4", b, act, res, tensor_scale=ts)
        R.check(y, X.linear_w4(x, w, b, act, res, dt, dt, False), act)
