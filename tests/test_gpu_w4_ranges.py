"""Weights of linear products in 4 bits at the ends of their types' ranges, on
the GPU (tests/experts_ref.py holds the values in 64 bits)."""

import pytest

torch = pytest.importorskip("torch")

import experts_ref as X  # noqa: E402
from test_gpu_experts import F32, HF, D, ints  # noqa: E402, F401

pytestmark = pytest.mark.gpu


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
