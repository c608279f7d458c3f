"""What a decoder layer runs around its attention, on the dense operators and
the paged experts.

``PagedBlock`` serves: the attention's output projection, the norm with the
residual's addition, the router, the routed experts (paged) next to a shared
expert, and the next layer's input norm with its 8-bit form in front of a
block-FP8 projection.  ``DenseBlock`` is the layer of the same stack that has
no routing (norm, gated feed-forward, residual), with its backward pass.
"""

from __future__ import annotations

import torch

from . import dense


class PagedBlock:
    """One layer from its attention's output to the next layer's projections.

    ``moe``: a PagedMoE; ``layer``: its layer.  bf16 weights: ``wo`` [H, A]
    output projection, ``norm`` [H], ``router`` [E, H], the shared expert's
    ``w13`` [2 I, H] and ``w2`` [H, I], ``next_norm`` [H].  ``wq`` [Q, H] E4M3
    with ``wq_scale`` [ceil(Q/128), ceil(H/128)]: the next layer's projections."""

    def __init__(self, moe, layer: int, *, wo, norm, router, w13, w2, next_norm, wq, wq_scale, eps: float = 1e-6):
        self.moe, self.layer, self.eps = moe, layer, eps
        self.wo, self.norm, self.router, self.w13, self.w2 = wo, norm, router, w13, w2
        self.next_norm, self.wq, self.wq_scale = next_norm, wq, wq_scale

    def forward(self, attn, residual):
        """attn [T, A], residual [T, H] -> (projections [T, Q] bf16, the new
        residual stream [T, H]).  Kernel launches only: capturable."""
        a = dense.linear(attn, self.wo)
        n = dense.rms_norm(a, self.norm, residual, self.eps)
        logits = dense.linear(n.y, self.router, out_dtype=torch.float32)
        routed = self.moe.forward(self.layer, n.y, logits)
        out = dense.gated_ffn(n.y, self.w13, self.w2, residual=routed)
        m = dense.rms_norm(out, self.next_norm, n.sum, self.eps, y=False, quant=True)
        return dense.linear(m.codes, self.wq, x_scale=m.scale, w_scale=self.wq_scale), m.sum


class DenseBlock:
    """x + gated_ffn(rms_norm(x)): a layer without routing, for training."""

    def __init__(self, *, norm, w13, w2, act: str = "silu", eps: float = 1e-6):
        self.norm, self.w13, self.w2, self.act, self.eps = norm, w13, w2, act, eps

    def forward(self, x):
        """(out, what backward needs)"""
        n = dense.rms_norm(x, self.norm, eps=self.eps, save=True)
        out, gu = dense.gated_ffn(n.y, self.w13, self.w2, act=self.act, residual=x, save=True)
        return out, (n, gu)

    def backward(self, dy, saved):
        """(dx, {"norm": , "w13": , "w2": } gradients)"""
        n, gu = saved
        dn, dw13, dw2 = dense.gated_ffn_backward(dy, n.y, self.w13, self.w2, gu, act=self.act)
        # dy also reaches x by the residual
        dx, dnorm = dense.rms_norm_backward(dn, n.sum, self.norm, n.rstd, dsum=dy)
        return dx, {"norm": dnorm, "w13": dw13, "w2": dw2}
