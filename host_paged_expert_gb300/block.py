"""What a decoder layer runs around its attention, on the dense operators and
the paged experts.

``PagedBlock`` serves: the attention's output projection, the norm with the
residual's addition, the router, the routed experts (paged) next to a shared
expert, and the next layer's input norm with its 8-bit form in front of a
block-FP8 projection.  ``DenseBlock`` is the layer of the same stack that has
no routing (norm, gated feed-forward, residual), with its backward pass.
``ExpertBlock`` is the layer with routing whose experts are resident: it trains
what ``PagedBlock`` serves.
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


class ExpertBlock:
    """x + the weighted sum of its tokens' experts (rms_norm(x)): a layer whose
    routed experts are resident, for training.

    bf16 or fp16: ``norm`` [H], ``router`` [E, H], ``w13`` [E, 2 I, H], ``w2``
    [E, H, I].  The router's logits are fp32; its choice has no gradient, its
    weights do."""

    def __init__(self, *, norm, router, w13, w2, top_k: int, act: str = "silu", eps: float = 1e-6):
        self.norm, self.router, self.w13, self.w2, self.top_k, self.act, self.eps = norm, router, w13, w2, top_k, act, eps

    def forward(self, x):
        """(out, what backward needs).  Kernel launches only: capturable."""
        n = dense.rms_norm(x, self.norm, eps=self.eps, save=True)
        r = dense.route(dense.linear(n.y, self.router, out_dtype=torch.float32), self.top_k)
        rows = dense.expand_rows(n.y, r.place)
        y, gu = dense.grouped_ffn(rows, self.w13, self.w2, r.offsets, self.act, save=True)
        return dense.combine_rows(y, r.place, r.weights, x), (n, r, rows, gu, y)

    def backward(self, dout, saved):
        """(dx, {"norm": , "router": , "w13": , "w2": } gradients)"""
        n, r, rows, gu, y = saved
        dy, dweights = dense.combine_rows_backward(dout, y, r.place, r.weights)
        drows, dw13, dw2 = dense.grouped_ffn_backward(dy, rows, self.w13, self.w2, gu, r.offsets, self.act)
        # the logits' gradient in the type that the product's MMA takes
        dlogits = dense.route_backward(dweights, r.weights, r.ids, self.router.shape[0]).to(n.y.dtype)
        dn, drouter, _ = dense.linear_backward(dlogits, n.y, self.router)
        dn = dense.combine_rows(drows, r.place, residual=dn)
        dx, dnorm = dense.rms_norm_backward(dn, n.sum, self.norm, n.rstd, dsum=dout)
        return dx, {"norm": dnorm, "router": drouter, "w13": dw13, "w2": dw2}
