"""64-bit forms of the operators of resident experts and of 4-bit products,
with bounds as in dense_ref (which see): one per element, from the places where
the operators round."""

import torch

import dense_ref as R
from dense_ref import Q, q

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
GROUP = {"int4": 128, "mxfp4": 32, "nvfp4": 16}


def values(codes, scales, fmt, ts=None):
    """[out, in] weights in float64 from packed codes and scales."""
    n, k = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(n, k).long()
    if fmt == "int4":
        v, s = (c - 8).double(), scales.double()
    else:
        v = E2M1.to(c.device)[c]
        s = torch.exp2(scales.view(torch.uint8).double() - 127) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).double() * ts.double()
    return v * s.repeat_interleave(GROUP[fmt], 1)[:, :k]


def linear_w4(x, w, bias, a, res, dt, out_dt, unpacked):
    """w in float64.  The tensor's scale and int4's group scales multiply fp32
    sums (one more rounding each); unpacked: w was rounded to dt first."""
    wq = Q(w, 2.0**-22 * w.abs())
    if unpacked:
        wq = wq.rounded(dt)
    z = R.mm(q(x), wq)
    if bias is not None:
        z = z + Q(bias.double()[None].expand_as(z.v))
    y, _ = R.act(a, z)
    if res is not None:
        y = y + q(res)
    return y.rounded(out_dt)


def route(logits, k):
    """(ids, weights as a quantity, offsets, place)"""
    t, e = logits.shape
    lg = torch.where(logits.isnan(), -torch.inf, logits.double()) + 0.0
    v, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    d = torch.where(v == v[:, :1], 0.0, v - v[:, :1])  # infinities that lead share the weight
    w = torch.exp(d)
    w = w / w.sum(1, keepdim=True)
    # exp to 2 units and its argument's rounding; a tree of five additions; a quotient
    wb = w * (2.0**-21 + 2.0**-23 * torch.where(d.isinf(), 0.0, d.abs()).clamp_max(200)) + 1e-37
    flat = ids.flatten().cpu()
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel())
    offsets = torch.zeros(e + 1, dtype=torch.int64)
    offsets[1:] = torch.bincount(flat, minlength=e).cumsum(0)
    return ids.int(), Q(w, wb), offsets.int().to(logits.device), place.view(t, k).int().to(logits.device)


def route_backward(dw, w, ids, e):
    w, dw = w.double(), dw.double()
    dot = (w * dw).sum(1, keepdim=True)
    dotb = 2.0**-21 * (w * dw).abs().sum(1, keepdim=True)
    g = w * (dw - dot)
    gb = w * dotb + 2.0**-22 * w * (dw.abs() + dot.abs())
    z = torch.zeros(w.shape[0], e, dtype=torch.float64, device=w.device)
    return Q(z.scatter_add(1, ids.long(), g), z.scatter_add(1, ids.long(), gb) + 1e-37)


def combine(y, place, w, res, dt):
    k = place.shape[1]
    there = (place >= 0) & (place < y.shape[0])
    if y.shape[0]:
        rows = torch.where(there[:, :, None], y[place.long().clamp(0, y.shape[0] - 1)].double(), 0.0)
    else:
        rows = torch.zeros(*place.shape, y.shape[1], dtype=torch.float64, device=y.device)
    p = rows * (w.double() if w is not None else torch.ones_like(place, dtype=torch.float64))[:, :, None]
    v, a = p.sum(1), p.abs().sum(1)
    if res is not None:
        v, a = v + res.double(), a + res.double().abs()
    return Q(v, (k + 1) * 2.0**-24 * a).rounded(dt)


def combine_backward(dout, y, place, w, dt):
    """(dy of the rows that entries name, dweights): dy as {row: quantity}"""
    d = dout.double()
    p = w.double()[:, :, None] * d[:, None]
    dy = Q(p, 2.0**-24 * p.abs()).rounded(dt)
    t = y[place.long()].double() * d[:, None]
    return dy, Q(t.sum(2), R.acc(y.shape[1]) * t.abs().sum(2) + 1e-37)


def _groups(offsets):
    o = offsets.tolist()
    return [slice(a, b) for a, b in zip(o, o[1:])]


def _cat(parts):
    return Q(torch.cat([p.v for p in parts]), torch.cat([p.b for p in parts]))


def _stack(parts):
    return Q(torch.stack([p.v for p in parts]), torch.stack([p.b for p in parts]))


def grouped_linear(x, w, offsets, dt):
    return _cat([R.mm(q(x[s]), q(w[g])) for g, s in enumerate(_groups(offsets))]).rounded(dt)


def grouped_linear_backward(dy, x, w, offsets, dt):
    gs = list(enumerate(_groups(offsets)))
    return {"dx": _cat([R.mm(q(dy[s]), q(w[g]).t()) for g, s in gs]).rounded(dt),
            "dw": _stack([R.mm(q(dy[s]).t(), q(x[s]).t()) for g, s in gs]).rounded(dt)}


def grouped_ffn(x, w13, w2, offsets, a, dt):
    """gu is kept in fp32."""
    gs = list(enumerate(_groups(offsets)))
    return {"y": _cat([R.gated_ffn(x[s], w13[g], w2[g], a, None, dt)["y"] for g, s in gs]),
            "gu": _cat([R.mm(q(x[s]), q(w13[g])) for g, s in gs]).rounded(torch.float32)}


def grouped_ffn_backward(dy, x, w13, w2, gu, offsets, a, dt):
    parts = [R.gated_ffn_backward(dy[s], x[s], w13[g], w2[g], gu[s], a, dt) for g, s in enumerate(_groups(offsets))]
    return {"dx": _cat([p["dx"] for p in parts]), "dw13": _stack([p["dw13"] for p in parts]), "dw2": _stack([p["dw2"] for p in parts])}
