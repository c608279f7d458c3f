"""64-bit forms of the dense operators with bounds on what a kernel that
follows the formulas may be off by.

A quantity is a pair (value, bound): the value in float64 and, per element,
how far a computation may be from it that
  * takes 16-bit operands as they are and accumulates products in fp32
    (rounded or truncated at each addition: 2^-23 relative each; over K terms
    8 sqrt(K) 2^-23 of the sum of the products' magnitudes, eight standard
    deviations of independent errors),
  * evaluates activations to 4e-6 relative to the larger of 1 and |z|,
  * rounds to 16 bits (half a unit in the last place: 2^-8 relative for bf16,
    2^-11 for fp16 and 2^-25 absolute where fp16 is subnormal) at the places
    that the operators name, and nowhere else.
Bounds pass through products and activations by their slopes.
"""

import math

import torch

U = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0**-24, torch.float32: 1e-38}
GROUP = 128


class Q:
    def __init__(self, v, b=None):
        self.v = v
        self.b = torch.zeros_like(v) if b is None else b

    def t(self):
        return Q(self.v.t(), self.b.t())

    def __add__(self, o):
        return Q(self.v + o.v, self.b + o.b + 2.0**-23 * (self.v + o.v).abs())

    def __mul__(self, o):
        v = self.v * o.v
        return Q(v, self.b * o.v.abs() + o.b * self.v.abs() + self.b * o.b + 2.0**-23 * v.abs())

    def rounded(self, dt):
        return Q(self.v, self.b + U[dt] * (self.v.abs() + self.b) + TINY[dt])


def q(t):
    return Q(t.double())


def acc(k):
    return 8 * math.sqrt(max(k, 1)) * 2.0**-23


def mm(a, b):
    """a b^T over the last axis of both."""
    k = a.v.shape[1]
    av, bv = a.v.abs(), b.v.abs()
    return Q(a.v @ b.v.t(), a.b @ (bv + b.b).t() + av @ b.b.t() + acc(k) * (av @ bv.t()))


def cat(a, b):
    return Q(torch.cat([a.v, b.v], 1), torch.cat([a.b, b.b], 1))


def phi(act, z):
    """(act(z), act'(z)) of a float64 tensor."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z**3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def act(name, z):
    """(act, act') as quantities: |act'| <= 1.2 and |act''| <= 1.2 for the
    smooth ones; relu's slope jumps where z may have either sign."""
    v, d = phi(name, z.v)
    if name == "none":
        return Q(v, z.b), Q(d)
    if name == "relu":
        return Q(v, z.b), Q(d, (z.v.abs() <= z.b).double())
    e = 4e-6 * z.v.abs().clamp_min(1)
    return Q(v, 1.2 * z.b + e), Q(d, 1.2 * z.b + e)


def rms_norm(x, w, res, eps, dt):
    s = q(x) + q(res) if res is not None else q(x)
    h = s.v.shape[1]
    r = (s.v.square().mean(1, keepdim=True) + eps).rsqrt()
    # the mean's terms are positive: its relative error halves in r
    rb = r * (acc(h) + 2.0**-21)
    y = s * Q(r, rb) * q(w)
    return {"y": y.rounded(dt), "sum": s.rounded(dt), "rstd": Q(r[:, 0], rb[:, 0]), "raw": y}


def scales(y):
    """The 8-bit form's scales (value, bound) from the unrounded y."""
    out = []
    for p, b in zip(y.v.split(GROUP, 1), y.b.split(GROUP, 1)):
        a = p.abs().amax(1)
        out.append((torch.where(a > 0, a / 448, torch.ones_like(a)), b.amax(1) / 448 + 2.0**-22 * a / 448))
    return Q(torch.stack([v for v, _ in out], 1), torch.stack([b for _, b in out], 1))


def rms_norm_backward(dy, s, w, rstd, dsum, dt):
    """From the 16-bit sum and the given rstd, as the kernel has them."""
    rows, h = s.shape
    r = Q(rstd.double()[:, None])
    xh, g = q(s) * r, q(dy) * q(w)
    dot = (g.v * xh.v).sum(1, keepdim=True) / h
    dotb = ((acc(h) + 2.0**-21) * (g.v * xh.v).abs().sum(1, keepdim=True)) / h
    dx = (g + Q(-1 * xh.v, xh.b) * Q(dot, dotb)) * r
    if dsum is not None:
        dx = dx + q(dsum)
    p = q(dy) * xh
    dw = Q(p.v.sum(0), p.b.sum(0) + acc(rows) * p.v.abs().sum(0))
    return {"dx": dx.rounded(dt), "dw": dw.rounded(dt)}


def spread(s, rows, r, c):
    return s.repeat_interleave(rows, 0)[:r].repeat_interleave(GROUP, 1)[:, :c]


def linear(x, w, bias, a, res, dt, out_dt, xs=None, ws=None):
    xq, wq = q(x.float()), q(w.float())
    if xs is not None:
        xq, wq = xq * Q(spread(xs.double(), 1, *x.shape)), wq * Q(spread(ws.double(), GROUP, *w.shape))
    z = mm(xq, wq)
    if bias is not None:
        z = z + Q(bias.double()[None].expand_as(z.v))
    y, _ = act(a, z)
    if res is not None:
        y = y + q(res)
    return {"y": y.rounded(out_dt), "z": z.rounded(dt)}


def linear_backward(dy, x, w, z, a, dt):
    """From the 16-bit z that was kept (None for act "none")."""
    raw = q(dy) if z is None else q(dy) * act(a, q(z))[1]
    dz = raw if z is None else raw.rounded(dt)
    db = Q(raw.v.sum(0), raw.b.sum(0) + acc(dy.shape[0]) * raw.v.abs().sum(0))
    return {"dx": mm(dz, q(w).t()).rounded(dt), "dw": mm(dz.t(), q(x).t()).rounded(dt), "db": db.rounded(dt)}


def gated_ffn(x, w13, w2, a, res, dt):
    i = w2.shape[1]
    gu = mm(q(x), q(w13))
    g, u = Q(gu.v[:, :i], gu.b[:, :i]), Q(gu.v[:, i:], gu.b[:, i:])
    h = (act(a, g)[0] * u).rounded(dt)
    y = mm(h, q(w2))
    if res is not None:
        y = y + q(res)
    return {"y": y.rounded(dt), "gu": gu.rounded(dt)}


def gated_ffn_backward(dy, x, w13, w2, gu, a, dt):
    """From the 16-bit gate and up products that were kept."""
    i = w2.shape[1]
    g, u = q(gu[:, :i]), q(gu[:, i:])
    f, d = act(a, g)
    h = (f * u).rounded(dt)
    dh = mm(q(dy), q(w2).t())
    dgu = cat((dh * u * d).rounded(dt), (dh * f).rounded(dt))
    return {"dx": mm(dgu, q(w13).t()).rounded(dt), "dw13": mm(dgu.t(), q(x).t()).rounded(dt),
            "dw2": mm(q(dy).t(), h.t()).rounded(dt)}


def check(got, want, name):
    """Every element within its bound; returns the worst share of it."""
    g = got.double()
    assert g.shape == want.v.shape, (name, g.shape, want.v.shape)
    if not g.numel():
        return 0.0
    assert torch.isfinite(g).all(), f"{name}: not finite"
    share = ((g - want.v).abs() / want.b.clamp_min(1e-300)).max().item()
    assert share <= 1, f"{name}: {share:.2f} of the bound"
    return share
