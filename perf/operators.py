"""Cases of the dense operators around a paged MoE layer, and what they compute.

A decoder layer of a mixture-of-experts model runs three more things next to
its routed experts, and these are the operators measured here:

* ``norm``    s = x + residual, y = s * rsqrt(mean(s^2) + eps) * weight, with y
              also as E4M3 codes with one fp32 scale per 128 features of a row;
              its backward pass.
* ``linear``  act(x W^T + bias) + residual: the attention's output projection
              (residual), a router's logits (fp32 out), W8A8 block-FP8
              products (x as E4M3 codes with a scale per row and 128 inputs,
              W with a scale per 128 x 128 block); its backward pass.
* ``ffn``     (act(x Wg^T) * (x Wu^T)) W2^T + residual: a shared expert or a
              dense layer; its backward pass.

``own`` False runs the plain forms (elementary torch operations, fp32, rounded
once at the end), True the calls of ``host_paged_expert_gb300.dense``.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")
EPS = 1e-6
GROUP = 128  # features of one 8-bit scale


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token of a 48-layer, hidden-2048 stack between attention and the experts: y for the routed
        # experts and its 8-bit form for a block-FP8 projection
        dict(name="norm decode 1x2048", op="norm", t=1, h=2048, dt="bf16", add=True, quant=True, train=False),
        # a prefill chunk of the same stack
        dict(name="norm chunk 2048x2048", op="norm", t=2048, h=2048, dt="bf16", add=True, quant=False, train=False),
        # many chunks together in front of an 8-bit product
        dict(name="norm large 16384x4096 fp8", op="norm", t=16384, h=4096, dt="bf16", add=True, quant=True, train=False),
        # a training step's norm on a ragged batch at the padded-width model's hidden size
        dict(name="norm train 4099x2880 f16", op="norm", t=4099, h=2880, dt="f16", add=True, quant=False, train=True),
        # the router of a decode batch: fp32 logits over 128 experts
        dict(name="router 8x2048 to 128", op="linear", t=8, k=2048, n=128, dt="bf16", out="f32", act="none", bias=False,
             res=False, fp8=False, train=False),
        # attention's output projection of one token, added to the residual stream
        dict(name="projection decode 1x4096 to 2048", op="linear", t=1, k=4096, n=2048, dt="bf16", out="bf16", act="none",
             bias=True, res=True, fp8=False, train=False),
        # a biased, activated projection of a prefill chunk
        dict(name="projection chunk 2048x4096", op="linear", t=2048, k=4096, n=4096, dt="bf16", out="bf16", act="gelu_tanh",
             bias=True, res=True, fp8=False, train=False),
        # block-FP8 weights and activations over a long batch
        dict(name="fp8 8192x2048 to 6144", op="linear", t=8192, k=2048, n=6144, dt="bf16", out="bf16", act="none",
             bias=False, res=True, fp8=True, train=False),
        # a training step of an activated projection, ragged batch
        dict(name="linear train 1021x2880 f16", op="linear", t=1021, k=2880, n=1536, dt="f16", out="f16", act="gelu", bias=True,
             res=True, fp8=False, train=True),
        # the shared expert of one decode token (expert width 768)
        dict(name="ffn decode 1x2048x768", op="ffn", t=1, h=2048, i=768, dt="bf16", act="silu", res=True, train=False),
        # a dense layer over a prefill chunk
        dict(name="ffn chunk 2048x2048x6144", op="ffn", t=2048, h=2048, i=6144, dt="bf16", act="silu", res=True, train=False),
        # a dense layer's training step
        dict(name="ffn train 4096x2048x8192", op="ffn", t=4096, h=2048, i=8192, dt="bf16", act="silu", res=False, train=True),
    ]


def _spread(rng, lo, hi, of=1):
    """A multiple of `of` between lo and hi, even over its logarithm; never 3072."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / of)) * of
        v = min(max(v, lo), hi)
        if v != 3072:
            return v


def draw(rng):
    most = _cost(work(listed()[-1]))
    while True:
        op = rng.choice(["norm", "linear", "linear", "ffn", "ffn"])
        dt = rng.choice(["bf16", "bf16", "f16"])
        train = rng.random() < 0.35
        if op == "norm":
            c = dict(op=op, t=_spread(rng, 1, 16384), h=_spread(rng, 256, 8192, 8), dt=dt, add=rng.random() < 0.7,
                     quant=not train and rng.random() < 0.5, train=train)
        elif op == "linear":
            fp8 = not train and rng.random() < 0.4
            out = dt if train or rng.random() < 0.8 else "f32"
            # fp32 results are router logits: few outputs, a model's width in
            c = dict(op=op, t=_spread(rng, 1, 8192), k=_spread(rng, 256, 4096 if out == "f32" else 8192, 16 if fp8 else 8),
                     n=_spread(rng, 16, 512, 1) if out == "f32" else _spread(rng, 64, 8192, 8), dt=dt, out=out,
                     act=rng.choice(_ACTS) if out != "f32" else "none", bias=rng.random() < 0.5,
                     res=out != "f32" and rng.random() < 0.5, fp8=fp8, train=train)
        else:
            c = dict(op=op, t=_spread(rng, 1, 8192), h=_spread(rng, 256, 4096, 8), i=_spread(rng, 128, 8192, 8), dt=dt,
                     act=rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]), res=rng.random() < 0.5, train=train)
        if _cost(work(c)) <= most:
            return c


# ----------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)


def _hidden(g, t, h, dt):
    """Hidden states: N(0, 1) with a few channels ten times as wide, as residual streams have."""
    wide = torch.ones(h, device="cuda")
    wide[torch.randint(h, (max(1, h // 256),), generator=g, device="cuda")] = 10.0
    return (torch.randn(t, h, generator=g, device="cuda") * wide).to(dt)


def _blocks(v, rows):
    """amax of each block of `rows` x 128 of a matrix, [ceil(R / rows), ceil(C / 128)]."""
    r, c = v.shape
    pr, pc = -(-r // rows) * rows, -(-c // GROUP) * GROUP
    p = torch.zeros(pr, pc, device=v.device, dtype=v.dtype)
    p[:r, :c] = v.abs()
    return p.view(pr // rows, rows, pc // GROUP, GROUP).amax(dim=(1, 3))


def _spread_scale(s, rows, r, c):
    return s.repeat_interleave(rows, 0)[:r].repeat_interleave(GROUP, 1)[:, :c]


def _to_e4m3(v, rows):
    s = _blocks(v, rows).clamp_min(1e-12) / 448.0
    return (v / _spread_scale(s, rows, *v.shape)).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], _DT[case["dt"]]
    t = case["t"]
    s = {"case": case}
    if op == "norm":
        h = case["h"]
        s["x"] = _hidden(g, t, h, dt)
        s["w"] = (1.0 + _randn(g, h, scale=0.1)).to(dt)
        s["res"] = _hidden(g, t, h, dt) if case["add"] else None
        if case["train"]:
            s["dy"] = _randn(g, t, h, scale=0.05, dt=dt)
            s["ds"] = _randn(g, t, h, scale=0.05, dt=dt) if case["add"] else None
    elif op == "linear":
        k, n = case["k"], case["n"]
        x, w = _hidden(g, t, k, torch.float32), _randn(g, n, k, scale=0.02)
        s["xs"] = s["ws"] = None
        if case["fp8"]:
            s["x"], s["xs"] = _to_e4m3(x, 1)
            s["w"], s["ws"] = _to_e4m3(w, GROUP)
        else:
            s["x"], s["w"] = x.to(dt), w.to(dt)
        s["b"] = _randn(g, n, scale=0.5, dt=dt) if case["bias"] else None
        s["res"] = _randn(g, t, n, dt=dt) if case["res"] else None
        if case["train"]:
            s["dy"] = _randn(g, t, n, scale=0.05, dt=dt)
    else:
        h, i = case["h"], case["i"]
        s["x"] = _randn(g, t, h, dt=dt)
        s["w13"], s["w2"] = _randn(g, 2 * i, h, scale=0.02, dt=dt), _randn(g, h, i, scale=0.02, dt=dt)
        s["res"] = _randn(g, t, h, dt=dt) if case["res"] else None
        if case["train"]:
            s["dy"] = _randn(g, t, h, scale=0.05, dt=dt)
    if own:
        from host_paged_expert_gb300 import dense

        s["dense"] = dense
    return s


# ----------------------------------------------------------------------------
# one pass


def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "ffn": _own_ffn}[c["op"]](state, c, state["dense"])
    return {"norm": _norm, "linear": _linear, "ffn": _ffn}[c["op"]](state, c, _DT[c["dt"]])


def _own_norm(s, c, d):
    r = d.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, quant=c["quant"], save=c["train"])
    out = {"y": r.y}
    if c["add"]:
        out["sum"] = r.sum
    if c["quant"]:
        out["codes"], out["scale"] = r.codes, r.scale
    if c["train"]:
        out["dx"], out["dw"] = d.rms_norm_backward(s["dy"], r.sum, s["w"], r.rstd, dsum=s["ds"])
    return out


def _own_linear(s, c, d):
    if not c["train"]:
        return {"y": d.linear(s["x"], s["w"], s["b"], act=c["act"], residual=s["res"], x_scale=s["xs"], w_scale=s["ws"],
                              out_dtype=_DT[c["out"]])}
    y, z = d.linear(s["x"], s["w"], s["b"], act=c["act"], residual=s["res"], save=True)
    dx, dw, db = d.linear_backward(s["dy"], s["x"], s["w"], z, act=c["act"], bias=c["bias"])
    out = {"y": y, "dx": dx, "dw": dw}
    if c["bias"]:
        out["db"] = db
    return out


def _own_ffn(s, c, d):
    if not c["train"]:
        return {"y": d.gated_ffn(s["x"], s["w13"], s["w2"], act=c["act"], residual=s["res"])}
    y, gu = d.gated_ffn(s["x"], s["w13"], s["w2"], act=c["act"], residual=s["res"], save=True)
    dx, dw13, dw2 = d.gated_ffn_backward(s["dy"], s["x"], s["w13"], s["w2"], gu, act=c["act"])
    return {"y": y, "dx": dx, "dw13": dw13, "dw2": dw2}


_C = math.sqrt(2.0 / math.pi)


def _act(z, act):
    """(act(z), act'(z))"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + u), 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * _C * (1 + 3 * 0.044715 * z * z)


def _norm(s, c, dt):
    x, w = s["x"].float(), s["w"].float()
    v = x + s["res"].float() if c["add"] else x
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    xh = v * rstd
    y = xh * w
    out = {"y": y.to(dt)}
    if c["add"]:
        out["sum"] = v.to(dt)
    if c["quant"]:
        t, h = y.shape
        q = torch.zeros(t, -(-h // GROUP) * GROUP, device=y.device)
        q[:, :h] = y
        q = q.view(t, -1, GROUP)
        amax = q.abs().amax(2, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        out["codes"] = (q / scale).view(t, -1)[:, :h].to(torch.float8_e4m3fn)
        out["scale"] = scale.view(t, -1)
    if c["train"]:
        dy = s["dy"].float()
        gw = dy * w
        dx = rstd * (gw - xh * (gw * xh).mean(1, keepdim=True))
        out["dx"] = (dx + s["ds"].float() if c["add"] else dx).to(dt)
        out["dw"] = (dy * xh).sum(0).to(dt)
    return out


def _linear(s, c, dt):
    x, w = s["x"].float(), s["w"].float()
    if c["fp8"]:
        x = x * _spread_scale(s["xs"], 1, *x.shape)
        w = w * _spread_scale(s["ws"], GROUP, *w.shape)
    z = torch.matmul(x, w.t())
    if c["bias"]:
        z = z + s["b"].float()
    y, d = _act(z, c["act"])
    if c["res"]:
        y = y + s["res"].float()
    out = {"y": y.to(_DT[c["out"]])}
    if c["train"]:
        dz = s["dy"].float() * d
        out["dx"] = torch.matmul(dz, w).to(dt)
        out["dw"] = torch.matmul(dz.t(), x).to(dt)
        if c["bias"]:
            out["db"] = dz.sum(0).to(dt)
    return out


def _ffn(s, c, dt):
    x, w13, w2, i = s["x"].float(), s["w13"].float(), s["w2"].float(), c["i"]
    z = torch.matmul(x, w13.t())
    g, u = z[:, :i], z[:, i:]
    a, da = _act(g, c["act"])
    h = a * u
    y = torch.matmul(h, w2.t())
    if c["res"]:
        y = y + s["res"].float()
    out = {"y": y.to(dt)}
    if c["train"]:
        dy = s["dy"].float()
        dh = torch.matmul(dy, w2)
        dz = torch.cat([dh * u * da, dh * a], 1)
        out["dx"] = torch.matmul(dz, w13).to(dt)
        out["dw13"] = torch.matmul(dz.t(), x).to(dt)
        out["dw2"] = torch.matmul(dy.t(), h).to(dt)
    return out


# ----------------------------------------------------------------------------
# the work that a pass cannot do without


def _cost(w):
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    t, e = case["t"], 2
    if case["op"] == "norm":
        h, add, train = case["h"], case["add"], case["train"]
        rows = (2 if add else 1) + (2 if add else 1)  # x, residual; y, sum
        b = rows * t * h * e + h * e
        if case["quant"]:
            b += t * h + 4 * t * -(-h // GROUP)
        if train:
            b += ((2 if add else 1) + 1) * t * h * e + h * e  # dy, dsum; dx, dw
        return {"bytes": b, "flops": t * h * (14 if train else 6)}
    if case["op"] == "linear":
        k, n, train = case["k"], case["n"], case["train"]
        b = (t * k + n * k) * (1 if case["fp8"] else e) + t * n * (4 if case["out"] == "f32" else e)
        if case["fp8"]:
            b += 4 * -(-k // GROUP) * (t + -(-n // GROUP))
        b += (n * e if case["bias"] else 0) + (t * n * e if case["res"] else 0)
        f = 2 * t * n * k
        if train:
            b += (t * n + t * k + n * k) * e + (n * e if case["bias"] else 0)
            f *= 3
        return {"bytes": b, "flops": f}
    h, i, train = case["h"], case["i"], case["train"]
    b = (2 * t * h + 3 * h * i) * e + (t * h * e if case["res"] else 0)
    f = 6 * t * h * i
    if train:
        b += (2 * t * h + 3 * h * i) * e
        f *= 3
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------------------
# the definitions in 64 bits


def _f64(v):
    return None if v is None else v.to(torch.float32).double() if v.dtype == torch.float8_e4m3fn else v.double()


def _sigma(z):
    return torch.sigmoid(z)


def _phi(act, z):
    """The activation and its slope at z, both in 64 bits."""
    one = torch.ones_like(z)
    if act == "silu":
        return torch.mul(z, _sigma(z)), _sigma(z) + z * _sigma(z) * _sigma(-z)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # 0.5 (1 + tanh a) = sigma(2a)
        a2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3))
        return z * _sigma(a2), _sigma(a2) + z * _sigma(a2) * _sigma(-a2) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z.square())
    if act == "relu":
        return torch.where(z > 0, z, 0 * one), torch.where(z > 0, one, 0 * one)
    return z, one


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: _f64(x) for k, x in s.items() if isinstance(x, torch.Tensor)}
    add = lambda a, k: a + v[k] if k in v else a  # noqa: E731
    out = {}
    if case["op"] == "norm":
        total = add(v["x"], "res")
        rms = torch.sqrt(torch.linalg.vector_norm(total, dim=1).square() / case["h"] + EPS)[:, None]
        unit = total / rms
        out["y"] = unit * v["w"]
        if case["add"]:
            out["sum"] = total
        if case["quant"]:
            parts = out["y"].split(GROUP, 1)
            tops = [p.abs().amax(1, keepdim=True) for p in parts]
            tops = [torch.where(p > 0, p / 448, torch.ones_like(p)) for p in tops]
            out["scale"] = torch.cat(tops, 1)
            out["codes"] = torch.cat([p / q for p, q in zip(parts, tops)], 1)
        if case["train"]:
            g = v["dy"] * v["w"]
            along = torch.einsum("th,th->t", g, unit)[:, None] / case["h"]
            out["dx"] = add((g - unit * along) / rms, "ds")
            out["dw"] = torch.einsum("th,th->h", v["dy"], unit)
    elif case["op"] == "linear":
        x, w = v["x"], v["w"]
        if case["fp8"]:
            kb = torch.arange(case["k"], device=x.device) // GROUP
            nb = torch.arange(case["n"], device=x.device) // GROUP
            x, w = x * v["xs"][:, kb], w * v["ws"][nb][:, kb]
        f, df = _phi(case["act"], add(torch.einsum("tk,nk->tn", x, w), "b"))
        out["y"] = add(f, "res")
        if case["train"]:
            dz = v["dy"] * df
            out["dx"] = torch.einsum("tn,nk->tk", dz, w)
            out["dw"] = torch.einsum("tn,tk->nk", dz, x)
            if case["bias"]:
                out["db"] = torch.einsum("tn->n", dz)
    else:
        i = case["i"]
        wg, wu, w2 = v["w13"][:i], v["w13"][i:], v["w2"]
        gate, up = torch.einsum("th,ih->ti", v["x"], wg), torch.einsum("th,ih->ti", v["x"], wu)
        f, df = _phi(case["act"], gate)
        mid = f * up
        out["y"] = add(torch.einsum("ti,hi->th", mid, w2), "res")
        if case["train"]:
            dmid = torch.einsum("th,hi->ti", v["dy"], w2)
            dgate, dup = dmid * up * df, dmid * f
            out["dx"] = torch.einsum("ti,ih->th", dgate, wg) + torch.einsum("ti,ih->th", dup, wu)
            out["dw13"] = torch.cat([torch.einsum("ti,th->ih", dgate, v["x"]), torch.einsum("ti,th->ih", dup, v["x"])])
            out["dw2"] = torch.einsum("th,ti->hi", v["dy"], mid)
    return out
