"""Cases of the operators of a layer whose experts are resident, and of 4-bit
projections, and what they compute.

A mixture-of-experts layer that is trained, or served with every expert in
HBM, is a router, rows moved to their experts, products grouped by expert and
rows moved back; a checkpoint with 4-bit experts has 4-bit projections next to
them:

* ``w4``      act(x W^T + bias) + residual with W in 4 bits: GPTQ int4 ((q - 8)
              times an fp16 scale per 128 inputs), MXFP4 (E2M1 times an E8M0
              scale per 32), NVFP4 (E2M1 times an E4M3 scale per 16 and one
              fp32 scale).
* ``route``   the top-k experts of each token by logit (ties to the lower id),
              softmax over the chosen, and each entry's row in the order sorted
              by expert; the gradient of the logits.
* ``rows``    x[t] to the rows of its entries, and the weighted sum of a token's
              rows plus the residual; their gradients.
* ``grouped`` y = x W_e^T over the rows of each expert e (ragged, some empty);
              its gradients.
* ``experts`` (act(x Wg_e^T) * (x Wu_e^T)) W2_e^T over the rows of each expert;
              its gradients.

``own`` False runs the plain forms (elementary torch operations, fp32, rounded
once at the end), True the calls of ``host_paged_expert_gb300.dense``.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")
_GROUP = {"int4": 128, "mxfp4": 32, "nvfp4": 16}  # inputs of one scale
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # the attention's output projection of one decoded token in a GPTQ checkpoint
        dict(name="int4 decode 1x4096 to 2048", op="w4", t=1, k=4096, n=2048, fmt="int4", dt="bf16", act="none", bias=False, res=True),
        # a biased projection of a small decode batch at the padded-width model's hidden size
        dict(name="mxfp4 5x2880 to 5120", op="w4", t=5, k=2880, n=5120, fmt="mxfp4", dt="bf16", act="none", bias=True, res=False),
        # 32 requests' logits over a vocabulary
        dict(name="nvfp4 32x4096 to 32000", op="w4", t=32, k=4096, n=32000, fmt="nvfp4", dt="bf16", act="none", bias=False, res=False),
        # a prefill chunk through an activated projection
        dict(name="int4 chunk 2048x4096", op="w4", t=2048, k=4096, n=4096, fmt="int4", dt="f16", act="gelu_tanh", bias=True, res=True),
        # the router's choice for a decode batch: top-8 of 128
        dict(name="route 8 of 128, 8 tokens", op="route", t=8, e=128, k=8, train=False),
        # the router of a training step
        dict(name="route 8 of 128, 16384 tokens, train", op="route", t=16384, e=128, k=8, train=True),
        # a decode batch's rows to its experts and back
        dict(name="rows 8x8x2048", op="rows", t=8, k=8, h=2048, dt="bf16", res=True, train=False),
        # the same of a training step, with the gradients; ragged
        dict(name="rows train 8191x8x2048", op="rows", t=8191, k=8, h=2048, dt="bf16", res=True, train=True),
        # one projection of every expert for 4 decoded tokens: one row or two each
        dict(name="grouped decode 4x8 of 128, 2048 to 1536", op="grouped", t=4, e=128, top=8, skew=1.0, k=2048, n=1536, dt="bf16", train=False),
        # its training step on a ragged batch with few wide experts
        dict(name="grouped train 1021x2 of 8, 2880 to 1440 f16", op="grouped", t=1021, e=8, top=2, skew=0.5, k=2880, n=1440, dt="f16", train=True),
        # every expert's feed-forward over a prefill chunk
        dict(name="experts chunk 2048x8 of 128, 2048x768", op="experts", t=2048, e=128, top=8, skew=1.0, h=2048, i=768, act="silu", dt="bf16", train=False),
        # the layer's training step
        dict(name="experts train 4096x8 of 128, 2048x768", op="experts", t=4096, e=128, top=8, skew=0.5, h=2048, i=768, act="silu", dt="bf16", train=True),
    ]


def _spread(rng, lo, hi, of=1):
    """A multiple of `of` between lo and hi, even over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / of)) * of
    return min(max(v, lo), hi)


def draw(rng):
    most = _cost(work(listed()[-1]))
    while True:
        op = rng.choice(["w4", "w4", "route", "rows", "grouped", "grouped", "experts", "experts"])
        dt, train = rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.4
        if op == "w4":
            # most calls are a decode batch's
            c = dict(op=op, t=_spread(rng, 1, rng.choice([8, 64, 4096])), k=_spread(rng, 256, 8192, 32), n=_spread(rng, 64, 16384, rng.choice([8, 8, 1])),
                     fmt=rng.choice(["int4", "mxfp4", "nvfp4"]), dt=dt, act=rng.choice(["none", "none", *_ACTS]), bias=rng.random() < 0.4, res=rng.random() < 0.4)
        elif op == "route":
            e = _spread(rng, 4, 512)
            c = dict(op=op, t=_spread(rng, 1, 32768), e=e, k=_spread(rng, 1, min(e, 16)), train=train)
        elif op == "rows":
            c = dict(op=op, t=_spread(rng, 1, 8192), k=_spread(rng, 1, 10), h=_spread(rng, 128, 8192, 8), dt=dt, res=rng.random() < 0.5, train=train)
        else:
            e = _spread(rng, 2, 256)
            c = dict(op=op, t=_spread(rng, 1, 4096), e=e, top=_spread(rng, 1, min(e, 8)), skew=rng.choice([0.0, 0.5, 1.0, 2.0]), dt=dt, train=train)
            if op == "grouped":
                c.update(k=_spread(rng, 128, 4096, 8), n=_spread(rng, 64, 4096, 8))
            else:
                c.update(h=_spread(rng, 128, 4096, 8), i=_spread(rng, 64, 2048, 8), act=rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]))
            if _weights(c) > 1.2e9:
                continue
        if _cost(work(c)) <= most:
            return c


def _weights(c):
    return c["e"] * (c["k"] * c["n"] if c["op"] == "grouped" else 3 * c["h"] * c["i"])


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


def _per_expert(g, e, n, k, dt):
    w = torch.empty(e, n, k, device="cuda", dtype=dt)
    for m in w:
        m.copy_(torch.randn(n, k, generator=g, device="cuda") * 0.02)
    return w


def _logits(g, t, e, skew):
    """Router logits: experts more and less popular, fresh noise per token."""
    return torch.randn(t, e, generator=g, device="cuda") + skew * torch.randn(e, generator=g, device="cuda")


def _sizes(g, c):
    """Rows of each expert."""
    ids = torch.topk(_logits(g, c["t"], c["e"], c["skew"]), c["top"], 1).indices
    return torch.bincount(ids.flatten(), minlength=c["e"])


def _four_bits(g, n, k, fmt):
    """(codes [n, k / 2], scales, the tensor's scale or None) of weights of about 0.02."""
    def codes():
        if fmt == "int4":
            return (8 + 2.5 * torch.randn(n, k, generator=g, device="cuda")).round().clamp(0, 15).to(torch.uint8)
        return torch.randint(16, (n, k), generator=g, device="cuda", dtype=torch.uint8)

    q = codes()
    q = q[:, 0::2] | (q[:, 1::2] << 4)
    shape = (n, -(-k // _GROUP[fmt]))
    if fmt == "int4":
        return q, (torch.randn(*shape, generator=g, device="cuda").abs() * 0.008 + 0.001).half(), None
    if fmt == "mxfp4":
        return q, torch.randint(119, 122, shape, generator=g, device="cuda", dtype=torch.uint8), None
    s = (1 + 0.25 * torch.randn(*shape, generator=g, device="cuda")).abs().to(torch.float8_e4m3fn)
    return q, s.view(torch.uint8), 0.007 * (1 + 0.1 * torch.randn(1, generator=g, device="cuda"))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s, t = {"case": case}, case["t"]
    dt = _DT.get(case.get("dt"))
    if op == "w4":
        k, n = case["k"], case["n"]
        s["x"] = _hidden(g, t, k, dt)
        s["q"], s["s"], s["ts"] = _four_bits(g, n, k, case["fmt"])
        s["b"] = _randn(g, n, scale=0.5, dt=dt) if case["bias"] else None
        s["res"] = _randn(g, t, n, dt=dt) if case["res"] else None
    elif op == "route":
        # logits of 16-bit products tie now and then
        s["logits"] = (_logits(g, t, case["e"], 1.0) * 64).round() / 64
        if case["train"]:
            s["dw"] = _randn(g, t, case["k"], scale=0.05)
    elif op == "rows":
        k, h = case["k"], case["h"]
        s["place"] = torch.randperm(t * k, generator=g, device="cuda").view(t, k).int()
        s["x"], s["y"] = _hidden(g, t, h, dt), _randn(g, t * k, h, dt=dt)
        s["w"] = torch.softmax(torch.randn(t, k, generator=g, device="cuda"), 1)
        s["res"] = _randn(g, t, h, dt=dt) if case["res"] else None
        if case["train"]:
            s["dout"] = _randn(g, t, h, scale=0.05, dt=dt)
            s["dxs"] = _randn(g, t * k, h, scale=0.05, dt=dt)
    else:
        sizes = _sizes(g, case)
        s["offsets"] = torch.zeros(case["e"] + 1, device="cuda", dtype=torch.int32)
        s["offsets"][1:] = sizes.cumsum(0)
        rows = t * case["top"]
        if not own:
            s["sizes"] = sizes.tolist()  # what the plain form's loop over the experts goes by
        if op == "grouped":
            s["x"], s["w"] = _hidden(g, rows, case["k"], dt), _per_expert(g, case["e"], case["n"], case["k"], dt)
            if case["train"]:
                s["dy"] = _randn(g, rows, case["n"], scale=0.05, dt=dt)
        else:
            h, i = case["h"], case["i"]
            s["x"] = _randn(g, rows, h, dt=dt)
            s["w13"], s["w2"] = _per_expert(g, case["e"], 2 * i, h, dt), _per_expert(g, case["e"], h, i, dt)
            if case["train"]:
                s["dy"] = _randn(g, rows, h, scale=0.05, dt=dt)
    if own:
        from host_paged_expert_gb300 import dense

        s["dense"] = dense
    return s


# ----------------------------------------------------------------------------
# one pass


def run(state):
    c = state["case"]
    if own:
        return {"w4": _own_w4, "route": _own_route, "rows": _own_rows, "grouped": _own_grouped, "experts": _own_experts}[c["op"]](
            state, c, state["dense"])
    return {"w4": _w4, "route": _route, "rows": _rows, "grouped": _grouped, "experts": _experts}[c["op"]](state, c, _DT.get(c.get("dt")))


def _own_w4(s, c, d):
    return {"y": d.linear_w4(s["x"], s["q"], s["s"], c["fmt"], s["b"], c["act"], s["res"], tensor_scale=s["ts"])}


def _own_route(s, c, d):
    r = d.route(s["logits"], c["k"])
    out = {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "place": r.place}
    if c["train"]:
        out["dlogits"] = d.route_backward(s["dw"], r.weights, r.ids, c["e"])
    return out


def _own_rows(s, c, d):
    out = {"xs": d.expand_rows(s["x"], s["place"]), "out": d.combine_rows(s["y"], s["place"], s["w"], s["res"])}
    if c["train"]:
        out["dx"] = d.combine_rows(s["dxs"], s["place"])
        out["dy"], out["dw"] = d.combine_rows_backward(s["dout"], s["y"], s["place"], s["w"])
    return out


def _own_grouped(s, c, d):
    out = {"y": d.grouped_linear(s["x"], s["w"], s["offsets"])}
    if c["train"]:
        out["dx"], out["dw"] = d.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"])
    return out


def _own_experts(s, c, d):
    if not c["train"]:
        return {"y": d.grouped_ffn(s["x"], s["w13"], s["w2"], s["offsets"], c["act"])}
    y, gu = d.grouped_ffn(s["x"], s["w13"], s["w2"], s["offsets"], c["act"], save=True)
    dx, dw13, dw2 = d.grouped_ffn_backward(s["dy"], s["x"], s["w13"], s["w2"], gu, s["offsets"], c["act"])
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


def _w4(s, c, dt):
    q, k = s["q"], c["k"]
    codes = torch.stack([q & 15, q >> 4], 2).view(c["n"], k)
    if c["fmt"] == "int4":
        w, sc = codes.float() - 8, s["s"].float()
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device)
        w = table[codes.int()]
        sc = torch.exp2(s["s"].float() - 127) if c["fmt"] == "mxfp4" else s["s"].view(torch.float8_e4m3fn).float() * s["ts"]
    w = w * sc.repeat_interleave(_GROUP[c["fmt"]], 1)[:, :k]
    z = torch.matmul(s["x"].float(), w.t())
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])[0]
    if c["res"]:
        y = y + s["res"].float()
    return {"y": y.to(dt)}


def _route(s, c, dt):
    lg, e, k = s["logits"], c["e"], c["k"]
    v, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    p = torch.exp(v - v[:, :1])
    w = p / p.sum(1, keepdim=True)
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=lg.device)
    offsets = torch.zeros(e + 1, device=lg.device, dtype=torch.int32)
    offsets[1:] = (flat[:, None] == torch.arange(e, device=lg.device)).sum(0).cumsum(0)
    out = {"ids": ids.int(), "weights": w, "offsets": offsets, "place": place.view_as(ids).int()}
    if c["train"]:
        g = w * (s["dw"] - (w * s["dw"]).sum(1, keepdim=True))
        out["dlogits"] = torch.zeros_like(lg).scatter_(1, ids, g)
    return out


def _rows(s, c, dt):
    t, k, h = c["t"], c["k"], c["h"]
    place = s["place"].long()
    xs = torch.empty(t * k, h, device=place.device, dtype=dt)
    xs[place.flatten()] = s["x"].repeat_interleave(k, 0)
    y = s["y"][place].float()
    o = (y * s["w"][:, :, None]).sum(1)
    if c["res"]:
        o = o + s["res"].float()
    out = {"xs": xs, "out": o.to(dt)}
    if c["train"]:
        out["dx"] = s["dxs"][place].float().sum(1).to(dt)
        d = s["dout"].float()
        dy = torch.empty_like(s["y"])
        dy[place.flatten()] = (s["w"][:, :, None] * d[:, None]).view(t * k, h).to(dt)
        out["dy"], out["dw"] = dy, (y * d[:, None]).sum(2)
    return out


def _grouped(s, c, dt):
    x, w = s["x"], s["w"]
    out = {"y": torch.empty(x.shape[0], c["n"], device=x.device, dtype=dt)}
    if c["train"]:
        out["dx"], out["dw"] = torch.empty_like(x), torch.empty_like(w)
    r = 0
    for e, m in enumerate(s["sizes"]):
        xe, we = x[r : r + m].float(), w[e].float()
        out["y"][r : r + m] = torch.matmul(xe, we.t()).to(dt)
        if c["train"]:
            dy = s["dy"][r : r + m].float()
            out["dx"][r : r + m] = torch.matmul(dy, we).to(dt)
            out["dw"][e] = torch.matmul(dy.t(), xe).to(dt)
        r += m
    return out


def _experts(s, c, dt):
    x, i = s["x"], c["i"]
    out = {"y": torch.empty_like(x)}
    if c["train"]:
        out["dx"], out["dw13"], out["dw2"] = torch.empty_like(x), torch.empty_like(s["w13"]), torch.empty_like(s["w2"])
    r = 0
    for e, m in enumerate(s["sizes"]):
        xe, w13, w2 = x[r : r + m].float(), s["w13"][e].float(), s["w2"][e].float()
        z = torch.matmul(xe, w13.t())
        g, u = z[:, :i], z[:, i:]
        a, da = _act(g, c["act"])
        h = a * u
        out["y"][r : r + m] = torch.matmul(h, w2.t()).to(dt)
        if c["train"]:
            dy = s["dy"][r : r + m].float()
            dh = torch.matmul(dy, w2)
            dz = torch.cat([dh * u * da, dh * a], 1)
            out["dx"][r : r + m] = torch.matmul(dz, w13).to(dt)
            out["dw13"][e] = torch.matmul(dz.t(), xe).to(dt)
            out["dw2"][e] = torch.matmul(dy.t(), h).to(dt)
        r += m
    return out


# ----------------------------------------------------------------------------
# the work that a pass cannot do without


def _cost(w):
    return max(w["bytes"], w["flops"] / 50)


def _active(c):
    """Experts that some row reaches, of so many tokens with distinct choices (popularity apart)."""
    return c["e"] * (1 - (1 - c["top"] / c["e"]) ** c["t"])


def work(case):
    t, op = case["t"], case["op"]
    train = case.get("train", False)
    if op == "w4":
        k, n = case["k"], case["n"]
        b = n * k / 2 + n * -(-k // _GROUP[case["fmt"]]) * (2 if case["fmt"] == "int4" else 1) + 2 * t * (k + n)
        return {"bytes": b + (2 * n if case["bias"] else 0) + (2 * t * n if case["res"] else 0), "flops": 2 * t * n * k}
    if op == "route":
        e, k = case["e"], case["k"]
        return {"bytes": t * (4 * e + 12 * k) + (t * (4 * e + 4 * k) if train else 0), "flops": t * (e + 8 * k) * (2 if train else 1)}
    if op == "rows":
        k, h = case["k"], case["h"]
        # x, y, the residual; xs, out; with the gradients dxs, dout, dx, dy
        b = 2 * t * h * (2 + 2 * k + (1 if case["res"] else 0)) + 8 * t * k
        b += 2 * t * h * (2 + 2 * k) + 4 * t * k if train else 0
        return {"bytes": b, "flops": 2 * t * h * k * (3.5 if train else 1)}
    rows, used = t * case["top"], _active(case)
    if op == "grouped":
        k, n = case["k"], case["n"]
        b = 2 * (rows * (k + n) + used * k * n)
        b += 2 * (rows * (k + n) + case["e"] * k * n) if train else 0
        return {"bytes": b, "flops": 2 * rows * k * n * (3 if train else 1)}
    h, i = case["h"], case["i"]
    b = 2 * (2 * rows * h + used * 3 * h * i)
    b += 2 * (2 * rows * h + case["e"] * 3 * h * i) if train else 0
    return {"bytes": b, "flops": 6 * rows * h * i * (3 if train else 1)}


# ----------------------------------------------------------------------------
# the definitions in 64 bits


def _phi(act, z):
    """The activation and its slope at z, both in 64 bits."""
    one = torch.ones_like(z)
    if act == "silu":
        p = torch.sigmoid(z)
        return torch.mul(z, p), p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # 0.5 (1 + tanh a) = sigma(2a)
        a2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3))
        p = torch.sigmoid(a2)
        return z * p, p + z * p * torch.sigmoid(-a2) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z.square())
    if act == "relu":
        return torch.where(z > 0, z, 0 * one), torch.where(z > 0, one, 0 * one)
    return z, one


def _value(q, fmt):
    """What a code stands for, by its bits."""
    q = q.long()
    if fmt == "int4":
        return (q - 8).double()
    sign, exponent, mantissa = q >> 3, (q >> 1) & 3, q & 1
    mag = torch.where(exponent > 0, (2 + mantissa).double() * 2.0 ** (exponent - 2).double(), mantissa.double() / 2)
    return torch.where(sign > 0, -mag, mag)


def _scale(s, fmt, ts):
    if fmt == "int4":
        return s.double()
    if fmt == "mxfp4":
        return 2.0 ** (s.double() - 127)
    b = s.long()
    exponent, mantissa = (b >> 3) & 15, (b & 7).double()
    v = torch.where(exponent > 0, (1 + mantissa / 8) * 2.0 ** (exponent - 7).double(), mantissa / 8 * 2.0**-6)
    return torch.where(b >> 7 > 0, -v, v) * ts.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    dev = s["x"].device if "x" in s else s["logits"].device
    if op == "w4":
        k, n, fmt = case["k"], case["n"], case["fmt"]
        y = torch.empty(case["t"], n, device=dev, dtype=torch.float64)
        group = torch.arange(k, device=dev) // _GROUP[fmt]
        x = s["x"].double()
        for a in range(0, n, 4096):  # rows of W at a time
            q = s["q"][a : a + 4096]
            w = torch.empty(q.shape[0], k, device=dev, dtype=torch.float64)
            w[:, 0::2], w[:, 1::2] = _value(q % 16, fmt), _value(q // 16, fmt)
            w *= _scale(s["s"][a : a + 4096], fmt, s["ts"])[:, group]
            y[:, a : a + 4096] = torch.einsum("tk,nk->tn", x, w)
        if case["bias"]:
            y += s["b"].double()
        y, _ = _phi(case["act"], y)
        return {"y": y + s["res"].double() if case["res"] else y}
    if op == "route":
        lg, e, k = s["logits"].double(), case["e"], case["k"]
        t = lg.shape[0]
        left, idx = lg.clone(), torch.arange(e, device=dev)
        ids, top = [], []
        for _ in range(k):  # the largest left, the lowest id among equals
            m = left.amax(1, keepdim=True)
            i = torch.where(left == m, idx, e).amin(1)
            ids.append(i)
            top.append(m[:, 0])
            left.scatter_(1, i[:, None], -math.inf)
        ids, w = torch.stack(ids, 1), torch.softmax(torch.stack(top, 1), 1)
        hit = torch.zeros(t * k, e, device=dev, dtype=torch.int32)
        hit[torch.arange(t * k, device=dev), ids.flatten()] = 1
        count = hit.sum(0)
        offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
        before = hit.cumsum(0, dtype=torch.int32).gather(1, ids.flatten()[:, None])[:, 0] - 1  # entries of the same expert ahead of this one
        out = {"ids": ids.int(), "weights": w, "offsets": offsets.int(), "place": (offsets[ids.flatten()] + before).view(t, k).int()}
        if case["train"]:
            dw = s["dw"].double()
            # the softmax's Jacobian
            jac = torch.diag_embed(w) - torch.einsum("ti,tj->tij", w, w)
            out["dlogits"] = torch.zeros_like(lg)
            out["dlogits"].scatter_add_(1, ids, torch.einsum("tij,tj->ti", jac, dw))
        return out
    if op == "rows":
        k, h, place = case["k"], case["h"], s["place"].long()
        w = s["w"].double()
        token = torch.empty(place.numel(), device=dev, dtype=torch.long)
        token[place.flatten()] = torch.arange(case["t"], device=dev).repeat_interleave(k)
        wr = torch.empty(place.numel(), device=dev, dtype=torch.float64)
        wr[place.flatten()] = w.flatten()
        out = {"xs": s["x"][token].double()}
        o = torch.zeros(case["t"], h, device=dev, dtype=torch.float64).index_add_(0, token, s["y"].double() * wr[:, None])
        out["out"] = o + s["res"].double() if case["res"] else o
        if case["train"]:
            out["dx"] = torch.zeros_like(o).index_add_(0, token, s["dxs"].double())
            d = s["dout"][token].double()
            out["dy"] = d * wr[:, None]
            out["dw"] = torch.einsum("rh,rh->r", d, s["y"].double())[place]
        return out
    train = case["train"]
    out = {k: [] for k in ("y", "dx", "dw", "dw13", "dw2")}
    at = s["offsets"].tolist()
    for e in range(case["e"]):
        rows = slice(at[e], at[e + 1])
        x = s["x"][rows].double()
        dy = s["dy"][rows].double() if train else None
        if op == "grouped":
            w = s["w"][e].double()
            out["y"].append(torch.einsum("rk,nk->rn", x, w))
            if train:
                out["dx"].append(torch.einsum("rn,nk->rk", dy, w))
                out["dw"].append(torch.einsum("rn,rk->nk", dy, x))
            continue
        i = case["i"]
        w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        gate, up = torch.einsum("rh,ih->ri", x, w13[:i]), torch.einsum("rh,ih->ri", x, w13[i:])
        f, df = _phi(case["act"], gate)
        mid = f * up
        out["y"].append(torch.einsum("ri,hi->rh", mid, w2))
        if train:
            dmid = torch.einsum("rh,hi->ri", dy, w2)
            dgate, dup = dmid * up * df, dmid * f
            out["dx"].append(torch.einsum("ri,ih->rh", dgate, w13[:i]) + torch.einsum("ri,ih->rh", dup, w13[i:]))
            out["dw13"].append(torch.cat([torch.einsum("ri,rh->ih", dgate, x), torch.einsum("ri,rh->ih", dup, x)]))
            out["dw2"].append(torch.einsum("rh,ri->hi", dy, mid))
    return {k: torch.stack(v) if k.startswith("dw") else torch.cat(v) for k, v in out.items() if v}
