"""Dense operators on the GPU against their 64-bit forms (tests/dense_ref.py
derives the bounds)."""

import pytest

torch = pytest.importorskip("torch")

import dense_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from host_paged_expert_gb300 import dense

    yield dense
    assert dense.error_word() == 0


def rand(*shape, seed=0, scale=1.0, dt=BF):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + shape[0] + 31 * shape[-1])
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def pitched(t, extra):
    """The same matrix with a wider row pitch, NaN in between."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device, dtype=torch.float32).to(t.dtype)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- RMS norm


@pytest.mark.parametrize("rows,h", [(1, 8), (1, 2048), (3, 136), (5, 2880), (2, 8192), (1, 32768), (33, 4096), (700, 1032), (2, 16392)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("add", [False, True])
def test_rms_norm(D, rows, h, dt, add):
    x, w = rand(rows, h, dt=dt), rand(h, seed=2, dt=dt)
    res = rand(rows, h, seed=1, scale=3, dt=dt) if add else None
    got = D.rms_norm(x, w, res, 1e-5, quant=True, save=True)
    want = R.rms_norm(x, w, res, 1e-5, dt)
    R.check(got.y, want["y"], "y")
    R.check(got.rstd, want["rstd"], "rstd")
    if add:
        R.check(got.sum, want["sum"], "sum")
    else:
        assert got.sum is x
    y, sc = want["raw"], R.scales(want["raw"])
    R.check(got.scale, sc, "scale")
    # codes: within half a step of E4M3 (2^-4 relative, 2^-10 below the normal numbers) of y / scale
    s = R.spread(got.scale.double(), 1, rows, h)
    c = got.codes.double()
    off = (c - y.v / s).abs() - y.b / s
    assert (off <= (y.v / s).abs() * 2.0**-4 * 1.0001 + 2.0**-10 * 1.0001).all()
    assert c.abs().max() <= 448
    # without the extras: the same bits
    assert same(D.rms_norm(x, w, res, 1e-5).y, got.y)
    only = D.rms_norm(x, w, res, 1e-5, y=False, quant=True)
    assert only.y is None and only.rstd is None and same(only.codes, got.codes) and same(only.scale, got.scale)


def test_rms_norm_odd_rows(D):
    """A row of zeros, one of huge and one of tiny values, an infinity and a
    NaN: each stays within its row."""
    h = 264
    x = rand(6, h)
    x[1] = 0
    x[2] = 1e15
    x[3] = 1e-30
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    w = rand(h, seed=1)
    got = D.rms_norm(x, w, quant=True, save=True)
    want = R.rms_norm(x[:4], w, None, 1e-6, BF)
    for k, name in ((got.y, "y"), (got.rstd, "rstd")):
        R.check(k[:4], R.Q(want[name].v, want[name].b), name)
    assert (got.codes[1].float() == 0).all() and (got.scale[1] == 1).all()
    assert got.y[4].isnan().sum() == 1 and got.y[4, 7].isnan()
    assert got.y[5].isnan().all() and got.codes[5].float().isnan().all() and got.scale[5].isnan().all()


@pytest.mark.parametrize("rows,h", [(1, 8), (1, 2048), (37, 136), (311, 2880), (2, 8200), (1, 32768), (1000, 1032)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("add", [False, True])
def test_rms_norm_backward(D, rows, h, dt, add):
    x, w, dy = rand(rows, h, dt=dt), rand(h, seed=2, dt=dt), rand(rows, h, seed=3, dt=dt)
    ds = rand(rows, h, seed=4, dt=dt) if add else None
    f = D.rms_norm(x, w, rand(rows, h, seed=1, dt=dt) if add else None, save=True)
    dx, dw = D.rms_norm_backward(dy, f.sum, w, f.rstd, ds)
    want = R.rms_norm_backward(dy, f.sum, w, f.rstd, ds, dt)
    R.check(dx, want["dx"], "dx")
    R.check(dw, want["dw"], "dw")
    again = D.rms_norm_backward(dy, f.sum, w, f.rstd, ds)
    assert same(dx, again[0]) and same(dw, again[1])


@pytest.mark.parametrize("rows,h", [(500, 8200), (333, 16376), (320, 32768)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_rms_norm_wide(D, rows, h, dt):
    """Rows wider than registers hold, several to a block."""
    test_rms_norm(D, rows, h, dt, True)
    test_rms_norm_backward(D, rows, h, dt, False)
    test_rms_norm_backward(D, rows, h, dt, True)


def test_rms_norm_strides(D):
    x, r, w, dy = rand(9, 264), rand(9, 264, seed=1), rand(264, seed=2), rand(9, 264, seed=3)
    a, b = D.rms_norm(x, w, r, save=True), D.rms_norm(pitched(x, 8), w, pitched(r, 24), save=True)
    assert same(a.y, b.y) and same(a.sum, b.sum)
    g, k = D.rms_norm_backward(dy, a.sum, w, a.rstd, r), D.rms_norm_backward(pitched(dy, 8), pitched(a.sum, 16), w, a.rstd, pitched(r, 8))
    assert same(g[0], k[0]) and same(g[1], k[1])


# ---- linear

SIZES = [(1, 8, 1), (1, 64, 3), (2, 1032, 777), (3, 264, 1000), (4, 2056, 130), (1, 4096, 2048), (8, 2048, 128), (17, 136, 60), (64, 264, 200), (129, 520, 264), (257, 1032, 777),
         (300, 72, 1024), (1024, 256, 512), (2, 8192, 40), (700, 2056, 1544), (2500, 264, 5000), (1300, 1032, 1928)]


@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("full", [False, True])
def test_linear(D, rows, k, n, dt, full):
    act = ACTS[(rows + k + n) % 5] if full else "none"
    x, w = rand(rows, k, dt=dt), rand(n, k, seed=1, scale=k**-0.5, dt=dt)
    b = rand(n, seed=2, dt=dt) if full else None
    res = rand(rows, n, seed=3, dt=dt) if full else None
    want = R.linear(x, w, b, act, res, dt, dt)
    y, z = D.linear(x, w, b, act, res, save=True)
    R.check(y, want["y"], "y")
    if act != "none":
        R.check(z, want["z"], "z")
    assert same(D.linear(x, w, b, act, res), y)
    y32 = D.linear(x, w, b, act, res, out_dtype=torch.float32)
    R.check(y32, R.linear(x, w, b, act, res, dt, torch.float32)["y"], "fp32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [5, 300])
def test_linear_activations(D, act, rows):
    """Each activation over a wide range of z."""
    x, w, b = rand(rows, 64, scale=4, dt=HF), rand(72, 64, seed=1, scale=0.3, dt=HF), rand(72, seed=2, dt=HF)
    R.check(D.linear(x, w, b, act), R.linear(x, w, b, act, None, HF, HF)["y"], act)


def quantised(v, rows):
    r, c = v.shape
    p = torch.zeros(-(-r // rows) * rows, -(-c // 128) * 128, device="cuda")
    p[:r, :c] = v.float().abs()
    s = p.view(-1, rows, p.shape[1] // 128, 128).amax(dim=(1, 3)).clamp_min(1e-10) / 448
    return (v.float() / R.spread(s, rows, r, c)).to(F8), s


@pytest.mark.parametrize("rows,k,n", [(1, 16, 1), (1, 2048, 512), (3, 1040, 333), (8, 2048, 200), (33, 144, 72), (130, 1040, 777), (200, 4096, 264),
                                      (513, 384, 1024), (1100, 2048, 520), (2500, 400, 5000)])
@pytest.mark.parametrize("full", [False, True])
def test_linear_fp8(D, rows, k, n, full):
    x, xs = quantised(rand(rows, k) * torch.linspace(0.1, 30, k, device="cuda"), 1)
    w, ws = quantised(rand(n, k, seed=1, scale=k**-0.5) * torch.linspace(0.2, 5, n, device="cuda")[:, None], 128)
    b, res = (rand(n, seed=2), rand(rows, n, seed=3)) if full else (None, None)
    act = "gelu_tanh" if full else "none"
    y = D.linear(x, w, b, act, res, x_scale=xs, w_scale=ws)
    R.check(y, R.linear(x, w, b, act, res, BF, BF, xs, ws)["y"], "y")
    assert same(D.linear(pitched(x, 16), w, b, act, res, x_scale=xs, w_scale=ws), y)
    y32 = D.linear(x, w, b, act, res, x_scale=xs, w_scale=ws, out_dtype=torch.float32)
    R.check(y32, R.linear(x, w, b, act, res, BF, torch.float32, xs, ws)["y"], "fp32")


@pytest.mark.parametrize("rows,k,n", [(1, 8, 1), (1, 256, 64), (13, 136, 60), (200, 264, 77), (129, 520, 264), (1021, 328, 136),
                                      (64, 2048, 128), (600, 1032, 776), (2500, 2312, 2056)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_linear_backward(D, rows, k, n, dt, act):
    x, w, dy = rand(rows, k, dt=dt), rand(n, k, seed=1, scale=k**-0.5, dt=dt), rand(rows, n, seed=3, dt=dt)
    _, z = D.linear(x, w, act=act, save=True)
    dx, dw, db = D.linear_backward(dy, x, w, z, act, bias=True)
    want = R.linear_backward(dy, x, w, z, act, dt)
    for g, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
        R.check(g, want[name], name)
    again = D.linear_backward(dy, x, w, z, act, bias=True)
    assert same(dx, again[0]) and same(dw, again[1]) and same(db, again[2])
    assert D.linear_backward(dy, x, w, z, act)[2] is None


def test_linear_gradient_matches_differences(D):
    """Along a direction v the loss sum(dy * y) of a plain product changes by
    exactly <dx, v>: both sides in fp32 from fp16 operands, so they agree to
    the rounding of dx (2^-11 of each term) and of the fp32 results."""
    x, w, dy, v = rand(40, 72, dt=HF), rand(56, 72, seed=1, dt=HF), rand(40, 56, seed=2, dt=HF), rand(40, 72, seed=3, dt=HF)
    dx, dw, _ = D.linear_backward(dy, x, w)
    f = lambda a: (D.linear(a, w, out_dtype=torch.float32).double() * dy.double()).sum().item()  # noqa: E731
    up, down = (x.double() + v.double()).to(HF), (x.double() - v.double()).to(HF)
    step = up.double() - down.double()
    bound = (2.0**-11 * (dx.double() * step).abs().sum() + 2.0**-18 * 72 * dy.double().abs().sum()).item()
    assert abs(f(up) - f(down) - (dx.double() * step).sum().item()) <= bound


def test_linear_strides(D):
    x, w, r, dy = rand(140, 264), rand(72, 264, seed=1), rand(140, 72, seed=2), rand(140, 72, seed=3)
    assert same(D.linear(x, w, residual=r), D.linear(pitched(x, 8), w, residual=pitched(r, 56)))
    a, b = D.linear_backward(dy, x, w), D.linear_backward(pitched(dy, 8), pitched(x, 24), w)
    assert same(a[0], b[0]) and same(a[1], b[1])


def test_offsets_past_32_bits(D):
    """Rows whose element offsets pass 2^32."""
    pitch = 1 << 28
    big = torch.empty(17 * pitch + 256, dtype=BF, device="cuda")
    x = rand(18, 256)
    v = big[: 17 * pitch + 256].as_strided((18, 256), (pitch, 1))
    v.copy_(x)
    w, n = rand(64, 256, seed=1), rand(256, seed=2)
    assert same(D.linear(v, w), D.linear(x, w))
    assert same(D.rms_norm(v, n, v).y, D.rms_norm(x, n, x).y)
    w13, w2 = rand(80, 256, seed=3), rand(256, 40, seed=4)
    assert same(D.gated_ffn(v, w13, w2, residual=v), D.gated_ffn(x, w13, w2, residual=x))


def test_values_next_to_the_edges_do_not_leak(D):
    """NaN and infinities in rows and weights only reach their own rows and
    columns, at sizes whose last tile is ragged."""
    for rows in (3, 131, 300):
        x, w = rand(rows, 136), rand(77, 136, seed=1)
        clean = D.linear(x, w)
        x2, w2 = x.clone(), w.clone()
        x2[rows - 1, 5] = float("nan")
        w2[76, 100] = float("inf")
        y = D.linear(x2, w2)
        assert y[rows - 1].isnan().all() and not y[: rows - 1, 76].isfinite().any()
        assert same(y[: rows - 1, :76], clean[: rows - 1, :76])


# ---- gated feed-forward

FFN = [(1, 8, 8), (1, 2048, 768), (2, 136, 520), (4, 256, 128), (67, 136, 72), (130, 264, 200), (257, 520, 1032), (600, 256, 768), (33, 2880, 136), (2500, 264, 2568), (1000, 1032, 1096)]


@pytest.mark.parametrize("rows,h,i", FFN)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("add", [False, True])
def test_gated_ffn(D, rows, h, i, dt, add):
    act = ["silu", "gelu_tanh", "relu", "gelu", "none"][(rows + h) % 5]
    x, w13, w2 = rand(rows, h, dt=dt), rand(2 * i, h, seed=1, scale=h**-0.5, dt=dt), rand(h, i, seed=2, scale=i**-0.5, dt=dt)
    res = rand(rows, h, seed=3, dt=dt) if add else None
    y, gu = D.gated_ffn(x, w13, w2, act, res, save=True)
    want = R.gated_ffn(x, w13, w2, act, res, dt)
    R.check(gu, want["gu"], "gu")
    R.check(y, want["y"], "y")
    assert same(D.gated_ffn(x, w13, w2, act, res), y)


@pytest.mark.parametrize("rows,h,i", FFN)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_ffn_backward(D, rows, h, i, dt, act):
    x, w13, w2 = rand(rows, h, dt=dt), rand(2 * i, h, seed=1, scale=h**-0.5, dt=dt), rand(h, i, seed=2, scale=i**-0.5, dt=dt)
    dy = rand(rows, h, seed=4, dt=dt)
    _, gu = D.gated_ffn(x, w13, w2, act, save=True)
    got = D.gated_ffn_backward(dy, x, w13, w2, gu, act)
    want = R.gated_ffn_backward(dy, x, w13, w2, gu, act, dt)
    for g, name in zip(got, ("dx", "dw13", "dw2")):
        R.check(g, want[name], name)
    again = D.gated_ffn_backward(pitched(dy, 8), pitched(x, 8), w13, w2, gu, act)
    assert all(same(a, b) for a, b in zip(got, again))


def test_gated_ffn_gradient_matches_differences(D):
    """The loss sum(dy * y) along a direction of x, by central differences of
    the forward call.  y is fp16, so each loss carries up to 2^-11 of
    sum |dy y| (and as much again from h); the third-order term of a step of
    2^-4 is below 2^-8 of the first at these scales."""
    x, w13, w2 = rand(16, 64, dt=HF), rand(96, 64, seed=1, scale=0.125, dt=HF), rand(64, 48, seed=2, scale=0.15, dt=HF)
    dy, v = rand(16, 64, seed=3, dt=HF), rand(16, 64, seed=4, dt=HF)
    y, gu = D.gated_ffn(x, w13, w2, save=True)
    dx = D.gated_ffn_backward(dy, x, w13, w2, gu)[0]
    f = lambda a: (D.gated_ffn(a, w13, w2).double() * dy.double()).sum().item()  # noqa: E731
    up, down = (x.double() + v.double() / 16).to(HF), (x.double() - v.double() / 16).to(HF)
    step = up.double() - down.double()
    first = (dx.double() * step).sum().item()
    h_noise = (dy.double().abs() @ w2.double().abs()) * R.gated_ffn(x, w13, w2, "silu", None, HF)["gu"].v[:, 48:].abs()
    bound = 2 * 2.0**-11 * ((dy.double() * y.double()).abs().sum() + h_noise.sum()).item() + 2.0**-8 * (dx.double() * step).abs().sum().item()
    assert abs(f(up) - f(down) - first) <= bound


# ---- rows that are not there, streams, graphs, refusals


def test_no_rows(D):
    x, w = rand(4, 64)[:0], rand(24, 64, seed=1)
    n = D.rms_norm(x, rand(64), x, quant=True, save=True)
    assert n.y.shape == (0, 64) and n.scale.shape == (0, 1)
    dx, dw = D.rms_norm_backward(x, x, rand(64), n.rstd)
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert D.linear(x, w).shape == (0, 24)
    dx, dw, db = D.linear_backward(rand(2, 24)[:0], x, w, bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    w13, w2 = rand(32, 64), rand(64, 16)
    y, gu = D.gated_ffn(x, w13, w2, save=True)
    assert y.shape == (0, 64)
    dx, dw13, dw2 = D.gated_ffn_backward(x, x, w13, w2, gu)
    assert (dw13 == 0).all() and (dw2 == 0).all()


def _all(D, x, w, w13, w2, **kw):
    n = D.rms_norm(x, w[0].contiguous(), x, quant=True, save=True, **kw)
    y, z = D.linear(n.y, w, act="silu", save=True, **kw)
    f, gu = D.gated_ffn(n.y, w13, w2, residual=x, save=True, **kw)
    return [n.y, n.codes, y, f, *D.linear_backward(y, n.y, w, z, "silu", bias=True, **kw),
            *D.gated_ffn_backward(f, n.y, w13, w2, gu, **kw), *D.rms_norm_backward(f, n.sum, w[0].contiguous(), n.rstd, **kw)]


@pytest.mark.parametrize("rows", [1, 300])
def test_other_stream_and_graph(D, rows):
    """The same bits on another stream (given as an argument) and from a
    captured graph replayed on new inputs."""
    x, w, w13, w2 = rand(rows, 256), rand(136, 256, seed=1, scale=0.06), rand(144, 256, seed=2, scale=0.06), rand(256, 72, seed=3, scale=0.1)
    want = [t.clone() for t in _all(D, x, w, w13, w2)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = _all(D, x, w, w13, w2, stream=s)
    s.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    buf = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _all(D, buf, w, w13, w2)
    buf.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(out, want))


def test_refusals(D):
    from host_paged_expert_gb300 import PEError

    x, w, n = rand(4, 64), rand(24, 64, seed=1), rand(64, seed=2)
    w13, w2 = rand(32, 64), rand(64, 16)
    for call in (
        lambda: D.rms_norm(x.float(), n.float()),
        lambda: D.rms_norm(x, n.half()),
        lambda: D.rms_norm(x, n[:32]),
        lambda: D.rms_norm(x, n, x[:3]),
        lambda: D.rms_norm(x[:, :60], n[:60].contiguous()),
        lambda: D.rms_norm(x.t(), rand(4)),
        lambda: D.rms_norm(x.view(2, 2, 64), n),
        lambda: D.rms_norm_backward(x, x, n, torch.ones(3, device="cuda")),
        lambda: D.linear(x, w.t()),
        lambda: D.linear(x, w, act="tanh"),
        lambda: D.linear(x, w, bias=n),
        lambda: D.linear(x, w, residual=x),
        lambda: D.linear(x, w, x_scale=torch.ones(4, 1, device="cuda"), w_scale=torch.ones(1, 1, device="cuda")),
        lambda: D.linear(x.to(F8), w.to(F8)),
        lambda: D.linear(x, w, out_dtype=HF),
        lambda: D.linear(x.cpu(), w),
        lambda: D.linear(x, w.cpu()),
        lambda: D.linear_backward(rand(4, 24), x, w, act="silu"),
        lambda: D.gated_ffn(x, w13, w2[:, :8]),
        lambda: D.gated_ffn(x, w13[:31], w2),
        lambda: D.gated_ffn(rand(4, 60), rand(32, 60), rand(60, 16)),
        lambda: D.gated_ffn_backward(x, x, w13, w2, rand(4, 16)),
    ):
        with pytest.raises(PEError):
            call()


# ---- together


def test_paged_block(D):
    """A decoder layer's second half: dense operators around the paged
    experts, against the same formulas in 64 bits from what each stage read."""
    import gpu_util as gu
    from host_paged_expert_gb300 import _lib, synth
    from host_paged_expert_gb300.block import PagedBlock

    s = synth.TINY
    wts = synth.ExpertWeights(s, seed=3)
    moe = _lib.PagedMoE(s, max_tokens=40)
    for e in range(s.num_experts):
        moe.load_expert(0, e, wts.row(0, e))
    H, I, Q = s.hidden, s.intermediate, 384
    wq, wqs = quantised(rand(Q, H, seed=9, scale=0.06), 128)
    b = PagedBlock(moe, 0, wo=rand(H, 128, seed=1, scale=0.1), norm=rand(H, seed=2), router=rand(s.num_experts, H, seed=3, scale=0.06),
                   w13=rand(2 * I, H, seed=4, scale=0.06), w2=rand(H, I, seed=5, scale=0.1), next_norm=rand(H, seed=6), wq=wq, wq_scale=wqs)
    for t in (1, 3, 40):
        attn, res = rand(t, 128, seed=7), rand(t, H, seed=8)
        proj, stream = b.forward(attn, res)
        a = D.linear(attn, b.wo)
        R.check(a, R.linear(attn, b.wo, None, "none", None, BF, BF)["y"], "wo")
        n = D.rms_norm(a, b.norm, res)
        logits = D.linear(n.y, b.router, out_dtype=torch.float32)
        R.check(logits, R.linear(n.y, b.router, None, "none", None, BF, torch.float32)["y"], "router")
        routed = moe.forward(0, n.y, logits)
        out = D.gated_ffn(n.y, b.w13, b.w2, residual=routed)
        R.check(out, R.gated_ffn(n.y, b.w13, b.w2, "silu", routed, BF)["y"], "ffn")
        m = D.rms_norm(out, b.next_norm, n.sum, y=False, quant=True)
        assert same(stream, m.sum)
        R.check(proj, R.linear(m.codes, wq, None, "none", None, BF, BF, m.scale, wqs)["y"], "projections")
    assert moe.stats(0)["error_word"] == 0
    moe.close()


def test_dense_block_backward(D):
    """DenseBlock's gradients against the formulas, chained in 64 bits from
    the 16-bit tensors that each stage kept; then descent with a step that is
    halved whenever it would not lower the loss: it has to find such steps."""
    from host_paged_expert_gb300.block import DenseBlock

    H, I, T = 128, 192, 200
    b = DenseBlock(norm=torch.ones(H, dtype=BF, device="cuda"), w13=rand(2 * I, H, seed=1, scale=H**-0.5), w2=rand(H, I, seed=2, scale=I**-0.5))
    x, target = rand(T, H, seed=3), rand(T, H, seed=4)
    out, (n, gu) = b.forward(x)
    dy = (out.float() - target.float()).to(BF)
    dx, g = b.backward(dy, (n, gu))
    f = R.gated_ffn_backward(dy, n.y, b.w13, b.w2, gu, "silu", BF)
    R.check(g["w13"], f["dw13"], "dw13")
    R.check(g["w2"], f["dw2"], "dw2")
    dn = D.gated_ffn_backward(dy, n.y, b.w13, b.w2, gu)[0]
    r = R.rms_norm_backward(dn, x, b.norm, n.rstd, dy, BF)
    R.check(dx, r["dx"], "dx")
    R.check(g["norm"], r["dw"], "dnorm")

    def loss_at():
        o, saved = b.forward(x)
        d = o.float() - target.float()
        return d.square().mean().item(), d, saved

    master = {k: getattr(b, k).float() for k in ("norm", "w13", "w2")}
    first, d, saved = loss_at()
    now, step = first, 0.5 / T
    for _ in range(20):
        _, g = b.backward(d.to(BF), saved)
        while step > 1e-9:
            for k in master:
                setattr(b, k, (master[k] - step * g[k].float()).to(BF))
            new, d2, saved2 = loss_at()
            if new < now:
                break
            step /= 2
        else:
            pytest.fail("no step along the negative gradient lowers the loss")
        master = {k: getattr(b, k).float() for k in master}
        now, d, saved = new, d2, saved2
    assert now < first
