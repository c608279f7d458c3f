"""The operators of resident experts and 4-bit products on the GPU against
their 64-bit forms (tests/experts_ref.py derives the bounds)."""

import pytest

torch = pytest.importorskip("torch")

import dense_ref as R  # noqa: E402
import experts_ref as X  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]
FMTS = ["int4", "mxfp4", "nvfp4"]


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from host_paged_expert_gb300 import dense

    yield dense
    assert dense.error_word() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(*shape, seed=0, scale=1.0, dt=BF):
    return (torch.randn(*shape, generator=gen(seed * 7919 + shape[0] + 31 * shape[-1]), device="cuda") * scale).to(dt)


def ints(lo, hi, shape, seed=0, dt=torch.uint8):
    return torch.randint(lo, hi, shape, generator=gen(seed * 104729 + shape[0]), device="cuda", dtype=dt)


def pitched(t, extra):
    """The same matrix with a wider row pitch, NaN in between."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device, dtype=F32).to(t.dtype)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- rows to experts and back

ROWS = [(1, 1, 8), (1, 8, 2048), (3, 2, 136), (7, 10, 264), (33, 8, 2880), (130, 17, 72), (2, 3, 8200), (1021, 4, 1032)]


def places(t, k, seed=0):
    return torch.randperm(t * k, generator=gen(seed), device="cuda").view(t, k).int()


@pytest.mark.parametrize("t,k,h", ROWS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_rows(D, t, k, h, dt):
    x, y, res, place = rand(t, h, dt=dt), rand(t * k, h, seed=1, dt=dt), rand(t, h, seed=2, dt=dt), places(t, k)
    w = torch.softmax(rand(t, k, seed=3, dt=F32), 1)
    xs = D.expand_rows(x, place)
    assert same(xs[place.flatten().long()], x.repeat_interleave(k, 0))
    R.check(D.combine_rows(y, place, w, res), X.combine(y, place, w, res, dt), "out")
    R.check(D.combine_rows(y, place), X.combine(y, place, None, None, dt), "sum")
    d = rand(t, h, seed=4, dt=dt)
    dy, dw = D.combine_rows_backward(d, y, place, w)
    want = X.combine_backward(d, y, place, w, dt)
    R.check(dy[place.long()], want[0], "dy")
    R.check(dw, want[1], "dw")
    again = D.combine_rows_backward(d, y, place, w)
    assert same(dy, again[0]) and same(dw, again[1])
    # wider pitches
    p = lambda m: pitched(m, 8)  # noqa: E731
    assert same(D.expand_rows(p(x), place), xs)
    assert same(D.combine_rows(p(y), place, w, p(res)), D.combine_rows(y, place, w, res))
    b = D.combine_rows_backward(p(d), p(y), place, w)
    assert same(b[0], dy) and same(b[1], dw)


def test_rows_left_out(D):
    """Entries without a row: skipped, whatever their weight; rows without an
    entry are not written."""
    t, k, h, rows = 5, 3, 72, 9
    place = torch.tensor([[0, -1, 4], [9, 100, 2**31 - 1], [8, 7, -(2**31)], [1, 3, 5], [-1, -1, -1]], device="cuda", dtype=torch.int32)
    x, y, d = rand(t, h), rand(rows, h, seed=1), rand(t, h, seed=2)
    w = rand(t, k, dt=F32)
    w[place < 0] = float("nan")
    there = (place >= 0) & (place < rows)
    xs = D.expand_rows(x, place, rows)
    assert same(xs[place[there].long()], x.repeat_interleave(k, 0)[there.flatten()])
    out = D.combine_rows(y, place, w)
    R.check(out, X.combine(y, place, torch.where(there, w, torch.zeros_like(w)), None, BF), "out")
    assert (out[1] == 0).all() and (out[4] == 0).all()
    dy, dw = D.combine_rows_backward(d, y, place, w)
    assert (dw[~there] == 0).all() and torch.isfinite(dw).all()
    for a in range(t):
        for b in range(k):
            if there[a, b]:
                want = w[a, b].double() * d[a].double()
                R.check(dy[place[a, b]], R.Q(want, 2.0**-24 * want.abs()).rounded(BF), "dy")


def test_rows_empty(D):
    z = torch.zeros(0, 4, device="cuda", dtype=torch.int32)
    assert D.expand_rows(rand(1, 64)[:0], z).shape == (0, 64)
    assert D.combine_rows(rand(1, 64)[:0], z).shape == (0, 64)
    out = D.combine_rows(rand(1, 64)[:0], torch.zeros(3, 4, device="cuda", dtype=torch.int32), residual=rand(3, 64))
    assert same(out, rand(3, 64))


def test_rows_past_32_bits(D):
    """Row offsets past 2^32 bytes and past 2^31 elements."""
    h, rows = 8192, 262144 + 5
    y = torch.zeros(rows, h, device="cuda", dtype=BF)
    y[-1] = rand(1, h)[0]
    place = torch.tensor([[rows - 1, 0]], device="cuda", dtype=torch.int32)
    assert same(D.combine_rows(y, place)[0], y[-1])
    xs = D.expand_rows(rand(1, h, seed=1), place, rows)
    assert same(xs[-1], rand(1, h, seed=1)[0])


# ---- route


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 4, 4), (1, 128, 8), (8, 128, 8), (31, 16, 2), (33, 33, 5), (128, 64, 6), (129, 64, 6), (200, 100, 3),
                                   (1000, 256, 8), (4096, 130, 4), (5000, 512, 16), (700, 1024, 32), (20000, 8, 2)])
def test_route(D, t, e, k):
    lg = (rand(t, e, dt=F32) * 8).round() / 4  # ties
    r = D.route(lg, k)
    ids, w, offsets, place = X.route(lg, k)
    assert torch.equal(r.ids, ids) and torch.equal(r.offsets, offsets) and torch.equal(r.place, place)
    R.check(r.weights, w, "weights")
    again = D.route(pitched(lg, 3), k)
    assert all(same(a, b) for a, b in zip(r, again))
    dw = rand(t, k, seed=1, dt=F32)
    R.check(D.route_backward(dw, r.weights, r.ids, e), X.route_backward(dw, r.weights, r.ids, e), "dlogits")


def test_route_odd_logits(D):
    inf, nan = float("inf"), float("nan")
    lg = torch.tensor([[nan, 1, 2, nan, -inf, 3], [nan] * 6, [-inf] * 6, [inf, 0, inf, 1, 2, 3], [0.0, -0.0, 0.0, -0.0, -1, -2], [-inf, 5, -inf, nan, -inf, -inf],
                       [3e38, -3e38, 1e-45, -1e-45, 0, 1e38]], device="cuda")
    for k in (1, 3, 6):
        r = D.route(lg, k)
        ids, w, offsets, place = X.route(lg, k)
        assert torch.equal(r.ids, ids) and torch.equal(r.offsets, offsets) and torch.equal(r.place, place)
        R.check(r.weights, w, "weights")


def test_route_nothing(D):
    r = D.route(torch.zeros(0, 16, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and (r.offsets == 0).all() and r.offsets.shape == (17,)
    assert D.route_backward(r.weights, r.weights, r.ids, 16).shape == (0, 16)


def test_route_backward_odd_ids(D):
    """An expert named twice gets both gradients; an id that is none gets nothing."""
    ids = torch.tensor([[3, 3, 0], [7, -1, 8], [2**31 - 1, 5, 5]], device="cuda", dtype=torch.int32)
    w, dw = torch.softmax(rand(3, 3, dt=F32), 1), rand(3, 3, seed=1, dt=F32)
    got = D.route_backward(dw, w, ids, 8)
    for t in range(3):
        one = X.route_backward(dw[t : t + 1], w[t : t + 1], torch.arange(3, device="cuda")[None], 3)
        want = torch.zeros(8, dtype=torch.float64, device="cuda")
        bound = torch.full_like(want, 1e-37)
        for i in range(3):
            if 0 <= ids[t, i] < 8:
                want[ids[t, i]] += one.v[0, i]
                bound[ids[t, i]] += one.b[0, i] + 2.0**-23 * one.v[0].abs().sum()
        R.check(got[t], R.Q(want, bound), "dlogits")


def test_route_gradient_against_differences(D):
    t, e, k = 5, 12, 3
    lg = rand(t, e, dt=F32)
    r = D.route(lg, k)
    c = rand(t, k, seed=1, dt=F32)
    g = D.route_backward(c, r.weights, r.ids, e)
    step = 1e-5
    for j in range(e):
        d = []
        for s in (step, -step):
            m = lg.double()
            m[:, j] += s
            w = torch.softmax(m.gather(1, r.ids.long()), 1)
            d.append((w * c.double()).sum(1))
        # central differences: third derivatives of a softmax are at most 1, times |c|
        want = (d[0] - d[1]) / (2 * step)
        assert ((g[:, j].double() - want).abs() <= (1e-9 + 1e-6) * c.abs().sum(1).double()).all()


# ---- products grouped by expert

# rows of each group
SIZES = [[1], [8], [0, 3, 0], [33, 0, 31, 32, 1], [64, 65, 63, 0, 0, 128], [256, 1, 255, 257], [700, 0, 300], [0, 0, 2049, 17], [3] * 70]


def offsets_of(sizes):
    o = torch.zeros(len(sizes) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(sizes).cumsum(0)
    return o.cuda()


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s[:6])))
@pytest.mark.parametrize("k,n", [(8, 8), (64, 256), (136, 72), (200, 520)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_grouped_linear(D, sizes, k, n, dt):
    rows, g = sum(sizes), len(sizes)
    x, w, dy = rand(rows, k, dt=dt), rand(g, n, k, seed=1, scale=k**-0.5, dt=dt), rand(rows, n, seed=2, dt=dt)
    off = offsets_of(sizes)
    y = D.grouped_linear(x, w, off)
    R.check(y, X.grouped_linear(x, w, off, dt), "y")
    dx, dw = D.grouped_linear_backward(dy, x, w, off)
    want = X.grouped_linear_backward(dy, x, w, off, dt)
    R.check(dx, want["dx"], "dx")
    R.check(dw, want["dw"], "dw")
    assert same(D.grouped_linear(pitched(x, 8), w, off), y)
    b = D.grouped_linear_backward(pitched(dy, 16), pitched(x, 8), w, off)
    assert same(b[0], dx) and same(b[1], dw)


@pytest.mark.parametrize("rows,g,k,n", [(512, 128, 264, 328), (3000, 4, 1032, 776), (2048, 200, 72, 136), (16, 1024, 64, 64)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_grouped_linear_more(D, rows, g, k, n, dt):
    cut = torch.sort(ints(0, rows + 1, (g - 1,), dt=torch.int32)).values.tolist()
    sizes = [b - a for a, b in zip([0] + cut, cut + [rows])]
    x, w, dy = rand(rows, k, dt=dt), rand(g, n, k, seed=1, scale=k**-0.5, dt=dt), rand(rows, n, seed=2, dt=dt)
    off = offsets_of(sizes)
    R.check(D.grouped_linear(x, w, off), X.grouped_linear(x, w, off, dt), "y")
    dx, dw = D.grouped_linear_backward(dy, x, w, off)
    want = X.grouped_linear_backward(dy, x, w, off, dt)
    R.check(dx, want["dx"], "dx")
    R.check(dw, want["dw"], "dw")


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s[:6])))
@pytest.mark.parametrize("h,i", [(64, 64), (136, 72), (264, 200)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_grouped_ffn(D, sizes, h, i, dt):
    rows, g = sum(sizes), len(sizes)
    act = ACTS[(rows + h) % 5]
    x, w13, w2 = rand(rows, h, dt=dt), rand(g, 2 * i, h, seed=1, scale=h**-0.5, dt=dt), rand(g, h, i, seed=2, scale=i**-0.5, dt=dt)
    off = offsets_of(sizes)
    y, gu = D.grouped_ffn(x, w13, w2, off, act, save=True)
    want = X.grouped_ffn(x, w13, w2, off, act, dt)
    R.check(gu, want["gu"], "gu")
    R.check(y, want["y"], "y")
    assert same(D.grouped_ffn(pitched(x, 8), w13, w2, off, act), y)
    dy = rand(rows, h, seed=3, dt=dt)
    got = D.grouped_ffn_backward(dy, x, w13, w2, gu, off, act)
    want = X.grouped_ffn_backward(dy, x, w13, w2, gu, off, act, dt)
    for v, name in zip(got, ("dx", "dw13", "dw2")):
        R.check(v, want[name], name)
    again = D.grouped_ffn_backward(pitched(dy, 8), pitched(x, 8), w13, w2, gu, off, act)
    assert all(same(a, b) for a, b in zip(got, again))


def test_groups_keep_to_themselves(D):
    """NaN in one group's rows and weights, in rows of no group and behind the
    operands' ends reaches nothing else."""
    sizes, k, n = [5, 40, 0, 70, 3, 64, 9], 72, 136
    rows, off = sum(sizes) + 20, offsets_of(sizes) + 7  # seven rows ahead of the first group, thirteen after the last
    x, w, dy = rand(rows, k), rand(7, n, k, seed=1, scale=0.1), rand(rows, n, seed=2)
    ref, back = D.grouped_linear(x, w, off), D.grouped_linear_backward(dy, x, w, off)
    o = off.tolist()
    bad = 3
    x2, w2, dy2 = x.clone(), w.clone(), dy.clone()
    nan = float("nan")
    for m in (x2, dy2):
        m[: o[0]] = nan
        m[o[7] :] = float("inf")
        m[o[bad] : o[bad + 1]] = nan
    w2[bad] = nan
    w2[2] = nan  # an empty group's
    y, (dx, dw) = D.grouped_linear(x2, w2, off), D.grouped_linear_backward(dy2, x2, w2, off)
    for g in range(7):
        s = slice(o[g], o[g + 1])
        if g == bad:
            assert y[s].isnan().all() and dx[s].isnan().all() and dw[g].isnan().all()
        else:
            assert same(y[s], ref[s]) and same(dx[s], back[0][s]) and same(dw[g], back[1][g])
    assert (dw[2] == 0).all()


def test_rows_of_no_group_stay(D):
    """The C call leaves rows of no group as they were."""
    from host_paged_expert_gb300._lib import lib

    sizes, k, n = [5, 40, 70], 72, 136
    rows, off = 200, offsets_of(sizes) + 7
    x, w, out = rand(rows, k), rand(3, n, k, seed=1), torch.full((rows, n), 3.0, device="cuda", dtype=BF)
    st = torch.cuda.current_stream().cuda_stream
    assert lib().pe_grouped_linear(x.data_ptr(), k, w.data_ptr(), off.data_ptr(), out.data_ptr(), rows, 3, k, n, 0, st) == 0
    assert (out[:7] == 3).all() and (out[122:] == 3).all()
    assert same(out[7:122], D.grouped_linear(x, w, off)[7:122])


@pytest.mark.parametrize("raw", [[0, 0, 0, 0], [-5, 10, 20, 100000], [0, 50, 20, 60], [2**31 - 1] * 4, [-(2**31), 2**31 - 1, 0, -1], [60, 40, 20, 0]])
def test_offsets_that_are_none(D, raw):
    """Clamped to the rows and never decreasing."""
    rows, k, n = 60, 64, 72
    x, w, dy = rand(rows, k), rand(3, n, k, seed=1), rand(rows, n, seed=2)
    clean, high = [], 0
    for v in raw:
        high = max(high, min(max(v, 0), rows))
        clean.append(high)
    o, c = torch.tensor(raw, dtype=torch.int32, device="cuda"), torch.tensor(clean, dtype=torch.int32, device="cuda")
    a, b = D.grouped_linear(x, w, o), D.grouped_linear(x, w, c)
    s = slice(clean[0], clean[3])
    assert same(a[s], b[s])
    a, b = D.grouped_linear_backward(dy, x, w, o), D.grouped_linear_backward(dy, x, w, c)
    assert same(a[0][s], b[0][s]) and same(a[1], b[1])


def test_grouped_nothing(D):
    w, off = rand(3, 64, 72), torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = rand(1, 72)[:0], rand(1, 64)[:0]
    assert D.grouped_linear(x, w, off).shape == (0, 64)
    dx, dw = D.grouped_linear_backward(dy, x, w, off)
    assert dx.shape == (0, 72) and (dw == 0).all()
    w13, w2 = rand(3, 32, 72), rand(3, 72, 16)
    y, gu = D.grouped_ffn(x, w13, w2, off, save=True)
    assert y.shape == (0, 72) and gu.shape == (0, 32)
    got = D.grouped_ffn_backward(x, x, w13, w2, gu, off)
    assert got[0].shape == (0, 72) and (got[1] == 0).all() and (got[2] == 0).all()


def test_grouped_gradient_against_differences(D):
    """The loss <y, c> along random directions, in fp16 with steps that it holds."""
    sizes, h, i = [5, 0, 9, 1], 64, 40
    rows, off = sum(sizes), offsets_of(sizes)
    x, w13, w2 = rand(rows, h, dt=HF), rand(4, 2 * i, h, seed=1, scale=0.1, dt=HF), rand(4, h, i, seed=2, scale=0.1, dt=HF)
    c = rand(rows, h, seed=3, dt=HF)
    y, gu = D.grouped_ffn(x, w13, w2, off, "silu", save=True)
    grads = D.grouped_ffn_backward(c, x, w13, w2, gu, off, "silu")

    def loss(a, b, d):
        total = 0.0
        for g, s in enumerate(X._groups(off)):
            z = a[s] @ b[g].t()
            f, _ = R.phi("silu", z[:, :i])
            total = total + ((f * z[:, i:]) @ d[g].t() * c[s].double()).sum()
        return total

    at = [t.double() for t in (x, w13, w2)]
    for which, g in enumerate(grads):
        u = torch.randn(g.shape, generator=gen(which), device="cuda", dtype=torch.float64)
        step = 1e-5
        lo, hi = [[t + s * u if j == which else t for j, t in enumerate(at)] for s in (-step, step)]
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        # each element of the gradient is off by a few of fp16's half steps, independent of u
        off_by = 8 * 2.0**-11 * (g.double() * u).norm() + 1e-6 * want.abs()
        assert (want - (g.double() * u).sum()).abs() <= off_by


# ---- 4-bit weights

W4 = [(1, 32, 1), (1, 64, 16), (2, 96, 17), (3, 160, 100), (8, 2048, 128), (9, 4096, 40), (16, 288, 264), (17, 2880, 136), (33, 544, 72), (64, 1056, 200),
      (1, 8192, 33), (65, 288, 136), (130, 1056, 200), (300, 96, 77)]


def weights(fmt, n, k, seed=0):
    codes = ints(0, 256, (n, k // 2), seed=seed + n)
    shape = (n, -(-k // X.GROUP[fmt]))
    if fmt == "int4":
        return codes, (rand(*shape, seed=seed, dt=F32) * 0.02).half(), None
    if fmt == "mxfp4":
        return codes, ints(115, 124, shape, seed=seed), None
    return codes, rand(*shape, seed=seed, dt=F32).to(F8), rand(1, seed=seed + 5, scale=0.02, dt=F32)


@pytest.mark.parametrize("rows,k,n", W4)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("full", [False, True])
def test_linear_w4(D, rows, k, n, fmt, dt, full):
    act = ACTS[(rows + k + n) % 5] if full else "none"
    c, s, ts = weights(fmt, n, k)
    x = rand(rows, k, dt=dt)
    b, res = (rand(n, seed=2, dt=dt), rand(rows, n, seed=3, dt=dt)) if full else (None, None)
    w = X.values(c, s, fmt, ts)
    y = D.linear_w4(x, c, s, fmt, b, act, res, tensor_scale=ts)
    R.check(y, X.linear_w4(x, w, b, act, res, dt, dt, rows > 128), "y")
    assert same(D.linear_w4(pitched(x, 8), c, s, fmt, b, act, res, tensor_scale=ts), y)
    f = D.linear_w4(x, c, s, fmt, b, act, res, tensor_scale=ts, out_dtype=F32)
    R.check(f, X.linear_w4(x, w, b, act, res, dt, F32, rows > 128), "y in fp32")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_every_code_and_scale(D, fmt, dt):
    """Rows of the identity pick single weights: every code with every scale
    that the element type holds, exactly."""
    k = 32
    if fmt == "int4":
        s = torch.tensor([0.0, 2.0**-14, 6e-8, 0.001, 1.0, 100.0, 0.333, -0.5], device="cuda").half()[:, None]
    elif fmt == "mxfp4":
        e = torch.arange(0, 247) if dt == BF else torch.arange(104, 141)
        s = e.to(torch.uint8).cuda()[:, None]
    else:
        e = torch.arange(256, dtype=torch.uint8)
        e = e[(e & 127) != 127].cuda()  # without the NaNs
        s = torch.stack([e, e.flip(0)], 1)
    ts = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
    n = s.shape[0]
    q = torch.arange(16, dtype=torch.uint8, device="cuda")
    q = torch.cat([q, q.flip(0)])
    codes = (q[0::2] | (q[1::2] << 4))[None].expand(n, 16).contiguous()
    w = X.values(codes, s, fmt, ts)
    eye = torch.eye(k, device="cuda", dtype=dt)
    got = D.linear_w4(eye, codes, s, fmt, tensor_scale=ts, out_dtype=F32)
    want = w.t()
    # fp32's own range: E8M0 times E2M1 may be subnormal or lie past it
    keep = (want.abs() < 2.0**127) & ((want == 0) | (want.abs() >= 2.0**-120))
    assert torch.equal(got.double()[keep], want[keep])


def test_scales_that_are_nan(D):
    """A NaN scale stays in its row."""
    k, n = 128, 24
    for fmt in FMTS:
        c, s, ts = weights(fmt, n, k)
        s = s.clone()
        if fmt == "int4":
            s[5, 0] = float("nan")
        else:
            s.view(torch.uint8)[5, 1] = 255 if fmt == "mxfp4" else 127
        for rows in (3, 40, 150):
            y = D.linear_w4(rand(rows, k), c, s, fmt, tensor_scale=ts)
            assert y[:, 5].isnan().all() and torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all()


def test_tokens_keep_to_themselves(D):
    c, s, _ = weights("int4", 40, 256)
    x = rand(9, 256)
    ref = D.linear_w4(x, c, s, "int4")
    x[4] = float("nan")
    x[6, 3] = float("inf")
    y = D.linear_w4(x, c, s, "int4")
    assert y[4].isnan().all() and not torch.isfinite(y[6]).any()
    for t in (0, 1, 2, 3, 5, 7, 8):
        assert same(y[t], ref[t])


def test_eight_bit_scales_as_their_type(D):
    c, s, ts = weights("nvfp4", 40, 256)
    x = rand(3, 256)
    assert same(D.linear_w4(x, c, s, "nvfp4", tensor_scale=ts), D.linear_w4(x, c, s.view(torch.uint8), "nvfp4", tensor_scale=ts))
    c, s, _ = weights("mxfp4", 40, 256)
    assert same(D.linear_w4(x, c, s, "mxfp4"), D.linear_w4(x, c, s.view(torch.float8_e8m0fnu), "mxfp4"))


# ---- streams and graphs


def _calls(D):
    x, off = rand(60, 128), offsets_of([10, 0, 50])
    w, w13, w2 = rand(3, 72, 128, seed=1), rand(3, 80, 128, seed=1, scale=0.1), rand(3, 128, 40, seed=2, scale=0.1)
    lg, dz = rand(30, 3, dt=F32), rand(60, 72, seed=4)
    c, s, _ = weights("int4", 72, 128)

    def run():
        r = D.route(lg, 2)
        xs = D.expand_rows(x[:30], r.place)
        y, gu = D.grouped_ffn(xs, w13, w2, r.offsets, save=True)
        out = D.combine_rows(y, r.place, r.weights, x[:30])
        dy, dw = D.combine_rows_backward(x[:30], y, r.place, r.weights)
        return [*r, xs, y, gu, out, dy, dw, *D.grouped_ffn_backward(dy, xs, w13, w2, gu, r.offsets), D.route_backward(dw, r.weights, r.ids, 3),
                D.grouped_linear(x, w, off), *D.grouped_linear_backward(dz, x, w, off),
                D.linear_w4(x[:5], c, s, "int4"), D.linear_w4(x[:30].repeat(3, 1), c, s, "int4")]

    return run


def test_other_streams(D):
    run = _calls(D)
    ref = run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = run()
    st.synchronize()
    assert all(same(a, b) for a, b in zip(ref, got))


def test_stream_argument(D):
    x, off, w = rand(60, 128), offsets_of([10, 0, 50]), rand(3, 72, 128, seed=1)
    ref = D.grouped_linear(x, w, off)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = D.grouped_linear(x, w, off, stream=st)
    r = D.route(rand(5, 16, dt=F32), 2, stream=st)
    st.synchronize()
    assert same(ref, got) and all(same(a, b) for a, b in zip(r, D.route(rand(5, 16, dt=F32), 2)))


def test_captured(D):
    run = _calls(D)
    ref = run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        graphs.append((g, got))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(same(a, b) for a, b in zip(ref, got))


# ---- the layer


def _block(seed=0, H=128, E=12, I=72, k=3, dt=BF):
    from host_paged_expert_gb300.block import ExpertBlock

    return ExpertBlock(norm=1 + rand(H, seed=seed, scale=0.1, dt=dt), router=rand(E, H, seed=seed + 1, scale=H**-0.5, dt=dt),
                       w13=rand(E, 2 * I, H, seed=seed + 2, scale=H**-0.5, dt=dt), w2=rand(E, H, I, seed=seed + 3, scale=I**-0.5, dt=dt), top_k=k)


@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("dt", [BF, HF])
def test_expert_block(D, T, dt):
    """Each stage of ExpertBlock against the formulas, from what the stage before
    it left."""
    b = _block(dt=dt)
    x, dout = rand(T, 128, seed=9, dt=dt), rand(T, 128, seed=10, dt=dt)
    out, saved = b.forward(x)
    n, r, rows, gu, y = saved
    logits = D.linear(n.y, b.router, out_dtype=F32)
    ids, w, offsets, place = X.route(logits, 3)
    assert torch.equal(r.ids, ids) and torch.equal(r.offsets, offsets) and torch.equal(r.place, place)
    assert same(rows[place.flatten().long()], n.y.repeat_interleave(3, 0))
    want = X.grouped_ffn(rows, b.w13, b.w2, offsets, "silu", dt)
    R.check(y, want["y"], "y")
    R.check(out, X.combine(y, place, r.weights, x, dt), "out")
    dx, g = b.backward(dout, saved)
    dy, dw = D.combine_rows_backward(dout, y, place, r.weights)
    f = X.grouped_ffn_backward(dy, rows, b.w13, b.w2, gu, offsets, "silu", dt)
    R.check(g["w13"], f["dw13"], "dw13")
    R.check(g["w2"], f["dw2"], "dw2")
    dl = D.route_backward(dw, r.weights, r.ids, 12).to(dt)
    lb = R.linear_backward(dl, n.y, b.router, None, "none", dt)
    R.check(g["router"], lb["dw"], "drouter")
    dn = D.combine_rows(D.grouped_ffn_backward(dy, rows, b.w13, b.w2, gu, offsets)[0], place, residual=D.linear_backward(dl, n.y, b.router)[0])
    nb = R.rms_norm_backward(dn, x, b.norm, n.rstd, dout, dt)
    R.check(dx, nb["dx"], "dx")
    R.check(g["norm"], nb["dw"], "dnorm")


def test_expert_block_against_differences(D):
    """The whole layer's gradients along random directions, against central
    differences of the layer's formula in 64 bits with the same choice of
    experts (the choice has no gradient)."""
    T, H, E, I, k = 40, 128, 12, 72, 3
    b = _block(dt=HF)
    x, c = rand(T, H, seed=9, dt=HF), rand(T, H, seed=10, dt=HF)
    out, saved = b.forward(x)
    ids = saved[1].ids.long()
    dx, g = b.backward(c, saved)

    def loss(x, norm, router, w13, w2):
        n = x * (x.square().mean(1, keepdim=True) + b.eps).rsqrt() * norm
        w = torch.softmax((n @ router.t()).gather(1, ids), 1)
        z = torch.einsum("th,tkih->tki", n, w13[ids])
        h = R.phi("silu", z[:, :, :I])[0] * z[:, :, I:]
        return ((x + (torch.einsum("tki,tkhi->tkh", h, w2[ids]) * w[:, :, None]).sum(1)) * c.double()).sum()

    at = [t.double() for t in (x, b.norm, b.router, b.w13, b.w2)]
    for which, got in enumerate((dx, g["norm"], g["router"], g["w13"], g["w2"])):
        u = torch.randn(got.shape, generator=gen(which), device="cuda", dtype=torch.float64)
        lo, hi = [[t + s * u if j == which else t for j, t in enumerate(at)] for s in (-1e-5, 1e-5)]
        want = (loss(*hi) - loss(*lo)) / 2e-5
        # independent roundings to fp16 of the activations and gradients on the way, a
        # dozen of half a step each, and as much again for sums of them
        off_by = 16 * 2.0**-11 * (got.double() * u).norm() + 1e-6 * want.abs()
        assert (want - (got.double() * u).sum()).abs() <= off_by, which


def test_expert_block_serves_as_the_paged_layer(D):
    """The same weights in a paged layer: the same choice and weights, bit for
    bit, and outputs that differ by their roundings alone."""
    import numpy as np

    from host_paged_expert_gb300 import _lib, synth

    s = synth.TINY
    H, E, I, k, T = s.hidden, s.num_experts, s.intermediate, s.top_k, 24
    moe = _lib.PagedMoE(s, max_tokens=T)
    w13, w2 = rand(E, 2 * I, H, seed=1, scale=H**-0.5), rand(E, H, I, seed=2, scale=I**-0.5)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    for e in range(E):
        moe.load_expert(0, e, {"w13": bits(w13[e]), "w2": bits(w2[e])})
    x, logits = rand(T, H, seed=3), rand(T, E, seed=4, dt=F32)
    paged = moe.forward(0, x, logits)
    torch.cuda.synchronize()
    plan = moe.read_plan(0, T)
    r = D.route(logits, k)
    assert np.array_equal(plan["topk_id"].reshape(T, k), r.ids.cpu().numpy())
    assert np.array_equal(plan["topk_w"].reshape(T, k).view(np.int32), r.weights.cpu().numpy().view(np.int32))
    y = D.grouped_ffn(D.expand_rows(x, r.place), w13, w2, r.offsets)
    out = D.combine_rows(y, r.place, r.weights)
    # h in 16 bits or not, y in 16 bits or not, the result's rounding on both sides
    a, p = out.double(), paged.double()
    assert ((a - p).norm(dim=1) / p.norm(dim=1)).max() <= 4 * 2.0**-8
    moe.close()


def test_expert_block_captured(D):
    b = _block()
    x, dout = rand(64, 128, seed=9), rand(64, 128, seed=10)

    def step():
        out, saved = b.forward(x)
        dx, g = b.backward(dout, saved)
        return [out, dx, *g.values()]

    ref = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    x.copy_(rand(64, 128, seed=11))
    g.replay()
    torch.cuda.synchronize()
    assert not same(got[0], ref[0])
    assert all(same(p, q) for p, q in zip(got, step()))


def test_two_host_threads(D):
    """Calls from two threads on two streams: each its own results."""
    import threading

    run = _calls(D)
    ref = run()
    torch.cuda.synchronize()
    wrong = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(10):
                got = run()
                st.synchronize()
                if not all(same(a, b) for a, b in zip(ref, got)):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_products_behind_what_writes_their_arguments(D):
    """A launch right before that makes the weights, the offsets or the rows: a
    block that is there early reads none of them."""
    sizes = [100, 0, 30, 70]
    rows, k, n = 200, 256, 264
    x, w, off = rand(rows, k), rand(4, n, k, seed=1, scale=0.1), offsets_of(sizes)
    c, s, _ = weights("int4", n, k)
    lg = rand(rows, 8, dt=F32)
    ref = [D.grouped_linear(x, w, off), D.linear_w4(x[:5], c, s, "int4"), D.linear_w4(x[:40], c, s, "int4"), *D.route(lg, 2)]
    x2, w2, off2, c2, lg2 = (torch.zeros_like(t) for t in (x, w, off, c, lg))
    for _ in range(20):
        for t in (x2, w2, off2, c2, lg2):
            t.zero_()
        x2.copy_(x), w2.copy_(w), off2.copy_(off)
        got = [D.grouped_linear(x2, w2, off2)]
        c2.copy_(c)
        got.append(D.linear_w4(x2[:5], c2, s, "int4"))
        c2.zero_()
        c2.copy_(c)
        got.append(D.linear_w4(x2[:40], c2, s, "int4"))
        lg2.copy_(lg)
        got += D.route(lg2, 2)
        assert all(same(a, b) for a, b in zip(ref, got))


def test_waits_that_run_out(D):
    """Each role of each kernel in turn gives up: the others follow, nothing
    hangs, and the calls after it are right."""
    for polls in (1, 1 << 12):
        assert D.selftest_expert_waits(polls) == [0x8] * 12  # PE_DEVERR_TIMEOUT
    assert D.error_word() == 0
    x, off, w = rand(60, 128), offsets_of([10, 0, 50]), rand(3, 72, 128, seed=1)
    R.check(D.grouped_linear(x, w, off), X.grouped_linear(x, w, off, BF), "y")
    c, s, _ = weights("int4", 72, 128)
    R.check(D.linear_w4(x, c, s, "int4"), X.linear_w4(x, X.values(c, s, "int4"), None, "none", None, BF, BF, False), "w4")


def test_each_gradient_alone(D):
    """What the C calls leave out on request changes nothing of the rest."""
    from host_paged_expert_gb300._lib import lib

    L, st = lib(), torch.cuda.current_stream().cuda_stream
    sizes, h, i = [5, 0, 70, 33], 136, 72
    rows, g, off = sum(sizes), len(sizes), offsets_of(sizes)
    x, w13, w2, dy = rand(rows, h), rand(g, 2 * i, h, seed=1, scale=0.1), rand(g, h, i, seed=2, scale=0.1), rand(rows, h, seed=3)
    _, gu = D.grouped_ffn(x, w13, w2, off, save=True)
    want = D.grouped_ffn_backward(dy, x, w13, w2, gu, off)
    ws = torch.empty(L.pe_grouped_ffn_backward_workspace(rows, i), dtype=torch.uint8, device="cuda")
    for which in range(3):
        out = torch.full_like(want[which], 7.0)
        at = [out.data_ptr() if j == which else None for j in range(3)]
        assert L.pe_grouped_ffn_backward(dy.data_ptr(), h, x.data_ptr(), h, w13.data_ptr(), w2.data_ptr(), gu.data_ptr(), off.data_ptr(), 1, *at, ws.data_ptr(),
                                         ws.numel(), rows, g, h, i, 0, st) == 0
        assert same(out, want[which])
    w, dz = rand(g, 72, h, seed=4), rand(rows, 72, seed=5)
    want = D.grouped_linear_backward(dz, x, w, off)
    for which in range(2):
        out = torch.full_like(want[which], 7.0)
        at = [out.data_ptr() if j == which else None for j in range(2)]
        assert L.pe_grouped_linear_backward(dz.data_ptr(), 72, x.data_ptr(), h, w.data_ptr(), off.data_ptr(), *at, rows, g, h, 72, 0, st) == 0
        assert same(out, want[which])
    # the weighted sum's: without dweights, and then without y
    place, wt = places(9, 3), rand(9, 3, dt=F32)
    y, d = rand(27, h, seed=6), rand(9, h, seed=7)
    want = D.combine_rows_backward(d, y, place, wt)[0]
    out = torch.full_like(want, 7.0)
    assert L.pe_combine_rows_backward(d.data_ptr(), h, None, 0, place.data_ptr(), wt.data_ptr(), out.data_ptr(), None, 9, 3, 27, h, 0, st) == 0
    assert same(out, want)


def test_many_groups_and_wide_features(D):
    """The most groups that a call takes, and a table that leaves the ring a
    stage less, in each kind of product."""
    g, h, i = 1024, 72, 40
    sizes = [(7 * j) % 5 for j in range(g)]
    rows, off = sum(sizes), offsets_of(sizes)
    x, w13, w2, dy = rand(rows, h), rand(g, 2 * i, h, seed=1, scale=0.1), rand(g, h, i, seed=2, scale=0.1), rand(rows, h, seed=3)
    y, gu = D.grouped_ffn(x, w13, w2, off, save=True)
    want = X.grouped_ffn(x, w13, w2, off, "silu", BF)
    R.check(y, want["y"], "y")
    R.check(gu, want["gu"], "gu")
    want = X.grouped_ffn_backward(dy, x, w13, w2, gu, off, "silu", BF)
    for v, name in zip(D.grouped_ffn_backward(dy, x, w13, w2, gu, off), ("dx", "dw13", "dw2")):
        R.check(v, want[name], name)
    # many feature tiles against one row
    w = rand(2, 20000, 64, seed=4, scale=0.1)
    off = offsets_of([1, 2])
    R.check(D.grouped_linear(x[:3, :64], w, off), X.grouped_linear(x[:3, :64], w, off, BF), "wide")
