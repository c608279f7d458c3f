"""Dense operators on the GPU, in the forms and at the values where a call can
go wrong without a test of whole matrices seeing it."""

import math
import threading

import pytest

torch = pytest.importorskip("torch")

import dense_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
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


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- the activations' tails

# relative error of the value and the slope at z < 0, in fp32: the argument of
# the exponential is off by some roundings of its own size (2^-24 each; six in
# u and its scaling, two in x log2 e), of erfc by z^2 / 2 times three, and the
# functions themselves by 2^-21.  The slope is a sum of two such terms, of
# which the larger is at most 1.5 times it at z <= -3.
TAIL = {
    "silu": lambda z: 2.0**-20 + z.abs() * 2.0**-22,
    "gelu": lambda z: 2.0**-20 + z * z * 2.0**-22,
    "gelu_tanh": lambda z: 2.0**-20 + 1.6 * (z.abs() + 0.045 * z.abs() ** 3) * 2.0**-21,
}


def tail(dt):
    return torch.linspace(-8, -3, 640, device="cuda").to(dt)


def exact(act, z):
    """(act(z), act'(z)) in 64 bits, without cancellation at z < 0."""
    z = z.double()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-k * (z + 0.044715 * z**3)))
    return z * s, s + z * s * (1 - s) * k * (1 + 3 * 0.044715 * z * z)


def through_linear(D, z, act, rows, **kw):
    """act(z) of every value of z, as a product whose z is exact: x = z e_0,
    weight rows e_0."""
    x = torch.zeros(rows, 8, dtype=z.dtype, device="cuda")
    x[:, 0] = z.repeat(-(-rows // len(z)))[:rows]
    w = torch.zeros(16, 8, dtype=z.dtype, device="cuda")
    w[:, 0] = 1
    return D.linear(x, w, act=act, **kw), x[:, 0]


TAILS = [(a, t) for a in TAIL for t in (BF, HF)]


@pytest.mark.parametrize("act,dt", TAILS)
@pytest.mark.parametrize("rows", [1, 3, 640, 20000])
def test_tail_of_the_activation(D, act, dt, rows):
    y, z = through_linear(D, tail(dt), act, rows, out_dtype=F32)
    want = exact(act, z)[0][:, None].expand(rows, 16)
    off = (y.double() - want).abs() / want.abs()
    assert (off <= TAIL[act](z.double())[:, None]).all(), (off / TAIL[act](z.double())[:, None]).max()


@pytest.mark.parametrize("act,dt", TAILS)
def test_tail_of_the_slope(D, act, dt):
    """dbias of one row is the slope, rounded once."""
    z = tail(dt)[None].contiguous()
    one, w = torch.ones_like(z), torch.zeros(z.shape[1], 8, dtype=dt, device="cuda")
    db = D.linear_backward(one, one[:, :8].contiguous(), w, z, act, bias=True)[2].double()
    want = exact(act, z[0])[1]
    bound = (R.U[dt] + 2 * TAIL[act](z[0].double())) * want.abs() + R.TINY[dt]
    assert ((db - want).abs() <= bound).all(), ((db - want).abs() / bound).max()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_huge_arguments(D, act):
    """Values and slopes where z^2 and z^3 pass the range of fp32: z and 1
    above, 0 and 0 below."""
    z = torch.tensor([1e19, 3e19, 1e25, 3e38, -1e19, -3e19, -1e25, -3e38], device="cuda").to(BF)
    y, at = through_linear(D, z, act, 8)
    assert torch.equal(y, torch.where(at > 0, at, 0 * at)[:, None].expand(8, 16))
    one, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(8, 8, dtype=BF, device="cuda")
    db = D.linear_backward(one, one, w, z[None], act, bias=True)[2]
    assert torch.equal(db, (z > 0).to(BF))
    # through the gated block: gate z, up 1, down 1
    x, w13, w2 = torch.zeros(8, 8, dtype=BF, device="cuda"), torch.zeros(16, 8, dtype=BF, device="cuda"), torch.zeros(8, 8, dtype=BF, device="cuda")
    x[:, 0], x[:, 1], w13[0, 0], w13[8, 1], w2[0, 0] = z, 1, 1, 1, 1
    y, gu = D.gated_ffn(x, w13, w2, act, save=True)
    assert torch.equal(y[:, 0], torch.where(z > 0, z, 0 * z))
    dy = torch.zeros_like(x)
    dy[:, 0] = 1
    dx = D.gated_ffn_backward(dy, x, w13, w2, gu, act)[0]
    assert torch.equal(dx[:, 0], (z > 0).to(BF)) and torch.equal(dx[:, 1], torch.where(z > 0, z, 0 * z))


# ---- fp32 results


@pytest.mark.parametrize("rows,k,n", [(5000, 512, 520), (6508, 344, 310), (3001, 72, 1000), (2500, 8, 2047), (4096, 512, 4096)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("full", [False, True])
def test_fp32_results_of_many_rows(D, rows, k, n, dt, full):
    """K of up to 512 and many rows: the kernel of CTA pairs, whole and ragged
    columns."""
    x, w = rand(rows, k, dt=dt), rand(n, k, seed=1, scale=k**-0.5, dt=dt)
    b, res, act = (rand(n, seed=2, dt=dt), rand(rows, n, seed=3, dt=dt), "silu") if full else (None, None, "none")
    y, z = D.linear(x, w, b, act, res, out_dtype=F32, save=True)
    want = R.linear(x, w, b, act, res, dt, F32)
    R.check(y, want["y"], "fp32")
    if full:
        R.check(z, want["z"], "z")
    assert same(D.linear(x, w, b, act, res, out_dtype=F32), y)


# ---- another stream


@pytest.mark.parametrize("rows", [1, 300])
def test_arguments_freed_behind_a_call_on_another_stream(D, rows):
    """Temporaries of a call on a busy stream, freed and their memory asked for
    again before the call's kernels have run."""
    x, w, w13, w2 = rand(rows, 256), rand(136, 256, seed=1), rand(144, 256, seed=2), rand(256, 72, seed=3)
    want = [D.linear(x, w), D.gated_ffn(x, w13, w2, residual=x), D.rms_norm(x, w[0].contiguous(), x).y]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b, c = x.clone(), x.clone(), x.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some ms
    got = [D.linear(a, w, stream=s), D.gated_ffn(b, w13, w2, residual=b, stream=s), D.rms_norm(c, w[0].contiguous(), c, stream=s).y]
    del a, b, c
    over = [torch.full_like(x, float("nan")) for _ in range(8)]
    s.synchronize()
    assert len(over) == 8 and all(same(g, h) for g, h in zip(got, want))


# ---- waits that run out


def test_waits_give_up_and_report(D):
    """Each role of the tensor-core kernels in turn gives up at once, the
    others when their polls run out: the words say so, nothing hangs, and what
    runs next is as it was."""
    x, w, w13, w2 = rand(300, 2048), rand(2048, 2048, seed=1, scale=0.02), rand(512, 2048, seed=2, scale=0.02), rand(2048, 256, seed=3, scale=0.06)
    run = lambda: [D.linear(x, w), D.linear(x[:8], w), D.gated_ffn(x, w13, w2), D.linear(x.repeat(9, 1), w)]  # noqa: E731
    want = run()
    for polls in (1, 1 << 6, 1 << 12):
        assert D.selftest_waits(polls) == [0x8] * 12  # PE_DEVERR_TIMEOUT
    assert D.error_word() == 0
    assert all(same(a, b) for a, b in zip(run(), want))


# ---- every activation's backward pass


@pytest.mark.parametrize("rows,k,n", [(5, 64, 72), (131, 264, 77), (700, 520, 264)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_of_each_activation(D, rows, k, n, dt, act):
    x, w, dy = rand(rows, k, dt=dt), rand(n, k, seed=1, scale=2 * k**-0.5, dt=dt), rand(rows, n, seed=3, dt=dt)
    _, z = D.linear(x, w, act=act, save=True)
    want = R.linear_backward(dy, x, w, z, act, dt)
    for g, name in zip(D.linear_backward(dy, x, w, z, act, bias=True), ("dx", "dw", "db")):
        R.check(g, want[name], name)


@pytest.mark.parametrize("rows,h,i", [(3, 64, 72), (131, 264, 200), (1100, 136, 520)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ACTS)
def test_gated_ffn_backward_of_each_activation(D, rows, h, i, dt, act):
    x, w13, w2 = rand(rows, h, dt=dt), rand(2 * i, h, seed=1, scale=2 * h**-0.5, dt=dt), rand(h, i, seed=2, scale=i**-0.5, dt=dt)
    dy = rand(rows, h, seed=4, dt=dt)
    _, gu = D.gated_ffn(x, w13, w2, act, save=True)
    want = R.gated_ffn_backward(dy, x, w13, w2, gu, act, dt)
    for g, name in zip(D.gated_ffn_backward(dy, x, w13, w2, gu, act), ("dx", "dw13", "dw2")):
        R.check(g, want[name], name)


def test_gradients_that_are_not_wanted(D):
    """The C calls with each gradient alone (which may take another kernel than
    all of them together, so it is the formulas that they are held against)."""
    from host_paged_expert_gb300 import _lib

    L, st = _lib.lib(), torch.cuda.current_stream().cuda_stream
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    x, w, dy = rand(131, 264), rand(77, 264, seed=1, scale=0.06), rand(131, 77, seed=3)
    _, z = D.linear(x, w, act="silu", save=True)
    want = R.linear_backward(dy, x, w, z, "silu", BF)
    for i, k in enumerate(("dx", "dw", "db")):
        out = [None, None, None]
        out[i] = torch.full_like(want[k].v, float("nan"), dtype=BF)
        need = [x if i == 1 else None, w if i == 0 else None]
        assert L.pe_linear_backward(p(dy), 77, p(need[0]), 264, p(need[1]), p(z), 1, *map(p, out), p(ws), ws.numel(), 131, 264, 77, 0, st) == 0
        R.check(out[i], want[k], k)
    h, i_ = 264, 200
    w13, w2, dy = rand(2 * i_, h, seed=1, scale=0.06), rand(h, i_, seed=2, scale=0.06), rand(131, h, seed=4)
    _, gu = D.gated_ffn(x, w13, w2, save=True)
    want = R.gated_ffn_backward(dy, x, w13, w2, gu, "silu", BF)
    for i, k in enumerate(("dx", "dw13", "dw2")):
        out = [None, None, None]
        out[i] = torch.full_like(want[k].v, float("nan"), dtype=BF)
        assert L.pe_gated_ffn_backward(p(dy), h, p(x if i == 1 else None), h, p(w13 if i == 0 else None), p(w2), p(gu), 1, *map(p, out),
                                       p(ws), ws.numel(), 131, h, i_, 0, st) == 0
        R.check(out[i], want[k], k)
    # a norm's results one by one
    n, res = rand(264, seed=5), rand(131, 264, seed=6)
    f = D.rms_norm(x, n, res, quant=True, save=True)
    for k in ("y", "sum", "rstd"):
        out = torch.full_like(getattr(f, k), float("nan"))
        a = {k: p(out)}
        assert L.pe_rms_norm(p(x), 264, p(res), 264, p(n), 1e-6, a.get("y"), a.get("sum"), None, None, a.get("rstd"), 131, 264, 0, st) == 0
        assert same(out, getattr(f, k))


# ---- the order of launches


@pytest.mark.parametrize("rows", [1, 4, 16, 64, 300])
def test_weights_rewritten_right_before(D, rows):
    """gated_ffn behind a launch that has just written w2, by a copy and by a
    product: its second kernel may ask for w2 while the first one runs, no
    earlier."""
    x, w13 = rand(rows, 512), rand(2048, 512, seed=1, scale=0.04)
    a, b, old = rand(512, 512, seed=2, scale=0.05), rand(1024, 512, seed=3), rand(512, 1024, seed=4)
    new = D.linear(a, b)
    torch.cuda.synchronize()
    want = D.gated_ffn(x, w13, new)
    torch.cuda.synchronize()
    for _ in range(20):
        w2 = old.clone()
        torch.cuda.synchronize()
        w2.copy_(new)
        y = D.gated_ffn(x, w13, w2)
        del w2
        stale = torch.full_like(new, float("nan"))
        del stale  # its memory is what the product below writes
        z = D.gated_ffn(x, w13, D.linear(a, b))
        assert same(y, want) and same(z, want)


@pytest.mark.parametrize("rows", [1, 3, 16, 64, 300, 2500])
def test_chains_of_launches(D, rows):
    """Each call reads what the one before it has just written, in a graph with
    nothing between the launches: the bits of calls that wait for each other."""
    h = 512
    x, n, wq = rand(rows, h), rand(h, seed=1), rand(640, h, seed=2, scale=0.05)
    w1, w2, w13, wd = rand(h, 640, seed=3, scale=0.05), rand(h, h, seed=4, scale=0.05), rand(768, h, seed=5, scale=0.05), rand(h, 384, seed=6, scale=0.05)
    codes, cs = (wq / 0.5).to(torch.float8_e4m3fn), torch.full((5, 4), 0.5, device="cuda")
    buf = x.clone()

    def chain(wait):
        out, v = [], buf
        for _ in range(4):
            for step in (
                lambda v: D.rms_norm(v, n, v, quant=True),
                lambda m: D.linear(m.codes, codes, x_scale=m.scale, w_scale=cs),
                lambda q: D.linear(q, w1, act="gelu"),
                lambda v: D.linear(v, w2, residual=v),
                lambda v: D.gated_ffn(v, w13, wd, residual=v),
                lambda v: D.rms_norm(v, n).y,
            ):
                v = step(v)
                if wait:
                    torch.cuda.synchronize()
                out.append(v.codes if isinstance(v, tuple) else v)
        return out

    want = [t.clone() for t in chain(True)]
    g = torch.cuda.CUDAGraph()
    buf.zero_()
    with torch.cuda.graph(g):
        got = chain(False)
    g.replay()
    buf.copy_(x)
    for _ in range(10):
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_two_host_threads(D):
    """Calls from two threads on streams of their own."""
    x, w, w13, w2, n = rand(300, 512), rand(264, 512, seed=1, scale=0.05), rand(528, 512, seed=2, scale=0.05), rand(512, 264, seed=3, scale=0.05), rand(512, seed=4)

    def calls(t):
        y, z = D.linear(x[:t], w, act="silu", save=True)
        return [y, D.gated_ffn(x[:t], w13, w2), D.rms_norm(x[:t], n, x[:t], quant=True).codes, *D.linear_backward(y, x[:t], w, z, "silu", bias=True)]

    want = {t: calls(t) for t in (1, 300)}
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(t):
        s = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = calls(t)
                s.synchronize()
                if not all(same(a, b) for a, b in zip(got, want[t])):
                    wrong.append(t)

    threads = [threading.Thread(target=work, args=(t,)) for t in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_fp16_range(D):
    """fp16's range, as documented: h above 65504 becomes infinite between the
    products, in its own row only; bf16 holds it."""
    for dt in (HF, BF):
        x, w13, w2 = torch.zeros(8, 8, dtype=dt, device="cuda"), torch.zeros(16, 8, dtype=dt, device="cuda"), torch.zeros(8, 8, dtype=dt, device="cuda")
        x[:, 0], w13[0, 0], w13[8, 0], w2[0, 0] = 1, 1, 1, 2.0**-10
        x[3, 0] = 1024  # h = 2^20, y = 2^10
        y = D.gated_ffn(x, w13, w2, "none")[:, 0].float().tolist()
        assert y == [2.0**-10] * 3 + [math.inf if dt == HF else 1024.0] + [2.0**-10] * 4
