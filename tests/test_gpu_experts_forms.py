"""Forms of the operators of resident experts and of 4-bit products at real
sizes, on the GPU against their 64-bit forms (tests/experts_ref.py)."""

import pytest

torch = pytest.importorskip("torch")

import dense_ref as R  # noqa: E402
import experts_ref as X  # noqa: E402
from test_gpu_experts import ACTS, BF, F32, FMTS, HF, D, _block, _calls, ints, offsets_of, pitched, rand, same, weights  # noqa: E402, F401
from w4_forms import FORMS  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,k,n", FORMS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear_w4_forms(D, rows, k, n, fmt, dt):  # noqa: F811
    c, s, ts = weights(fmt, n, k)
    x, b, res = rand(rows, k, dt=dt), rand(n, seed=2, dt=dt), rand(rows, n, seed=3, dt=dt)
    w = X.values(c, s, fmt, ts)
    rounded = rows > 128 and fmt == "int4"  # weights
    y = D.linear_w4(x, c, s, fmt, tensor_scale=ts)
    R.check(y, X.linear_w4(x, w, None, "none", None, dt, dt, rounded), "y")
    act = ACTS[(rows + k + n) % 5]
    f = D.linear_w4(x, c, s, fmt, b, act, res, tensor_scale=ts, out_dtype=F32)
    R.check(f, X.linear_w4(x, w, b, act, res, dt, F32, rounded), "with everything")
    wide = pitched(res, 8) if n % 8 == 0 else res  # a residual of ragged rows is contiguous
    assert same(D.linear_w4(pitched(x, 8), c, s, fmt, b, act, wide, tensor_scale=ts, out_dtype=F32), f)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear_w4_captured(D, fmt, dt):  # noqa: F811
    """Every class of rows in two graphs that are replayed in turn."""
    k, n = 416, 264
    c, s, ts = weights(fmt, n, k)
    x = rand(200, k, dt=dt)

    def run():
        return [D.linear_w4(x[:r], c, s, fmt, tensor_scale=ts) for r in (1, 16, 40, 128, 200)]

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
    assert all(same(a, b) for _, got in graphs for a, b in zip(ref, got))


def ragged(rows, groups, seed=0):
    cut = torch.sort(ints(0, rows + 1, (groups - 1,), seed=seed, dt=torch.int32)).values.tolist()
    return [b - a for a, b in zip([0] + cut, cut + [rows])]


@pytest.mark.parametrize("rows,g,k,n,dt", [(2042, 8, 2880, 1440, HF), (2042, 8, 2880, 1440, BF), (32, 128, 2048, 1536, BF), (5000, 3, 4096, 328, BF)])
def test_grouped_linear_of_a_models_size(D, rows, g, k, n, dt):  # noqa: F811
    x, w, dy = rand(rows, k, dt=dt), rand(g, n, k, seed=1, scale=k**-0.5, dt=dt), rand(rows, n, seed=2, dt=dt)
    off = offsets_of(ragged(rows, g))
    R.check(D.grouped_linear(x, w, off), X.grouped_linear(x, w, off, dt), "y")
    dx, dw = D.grouped_linear_backward(dy, x, w, off)
    want = X.grouped_linear_backward(dy, x, w, off, dt)
    R.check(dx, want["dx"], "dx")
    R.check(dw, want["dw"], "dw")


@pytest.mark.parametrize("rows,g,h,i,act", [(2048, 128, 2048, 768, "silu"), (600, 8, 2880, 1440, "gelu_tanh")])
def test_grouped_ffn_of_a_models_size(D, rows, g, h, i, act):  # noqa: F811
    x, w13, w2 = rand(rows, h), rand(g, 2 * i, h, seed=1, scale=h**-0.5), rand(g, h, i, seed=2, scale=i**-0.5)
    off = offsets_of(ragged(rows, g))
    y, gu = D.grouped_ffn(x, w13, w2, off, act, save=True)
    want = X.grouped_ffn(x, w13, w2, off, act, BF)
    R.check(gu, want["gu"], "gu")
    R.check(y, want["y"], "y")
    del want
    dy = rand(rows, h, seed=3)
    got = D.grouped_ffn_backward(dy, x, w13, w2, gu, off, act)
    want = X.grouped_ffn_backward(dy, x, w13, w2, gu, off, act, BF)
    for v, name in zip(got, ("dx", "dw13", "dw2")):
        R.check(v, want[name], name)


def test_expert_block_of_no_tokens(D):  # noqa: F811
    b = _block()
    out, saved = b.forward(rand(1, 128)[:0])
    assert out.shape == (0, 128)
    dx, g = b.backward(out, saved)
    assert dx.shape == (0, 128) and all((v == 0).all() for v in g.values())


def test_calls_of_two_host_threads_all_finish(D):  # noqa: F811
    """What a call raises in a thread reaches the test."""
    from concurrent.futures import ThreadPoolExecutor

    run = _calls(D)
    ref = run()
    torch.cuda.synchronize()

    def work(_):
        done, st = 0, torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(10):
                got = run()
                st.synchronize()
                assert all(same(a, b) for a, b in zip(ref, got))
                done += 1
        return done

    with ThreadPoolExecutor(2) as pool:
        assert list(pool.map(work, range(2))) == [10, 10]
