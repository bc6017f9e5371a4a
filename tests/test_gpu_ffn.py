"""The dense gated feed-forward block and its gradients against their definition in 64 bits."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    yield P
    assert P.block_check() == P.MOE_OK  # no wait ran out


def randn(*shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def weights(d, f, seed=1):
    return (randn(f, d, seed=seed, std=d ** -0.5), randn(f, d, seed=seed + 1, std=d ** -0.5),
            randn(d, f, seed=seed + 2, std=f ** -0.5))


def check_y(y, r, wd, add=None):
    ref = r["y"] if add is None else r["y"] + add.double()
    extra = 0.0 if add is None else add.double().abs() * 2.0 ** -23
    R.near(y, ref, R.product_tolerance(ref, [(r["h"], wd.double().T)], y.dtype, extra), "y")


TOKENS = [1, 2, 7, 8, 9, 16, 17, 32, 33, 100, 128, 129, 300]


@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("d,f", [(8, 8), (64, 128), (256, 1000), (1000, 264), (2048, 768)])
def test_forward(P, n, d, f):
    w = weights(d, f)
    x = randn(n, d, seed=5)
    r = R.ffn(x, *w)
    y = P.ffn_forward(x, *w)
    check_y(y, r, w[2])
    assert torch.equal(y, P.ffn_forward(x, *w))
    y2, saved = P.ffn_forward(x, *w, save=True)
    assert torch.equal(y, y2)
    for s, k, wt in zip(saved, ("g", "u"), w):
        mag = x.double().abs() @ wt.double().abs().T
        R.near(s, r[k], mag * 2.0 ** -13 + 1e-30, k)
    add = randn(n, d, seed=6, dtype=F)
    out = add.clone()
    assert P.ffn_forward(x, *w, add=out, out=out) is out
    check_y(out, r, w[2], add)
    check_y(P.ffn_forward(x, *w, add=add.to(BF)), r, w[2], add.to(BF))


def check_gradients(got, x, w, dy, r):
    bf = torch.bfloat16
    want = {
        "dx": [(r["dg"], w[0].double()), (r["du"], w[1].double())],
        "dwg": [(r["dg"].T, x.double())], "dwu": [(r["du"].T, x.double())],
        "dwd": [(r["h"].T, dy.double())],
    }
    for v, name in zip(got, ("dx", "dwg", "dwu", "dwd")):
        if v is not None:
            ref = r[name].T if name == "dwd" else r[name]
            tol = R.product_tolerance(ref, want[name], bf)
            R.near(v.T if name == "dwd" else v, ref, tol, name)


@pytest.mark.parametrize("n", [1, 8, 33, 64, 65, 128, 300, 1180])
@pytest.mark.parametrize("d,f", [(8, 8), (64, 128), (256, 1000), (1000, 264), (2048, 768)])
def test_backward(P, n, d, f):
    w = weights(d, f)
    x, dy = randn(n, d, seed=5), randn(n, d, seed=6, std=0.1)
    _, saved = P.ffn_forward(x, *w, save=True)
    got = P.ffn_backward(dy, x, *w, saved)
    check_gradients(got, x, w, dy, R.ffn(x, *w, dy))
    again = P.ffn_backward(dy, x, *w, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    part = P.ffn_backward(dy, x, *w, saved, need_dw=False)
    assert torch.equal(part[0], got[0]) and part[1:] == (None, None, None)
    part = P.ffn_backward(dy, x, *w, saved, need_dx=False)
    assert part[0] is None and all(torch.equal(a, b) for a, b in zip(part[1:], got[1:]))


@pytest.mark.parametrize("n", [3, 8, 12, 40, 130, 300])
@pytest.mark.parametrize("d,f", [(512, 8192), (200, 4104)])
def test_long_products_of_few_tokens(P, n, d, f):
    """The down product and dx run over many more values than they have results."""
    w = weights(d, f)
    x, dy = randn(n, d, seed=5), randn(n, d, seed=6, std=0.1)
    r = R.ffn(x, *w, dy)
    add = randn(n, d, seed=7, dtype=F)
    for kw in ({}, {"add": add, "out_dtype": F}, {"add": add.to(BF)}):
        y = P.ffn_forward(x, *w, **kw)
        check_y(y, r, w[2], kw.get("add"))
        assert torch.equal(y, P.ffn_forward(x, *w, **kw))
    _, saved = P.ffn_forward(x, *w, save=True)
    got = P.ffn_backward(dy, x, *w, saved)
    check_gradients(got, x, w, dy, r)
    assert torch.equal(P.ffn_backward(dy, x, *w, saved, need_dw=False)[0], got[0])
    assert torch.equal(P.ffn_backward(dy, x, *w, saved, need_dx=False)[3], got[3])


@pytest.mark.parametrize("n", [9, 127, 129, 500])
@pytest.mark.parametrize("d,f", [(4096, 776), (2056, 40), (72, 8192)])
def test_narrow_blocks_and_models(P, n, d, f):
    """Products with few tiles and long rows, in each of the three epilogues; rows behind the last stay."""
    w = weights(d, f)
    x, dy = randn(n, d, seed=5), randn(n, d, seed=6, std=0.1)
    r = R.ffn(x, *w, dy)
    rows = torch.full((n + 2, d), 7.0, device="cuda")
    rows[:n] = randn(n, d, seed=7, dtype=F)
    add = rows[:n].clone()
    y, saved = P.ffn_forward(x, *w, add=rows[:n], out=rows[:n], save=True)
    check_y(y, r, w[2], add)
    assert (rows[n:] == 7.0).all()
    for v, k, wt in zip(saved, ("g", "u"), w):
        R.near(v, r[k], x.double().abs() @ wt.double().abs().T * 2.0 ** -13 + 1e-30, k)
    got = P.ffn_backward(dy, x, *w, saved)
    check_gradients(got, x, w, dy, r)
    assert all(torch.equal(a, b) for a, b in zip(got, P.ffn_backward(dy, x, *w, saved)))
    assert torch.equal(P.ffn_backward(dy, x, *w, saved, need_dw=False)[0], got[0])


def test_two_streams_at_once(P):
    """Calls of several shapes and forms beside one another: the bits of each alone."""
    shapes = [(64, 1024, 512), (200, 512, 1024), (5, 1024, 1024), (700, 256, 768)]
    data = [(randn(n, d, seed=i), randn(n, d, seed=i + 9, std=0.1), weights(d, f, seed=20 * i)) for i, (n, d, f) in enumerate(shapes)]

    def step(x, dy, w):
        y, saved = P.ffn_forward(x, *w, save=True)
        return (y, *P.ffn_backward(dy, x, *w, saved))

    want = [step(*v) for v in data]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, v in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(step(*v))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, h in zip(got, want) for a, b in zip(g, h))


def test_large(P):
    n, d, f = 2500, 2048, 2304
    w = weights(d, f)
    x, dy = randn(n, d, seed=5), randn(n, d, seed=6, std=0.1)
    y, saved = P.ffn_forward(x, *w, save=True)
    r = R.ffn(x, *w, dy)
    check_y(y, r, w[2])
    check_gradients(P.ffn_backward(dy, x, *w, saved), x, w, dy, r)


@pytest.mark.parametrize("n", [5, 200])
def test_strided_rows_and_rows_behind_the_last(P, n):
    d, f = 128, 200
    w = weights(d, f)
    wide = randn(n + 3, d + 64, seed=5)
    x = wide[:n, 8:8 + d]
    y = P.ffn_forward(x.contiguous(), *w)
    buf = torch.full((n + 3, d + 16), 7.0, dtype=BF, device="cuda")
    out = P.ffn_forward(x, *w, out=buf[:n, 8:8 + d])
    assert torch.equal(out, y) and (buf[n:] == 7).all() and (buf[:, :8] == 7).all() and (buf[:, 8 + d:] == 7).all()
    _, saved = P.ffn_forward(x, *w, save=True)
    dy = randn(n, d + 8, seed=6)[:, :d]
    a, b = P.ffn_backward(dy, x, *w, saved), P.ffn_backward(dy.contiguous(), x.contiguous(), *w, saved)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("n", [6, 140])
def test_values_that_are_not_finite_stay_in_their_row(P, n):
    d, f = 64, 72
    w = weights(d, f)
    x = randn(n, d, seed=5)
    y = P.ffn_forward(x, *w)
    x[2, 3] = float("nan")
    z = P.ffn_forward(x, *w)
    keep = torch.arange(n, device="cuda") != 2
    assert torch.isnan(z[2]).all() and torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("n", [6, 140])
def test_graph_and_stream(P, n):
    """Captured and replayed on new inputs, beside eager calls on the same weights: the same bits."""
    d, f = 256, 320
    w = weights(d, f)
    x, dy = randn(n, d, seed=5), randn(n, d, seed=6)

    def step():
        y, saved = P.ffn_forward(x, *w, save=True)
        return (y, *P.ffn_backward(dy, x, *w, saved))

    step()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for k in range(2):
        x.copy_(randn(n, d, seed=50 + k))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_gradients_against_differences(P):
    """Of the kernels' own forward: sum(dy * y) along random signs, on values that bf16 holds at both ends
    of the step e.  x and dy are +-1, the weights +-2^-3, so g, u, h are of order 1 and so is the sum over
    d of dy wd: the rounding of h (standard deviation 2^-9 of it), over n f = 512 values, leaves about
    2^-9 sqrt(512) in each of the two losses and sqrt(2) of that over 2 e in the difference; four standard
    deviations are allowed.  A step moves g and u by about 2^-3: the third-order part is some
    (2^-3)^2 / 6 times factors of order 1 of the derivative; 1/32 of the gradient's 2-norm is allowed."""
    n, d, f = 8, 64, 64

    def signs(*s, seed):
        return randn(*s, seed=seed, dtype=F).sign()

    at = [signs(n, d, seed=7)] + [signs(*s, seed=i) * 0.125 for i, s in enumerate([(f, d), (f, d), (d, f)])]
    dy = signs(n, d, seed=8).to(BF)

    def loss(v):
        return (P.ffn_forward(*[t.to(BF) for t in v], out_dtype=F).double() * dy.double()).sum().item()

    b = [t.to(BF) for t in at]
    _, saved = P.ffn_forward(*b, save=True)
    for i, grad in enumerate(P.ffn_backward(dy, *b, saved)):
        step = 2.0 ** -4 if i == 0 else 2.0 ** -6
        v = signs(*at[i].shape, seed=30 + i)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * v, at[i] - step * v
        diff = (loss(up) - loss(down)) / (2 * step)
        want = (grad.double() * v.double()).sum().item()
        norm = grad.double().norm().item()
        noise = 4 * 2 ** 0.5 * 2.0 ** -9 * (n * f) ** 0.5 / (2 * step)
        assert norm > 4 * noise and abs(diff - want) <= noise + norm / 32, (i, diff, want, norm, noise)
