"""The norms before and after a block, with gate, residual scale and gradients, against their
definition in 64 bits."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    return P


def randn(*shape, seed, std=1.0, mean=0.0, dtype=F):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def gate_of(kind, n, d, dtype, seed=7):
    shape = {"none": None, "channel": (d,), "token": (n, 1), "full": (n, d)}[kind]
    return None if shape is None else randn(*shape, seed=seed, dtype=dtype)


@pytest.mark.parametrize("n,d", [(1, 1), (1, 8), (3, 7), (5, 33), (2, 256), (9, 1001), (7, 2048), (4, 2056), (3, 4096),
                                 (2, 8192), (2, 8191), (700, 128)])
@pytest.mark.parametrize("xt,wt,ht", [(F, F, BF), (BF, F, F), (BF, BF, BF), (F, BF, F)])
def test_norm_in(P, n, d, xt, wt, ht):
    x, w = randn(n, d, seed=1, std=3.0, dtype=xt), randn(d, seed=2, std=0.3, mean=1.0, dtype=wt)
    for off in (0, 1):
        h = P.norm_in(x, w, eps=R.EPS, unit_offset=bool(off), out_dtype=ht)
        ref = R.norm_in(x, w, off)
        R.near(h, ref, ref.abs() * (R.NORM + R.HALF[ht]), "h")
        assert h.dtype == ht and torch.equal(h, P.norm_in(x, w, eps=R.EPS, unit_offset=bool(off), out_dtype=ht))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("act", ["linear", "sigmoid"])
@pytest.mark.parametrize("n,d,ot,rt", [(1, 2048, F, F), (8, 2048, BF, F), (5, 77, F, BF), (130, 1000, BF, BF), (3, 5000, F, F)])
def test_norm_out(P, gate, act, n, d, ot, rt):
    o, res = randn(n, d, seed=1, std=0.5, dtype=ot), randn(n, d, seed=2, std=2.0, dtype=rt)
    w, wn = randn(d, seed=3, std=0.3, mean=1.0), randn(d, seed=4, std=0.3, mean=1.0)
    for gt in (F, BF):
        g = gate_of(gate, n, d, gt)
        for post in (w, None):
            kw = dict(weight=post, eps=R.EPS, gate=g, gate_act=act, scale=0.7)
            out, h = P.norm_out(o, res, next_weight=wn, next_eps=R.EPS, next_dtype=BF, **kw)
            ref, term = R.norm_out(o, res, post, g, act, 0.7)
            R.near(out, ref, term * R.NORM + ref.abs() * (2.0 ** -23 + R.HALF[rt]), "res")
            href = R.norm_in(out, wn)
            R.near(h, href, href.abs() * (R.NORM + R.HALF[BF]), "h")
            # one pass or two: the same bits
            assert torch.equal(out, P.norm_out(o, res, **kw))
            assert torch.equal(h, P.norm_in(out, wn, eps=R.EPS, out_dtype=BF))


def test_norm_out_types_and_offset(P):
    n, d = 6, 512
    o, res = randn(n, d, seed=1, dtype=BF), randn(n, d, seed=2, dtype=F)
    w, wn = randn(d, seed=3, std=0.1, dtype=BF), randn(d, seed=4, std=0.1, dtype=BF)
    out, h = P.norm_out(o, res, weight=w, unit_offset=True, next_weight=wn, next_dtype=F, out_dtype=BF, scale=-2.0)
    ref, term = R.norm_out(o, res, w, None, "linear", -2.0, off=1.0)
    R.near(out, ref, term * R.NORM + ref.abs() * (2.0 ** -23 + R.HALF[BF]), "res")
    href = R.norm_in(out, wn, 1.0)
    R.near(h, href, href.abs() * R.NORM, "h")
    assert out.dtype == BF and h.dtype == F


@pytest.mark.parametrize("d", [1000, 1001])
def test_strided_rows_offsets_and_in_place(P, d):
    """Rows inside wider ones, starts off a 16-byte boundary, outputs over inputs, rows behind the last."""
    n = 5
    wide = randn(n + 2, d + 40, seed=1)
    for at in (0, 1, 8):
        o, res = wide[:n, at:at + d], randn(n + 2, d + 9, seed=2, dtype=BF)[:n, :d]
        w = randn(d, seed=3, mean=1.0)
        g = randn(n, d + 5, seed=4, dtype=BF)[:, 2:2 + d]
        kw = dict(weight=w, gate=g, gate_act="sigmoid", scale=0.5)
        # rows off a 16-byte boundary are summed in another order than vectors, so the root's last bit, and
        # with it a result's, may differ from that of contiguous rows: each is held to the definition
        got = P.norm_out(o, res, next_weight=w, **kw)
        ref, term = R.norm_out(o, res, w, g, "sigmoid", 0.5)
        R.near(got[0], ref, term * R.NORM + ref.abs() * (2.0 ** -23 + R.HALF[BF]), "res")
        href = R.norm_in(got[0], w)
        R.near(got[1], href, href.abs() * R.NORM, "h")
    buf = randn(n + 2, d, seed=5)
    keep = buf.clone()
    o = randn(n, d, seed=6)
    want = P.norm_out(o, buf[:n].clone(), weight=w, next_weight=w)
    o2 = o.clone()
    P.norm_out(o2, buf[:n], weight=w, next_weight=w, out=buf[:n], next_out=o2)
    assert torch.equal(buf[:n], want[0]) and torch.equal(o2, want[1]) and torch.equal(buf[n:], keep[n:])
    x = buf[:n].clone()
    want = P.norm_in(x, w)
    P.norm_in(x, w, out=x)
    assert torch.equal(x, want)


def test_zero_rows_and_values_that_are_not_finite(P):
    d = 300
    w = randn(d, seed=1, mean=1.0)
    x = randn(4, d, seed=2)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    h = P.norm_in(x, w, eps=R.EPS)
    assert (h[0] == 0).all() and torch.isnan(h[1]).all()
    assert torch.isnan(h[2, 7]) and (h[2, :7] == 0).all()  # inf / inf, finite / inf
    ref = R.norm_in(x[3:], w)
    R.near(h[3:], ref, ref.abs() * R.NORM, "a row beside them")
    # a gate at both ends of the sigmoid
    g = torch.tensor([[-float("inf")], [float("inf")], [-1e4], [1e4]], device="cuda")
    o, res = randn(4, d, seed=3), randn(4, d, seed=4)
    out = P.norm_out(o, res, gate=g, gate_act="sigmoid")
    assert torch.equal(out[0], res[0]) and torch.equal(out[2], res[2])
    assert torch.equal(out[1], res[1] + o[1]) and torch.equal(out[3], res[3] + o[3])


@pytest.mark.parametrize("n,d", [(1, 1), (1, 2048), (5, 77), (33, 1001), (400, 512), (700, 2048), (2, 8192), (3, 8191)])
@pytest.mark.parametrize("xt,dt", [(F, BF), (BF, F)])
def test_norm_in_backward(P, n, d, xt, dt):
    x, dh = randn(n, d, seed=1, std=2.0, dtype=xt), randn(n, d, seed=2, std=0.1, dtype=dt)
    dres = randn(n, d, seed=3, std=0.1, dtype=xt)
    for wt in (F, BF):
        for dr in (None, dres):
            w = randn(d, seed=4, std=0.3, mean=1.0, dtype=wt)
            dx, dw = P.norm_in_backward(x, w, dh, eps=R.EPS, d_residual=dr)
            rx, rw, sx, sw = R.norm_in_backward(x, w, dh, dr)
            R.near(dx, rx, sx * R.NORM + rx.abs() * R.HALF[xt], "dx")
            R.near(dw, rw, sw * 2 * R.NORM + rw.abs() * R.HALF[wt], "dw")
            again = P.norm_in_backward(x, w, dh, eps=R.EPS, d_residual=dr)
            assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("act", ["linear", "sigmoid"])
@pytest.mark.parametrize("n,d,ot,rt", [(1, 8, F, F), (5, 77, BF, F), (600, 1000, F, BF), (3, 4096, BF, BF), (2, 8191, F, F)])
def test_norm_out_backward(P, gate, act, n, d, ot, rt):
    o, dres = randn(n, d, seed=1, std=0.5, dtype=ot), randn(n, d, seed=2, std=0.1, dtype=rt)
    w = randn(d, seed=3, std=0.3, mean=1.0)
    for gt in (F, BF):
        g = gate_of(gate, n, d, gt)
        for post in (w, None):
            got = P.norm_out_backward(o, dres, weight=post, eps=R.EPS, gate=g, gate_act=act, scale=0.7)
            ref = R.norm_out_backward(o, dres, post, g, act, 0.7)
            assert (got[1] is None) == (post is None) and (got[2] is None) == (g is None)
            for v, name, t in zip(got, ("d_o", "d_w", "d_gate"), (ot, F, gt)):
                if v is not None:
                    r, size = ref[name]
                    assert v.dtype == t
                    R.near(v, r, size * 2 * R.NORM + r.abs() * R.HALF[t], name)


@pytest.mark.parametrize("n,d,ot,rt,gate", [(592, 8, F, F, "full"), (2000, 264, BF, F, "token"), (5000, 1000, F, BF, "full"),
                                            (1500, 2048, F, F, "channel"), (2500, 4096, BF, BF, "full"), (600, 8192, F, F, "none"),
                                            (600, 8192, F, F, "full"), (8192, 32, BF, BF, "channel"), (700, 5000, BF, F, "full")])
def test_many_rows(P, n, d, ot, rt, gate):
    """The sizes at which blocks walk over rows, strided and not."""
    wide = randn(n, d + 8, seed=1, std=0.5, dtype=ot)
    res, dres, dh = randn(n, d, seed=2, std=2.0, dtype=rt), randn(n, d, seed=5, std=0.1, dtype=rt), randn(n, d, seed=6, std=0.1, dtype=BF)
    w, wn, g = randn(d, seed=3, std=0.3, mean=1.0), randn(d, seed=4, std=0.3, mean=1.0), gate_of(gate, n, d, BF)
    kw = dict(weight=w, eps=R.EPS, gate=g, gate_act="sigmoid", scale=0.7)
    for o in (wide[:, 8:], wide[:, 8:].contiguous()):
        out, h = P.norm_out(o, res, next_weight=wn, next_eps=R.EPS, next_dtype=BF, **kw)
        ref, term = R.norm_out(o, res, w, g, "sigmoid", 0.7)
        R.near(out, ref, term * R.NORM + ref.abs() * (2.0 ** -23 + R.HALF[rt]), "res")
        href = R.norm_in(out, wn)
        R.near(h, href, href.abs() * (R.NORM + R.HALF[BF]), "h")
        assert torch.equal(h, P.norm_in(out, wn, eps=R.EPS, out_dtype=BF))
        dx, dwn = P.norm_in_backward(out, wn, dh, eps=R.EPS, d_residual=dres)
        rx, rw, sx, sw = R.norm_in_backward(out, wn, dh, dres)
        R.near(dx, rx, sx * R.NORM + rx.abs() * R.HALF[rt], "dx")
        R.near(dwn, rw, sw * 2 * R.NORM + rw.abs() * R.HALF[F], "dwn")
        got = P.norm_out_backward(o, dres, **kw)
        want = R.norm_out_backward(o, dres, w, g, "sigmoid", 0.7)
        for v, name, t in zip(got, ("d_o", "d_w", "d_gate"), (ot, F, BF)):
            if v is not None:
                r, size = want[name]
                R.near(v, r, size * 2 * R.NORM + r.abs() * R.HALF[t], name)
        again = P.norm_out_backward(o, dres, **kw)
        assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    few = P.norm_out(wide[:9, 8:], res[:9], next_weight=wn, next_eps=R.EPS, next_dtype=BF,
                     **{**kw, "gate": g[:9] if gate in ("token", "full") else g})
    assert torch.equal(few[0], out[:9]) and torch.equal(few[1], h[:9])  # a row does not depend on their number
    assert P.block_check() == P.MOE_OK


def test_gradients_against_differences(P):
    """Of the kernels' own forward: sum(dres * res_out) + sum(dh * h) along a direction.  The values are
    of order 1, n d = 4096 of them: an fp32 result is 2^-23 off, so the difference over 2 e is off by
    about 2^-23 sqrt(4096) / (2 e) = 4e-4 for e = 2^-7, and by e^2 / 6 times a third derivative (of order
    the sum's size, sqrt(4096)) = 1e-3 sqrt(4096) / 6 = 7e-4; 4e-3 leaves room for their constants."""
    n, d, e = 4, 1024, 2.0 ** -7
    o, res, w, wn = (randn(*s, seed=i) for i, s in enumerate([(n, d), (n, d), (d,), (d,)]))
    g = randn(n, 1, seed=9)
    dres, dh = randn(n, d, seed=10), randn(n, d, seed=11)
    kw = dict(eps=R.EPS, gate_act="sigmoid", scale=0.8)

    def loss(o, w, g, wn):
        out, h = P.norm_out(o, res, weight=w, gate=g, next_weight=wn, next_eps=R.EPS, next_dtype=F, **kw)
        return ((out.double() * dres.double()).sum() + (h.double() * dh.double()).sum()).item()

    out = P.norm_out(o, res, weight=w, gate=g, **kw)
    dr, dwn = P.norm_in_backward(out, wn, dh, eps=R.EPS, d_residual=dres)
    do, dw, dg = P.norm_out_backward(o, dr, weight=w, gate=g, **kw)
    for i, (grad, val) in enumerate(((do, o), (dw, w), (dg, g), (dwn, wn))):
        v = randn(*val.shape, seed=20 + i)
        v = v / v.norm()
        at = [o, w, g, wn]
        at[i] = val + e * v
        up = loss(*at)
        at[i] = val - e * v
        diff = (up - loss(*at)) / (2 * e)
        want = (grad.double() * v.double()).sum().item()
        assert abs(diff - want) <= 4e-3 * max(1.0, abs(want)), (i, diff, want)


def test_graph_and_stream(P):
    """Captured and replayed on new inputs, on a stream of its own: the eager bits."""
    n, d = 37, 1000
    o, res, w = randn(n, d, seed=1), randn(n, d, seed=2), randn(d, seed=3, mean=1.0)
    dres = randn(n, d, seed=4)
    g = randn(d, seed=5, dtype=BF)

    def step():
        out, h = P.norm_out(o, res, weight=w, gate=g, next_weight=w)
        dr, dwn = P.norm_in_backward(out, w, h, d_residual=dres)
        return (out, h, dr, dwn, *P.norm_out_backward(o, dr, weight=w, gate=g))

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            held = step()
    torch.cuda.current_stream().wait_stream(s)
    for k in range(2):
        o.copy_(randn(n, d, seed=30 + k))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("n,d", [(5, 77), (9, 1000), (1, 8), (2000, 264), (2500, 4096), (700, 5000)])
def test_gradient_of_a_saturated_gate(P, gate, n, d):
    """Gates from -40 to 40: the slope sigmoid(g) sigmoid(-g) down to 4e-18, to the same relative error as others.
    (An exponential of z = 40 from the rounded product z log2 e, below 64: half a step, 2^-19, and the constant's
    own 2^-25 of 58, together 2^-18.2, times log 2: 2^-18.7, inside R.NORM for a single factor.)"""
    o, dres = randn(n, d, seed=1, std=0.5), randn(n, d, seed=2, std=0.1)
    w, g = randn(d, seed=3, std=0.3, mean=1.0), gate_of(gate, n, d, F)
    values = torch.tensor([-40.0, -20.0, -10.0, -1.0, 0.0, 1.0, 10.0, 16.0, 17.0, 20.0, 40.0], device="cuda")
    flat = g.view(-1)
    flat.copy_(values[torch.arange(flat.numel(), device="cuda") % len(values)])
    for post in (w, None):
        got = P.norm_out_backward(o, dres, weight=post, eps=R.EPS, gate=g, gate_act="sigmoid", scale=0.7)
        ref = R.norm_out_backward(o, dres, post, g, "sigmoid", 0.7)
        # the reference's 1 - a in 64 bits has 2^-53 of 1 against a slope of 4e-18: taken as sigmoid(-g)
        s = torch.sigmoid(g.double())
        dz = 0.7 * dres.double()
        u = R.post(o, post)
        t = dz * u * (s * torch.sigmoid(-g.double()))
        size = t.abs()
        if gate == "channel":
            t, size = t.sum(0), size.sum(0)
        elif gate == "token":
            t, size = t.sum(1, keepdim=True), size.sum(1, keepdim=True)
        R.near(got[2], t, size * 2 * R.NORM + t.abs() * R.HALF[F], "d_gate")
        for v, name in zip(got[:2], ("d_o", "d_w")):
            if v is not None:
                r, size = ref[name]
                R.near(v, r, size * 2 * R.NORM + r.abs() * R.HALF[F], name)


def test_gates_at_the_ends(P):
    """Gates of +-infinity: weight 1 or 0, slope 0; NaN stays in its own place."""
    o, dres = randn(6, 64, seed=1), randn(6, 64, seed=2)
    g = torch.zeros(6, 64, device="cuda")
    g[0], g[1], g[2], g[3], g[4, 5] = float("inf"), -float("inf"), 200.0, -200.0, float("nan")
    do, _, dg = P.norm_out_backward(o, dres, gate=g, gate_act="sigmoid")
    assert torch.equal(do[0], dres[0]) and torch.equal(do[2], dres[2]) and (do[1] == 0).all() and (do[3] == 0).all()
    assert (dg[:4] == 0).all()
    assert torch.isnan(do[4, 5]) and torch.isnan(dg[4, 5]) and torch.isnan(do).sum() == 1 and torch.isnan(dg).sum() == 1


@pytest.mark.parametrize("kind", ["channel", "full"])
def test_sigmoid_of_gates_by_the_value(P, kind):
    """o = 1 and a residual of 0 leave the gate's sigmoid alone.  Its exponential has the argument z log2 e rounded
    (2^-24 of it) with a constant that is 2^-26 off, so an error of 1.25 |z| 2^-24, and is itself good to 2^-22; a
    reciprocal good to 2^-23 and the rounding of 1 + e follow: (1.25 |z| + 7) 2^-24."""
    n, d = (1, 4096) if kind == "channel" else (16, 4096)
    g = torch.rand(n, d, generator=torch.Generator().manual_seed(1), dtype=torch.float64).mul(100).sub(80).float().cuda()
    one, zero = torch.ones(n, d, device="cuda"), torch.zeros(n, d, device="cuda")
    gate = g.reshape(-1) if kind == "channel" else g
    ref = torch.sigmoid(g.double())
    tol = ref * (1.25 * g.double().abs() + 7) * 2.0 ** -24
    R.near(P.norm_out(one, zero, gate=gate, gate_act="sigmoid"), ref, tol, "forward")
    # the gradient's factor: the same, or 1 minus the other one (half a step more)
    R.near(P.norm_out_backward(one, one, gate=gate, gate_act="sigmoid")[0], ref, tol + ref * 2.0 ** -24, "backward")


def test_parameters_under_no_grad(P):
    x, w, g = randn(3, 64, seed=1), randn(64, seed=2), randn(3, 64, seed=3)
    want = P.norm_out(x, x, weight=w, gate=g)
    p, q, r = (torch.nn.Parameter(t.clone()) for t in (x, w, g))
    for bad in ((p, x, w, g), (x, p, w, g), (x, x, q, g), (x, x, w, r)):
        with pytest.raises(ValueError, match="requires grad"):
            P.norm_out(bad[0], bad[1], weight=bad[2], gate=bad[3])
    with torch.no_grad():
        got = P.norm_out(p, p, weight=q, gate=r)
    assert torch.equal(got, want) and not got.requires_grad


@pytest.mark.parametrize("n,d", [(5, 64), (3, 77), (2000, 264)])
def test_column_ranges_of_one_matrix(P, n, d):
    """Inputs and outputs between each other's rows share no memory; one column more and they do."""
    o, w = randn(n, d, seed=1), randn(d, seed=3, mean=1.0)
    both = randn(n, 3 * d + 2, seed=2)
    keep = both.clone()
    res, new, h = both[:, :d], both[:, d:2 * d], both[:, 2 * d + 1:3 * d + 1]
    # (rows off a 16-byte boundary are summed in another order than vectors: each is held to the definition)
    ref, term = R.norm_out(o, res, w, None, "linear", 1.0)
    P.norm_out(o, res, weight=w, next_weight=w, out=new, next_out=h)
    R.near(new, ref, term * R.NORM + ref.abs() * (2.0 ** -23 + R.HALF[F]), "res")
    ref = R.norm_in(new, w)
    R.near(h, ref, ref.abs() * (R.NORM + R.HALF[F]), "h")
    P.norm_in(new, w, out=res)
    R.near(res, ref, ref.abs() * (R.NORM + R.HALF[F]), "h")
    assert torch.equal(both[:, 2 * d], keep[:, 2 * d]) and torch.equal(both[:, 3 * d + 1], keep[:, 3 * d + 1])
    for out in (both[:, 1:d + 1], both[:, d - 1:2 * d - 1], both[:, :d]):
        with pytest.raises(ValueError, match="overlaps"):
            P.norm_out(o, both[:, :d], out=both[:, d:2 * d], next_weight=w, next_out=out)
    with pytest.raises(ValueError, match="overlaps"):
        P.norm_in(both[1:, :d], w, out=both[:-1, d - 1:2 * d - 1])
    P.norm_in(both[1:, :d], w, out=both[:-1, d:2 * d])  # of other rows
