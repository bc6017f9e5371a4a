"""The block operators' definitions in 64 bits (torch tensors in, float64 tensors out), and how far a
kernel's result may be from them.

Tolerances count roundings.  HALF[t] is half a step of type t relative to a value.  In fp32 a norm's
sum of d <= 8192 squares passes at most 32 additions in a thread, 5 shuffles and 8 warps, so
q = rsqrt(.) is good to (47 / 2 + 4) 2^-24; a sigmoid by a hardware exponential to about 2^-20 for the
gates used here; with the few products around them a term is good to NORM = 2^-18 of its magnitude.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
NORM = 2.0 ** -18
EPS = 1e-6


def f64(t):
    return None if t is None else t.detach().double()


def act(g, kind):
    return torch.sigmoid(g) if kind == "sigmoid" else g


def rms_root(x, eps=EPS):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def norm_in(x, w, off=0.0, eps=EPS):
    x = f64(x)
    return x * rms_root(x, eps) * (f64(w) + off)


def post(o, w, off=0.0, eps=EPS):
    o = f64(o)
    return o if w is None else o * rms_root(o, eps) * (f64(w) + off)


def norm_out(o, res, w, gate, gate_act, scale, off=0.0, eps=EPS):
    """(result, magnitude of the gated term)"""
    u = post(o, w, off, eps)
    a = 1.0 if gate is None else act(f64(gate), gate_act)
    t = scale * a * u
    return f64(res) + t, t.abs()


def _rms_gradient(x, t, q):
    """Gradient of x rsqrt(mean x^2 + eps) and the magnitude of its parts."""
    m = (t * x).mean(-1, keepdim=True)
    size = q * (t.abs() + x.abs() * q * q * (t * x).abs().mean(-1, keepdim=True))
    return q * (t - x * q * q * m), size


def norm_in_backward(x, w, dh, dres=None, off=0.0, eps=EPS):
    """dx, dw and the magnitudes of what they are sums of"""
    x, w, dh = f64(x), f64(w) + off, f64(dh)
    q = rms_root(x, eps)
    dx, size = _rms_gradient(x, dh * w, q)
    terms = dh * x * q
    if dres is not None:
        dx, size = dx + f64(dres), size + f64(dres).abs()
    return dx, terms.sum(0), size, terms.abs().sum(0)


def norm_out_backward(o, dres, w, gate, gate_act, scale, off=0.0, eps=EPS):
    """{name: (gradient, magnitude)} of d_o, d_w (if w), d_gate (if gate)"""
    o, dz = f64(o), scale * f64(dres)
    g = None if gate is None else f64(gate)
    a = torch.ones_like(o) if g is None else act(g, gate_act).expand_as(o) + 0 * o
    q = rms_root(o, eps) if w is not None else torch.ones_like(o[:, :1])
    ww = torch.ones_like(o[0]) if w is None else f64(w) + off
    out = {}
    if w is not None:
        out["d_o"] = _rms_gradient(o, dz * a * ww, q)
        terms = dz * a * o * q
        out["d_w"] = terms.sum(0), terms.abs().sum(0)
    else:
        out["d_o"] = dz * a, (dz * a).abs()
    if g is not None:
        slope = a * (1 - a) if gate_act == "sigmoid" else torch.ones_like(a)
        t = dz * o * q * ww * slope
        s = t.abs()
        if g.dim() == 1:
            t, s = t.sum(0), s.sum(0)
        elif g.shape[1] == 1 and o.shape[1] != 1:
            t, s = t.sum(1, keepdim=True), s.sum(1, keepdim=True)
        out["d_gate"] = t, s
    return out


def near(got, ref, tol, what):
    """Every value within its tolerance; the same infinities and NaN."""
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), f"{what}: not the same finite values"
    bad = ((got - ref).abs() > tol) & fin
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{got[tuple(i)].item():.8g}, expected {ref[tuple(i)].item():.8g} "
                             f"within {tol[tuple(i)].item():.3g}")


def adapters(x, base, ids, a, b, scales):
    """(out, magnitude of the products' sums): a, b, scales by slot (None: empty)"""
    y, size = f64(base).clone(), torch.zeros(base.shape, dtype=torch.float64, device=base.device)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < len(a) and a[i] is not None:
            xa, aa, bb = f64(x[t]), f64(a[i]).to(y.device), f64(b[i]).to(y.device)
            y[t] += scales[i] * (bb @ (aa @ xa))
            size[t] = abs(scales[i]) * (bb.abs() @ (aa.abs() @ xa.abs()))
    return y, size


def adapters_tolerance(ref, size, base, d_in, rank, out_dtype):
    # fp32 sums of d_in and of `rank` products (one step lost per addition at most), bf16 out: v and an
    # fp32 x in two parts, 2^-16 each; then the add and the rounding
    t = size * (d_in + rank + 16) * 2.0 ** -23
    if out_dtype == torch.bfloat16:
        t = t + size * 2.0 ** -15
    return t + (ref.abs() + base.double().abs()) * 2.0 ** -23 + ref.abs() * HALF[out_dtype] + 1e-30


def ffn(x, wg, wu, wd, dy=None):
    """g, u, h, y and, from dy, the gradients, all in 64 bits"""
    x, wg, wu, wd = f64(x), f64(wg), f64(wu), f64(wd)
    g, u = x @ wg.T, x @ wu.T
    s = torch.sigmoid(g)
    r = {"g": g, "u": u, "h": g * s * u}
    r["y"] = r["h"] @ wd.T
    if dy is not None:
        dy = f64(dy)
        dh = dy @ wd
        r["dg"], r["du"] = dh * u * s * (1 + g * (1 - s)), dh * g * s
        r["dx"] = r["dg"] @ wg + r["du"] @ wu
        r["dwg"], r["dwu"], r["dwd"] = r["dg"].T @ x, r["du"].T @ x, dy.T @ r["h"]
    return r


def product_tolerance(ref, pairs, out_dtype, extra=0.0):
    """Of sums of products a b whose first factors were rounded to bf16: `pairs` of (a, b) with result
    a @ b.  The roundings of a are independent, each at most 2^-8 of its value (uniform: standard
    deviation 2^-8 / sqrt 3 at most); eight standard deviations of their sum.  a itself was computed in
    fp32 from sums of up to 8192 products and a sigmoid: 2^-14 of it, and as much for the sums here,
    relative to the sum of magnitudes."""
    var = sum((a * a) @ (b * b) for a, b in pairs)
    mag = sum(a.abs() @ b.abs() for a, b in pairs)
    return 8 * 2.0 ** -8 / 3 ** 0.5 * var.sqrt() + mag * 2.0 ** -13 + ref.abs() * HALF[out_dtype] + extra + 1e-30
