"""What the block operators are measured on: the norms around a block, the low-rank adapters of many
requests beside it, and the dense gated feed-forward block with its gradients.

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once at the
end) or, where `own` is true, by the calls a user of this package makes.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
_BYTES = {BF16: 2, F32: 4}
EPS = 1e-6
SCALE = 0.7  # residual scale of the norm cases


# ------------------------------------------------------------------------------------------ cases
def _norm(n, d, o, res, gate, nxt, back, name=None):
    """gate: "none", "channel", "token" or "full"; nxt: the next block's input norm in the same pass;
    back: forward and gradients."""
    c = {"op": "norm", "n": n, "d": d, "o": o, "res": res, "gate": gate, "next": nxt, "back": back}
    return dict(c, name=name) if name else c


def _adapters(n, d_in, d_out, slots, rank, mixed, x, out, runs, name=None):
    """mixed: ranks from 1 to `rank` and some tokens without an adapter, else `rank` throughout;
    runs: a request's tokens stand together (prompts), else in any order (one token a request)."""
    c = {"op": "adapters", "n": n, "d_in": d_in, "d_out": d_out, "slots": slots, "rank": rank, "mixed": mixed,
         "x": x, "out": out, "runs": runs}
    return dict(c, name=name) if name else c


def _ffn(n, d, f, back, name=None):
    c = {"op": "ffn", "n": n, "d": d, "f": f, "back": back}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token between two blocks: post norm, gate, residual, the next block's input norm
        _norm(1, 2048, F32, F32, "token", True, False, "norm 1 token"),
        # a prompt chunk of the length the library's prompt benchmark uses, expert outputs in fp32
        _norm(1180, 2048, F32, F32, "channel", True, False, "norm 1180 tokens"),
        # the longest chunk a call takes at the widest model, with a gate of its own for every value
        _norm(8192, 4096, BF16, BF16, "full", False, False, "norm 8192 full gate"),
        # layer-wise training: forward and every gradient, a width off every vector length
        _norm(1177, 1001, BF16, F32, "channel", True, True, "norm train odd"),
        # a verify batch: eight tokens, each of another request with its own adapter
        _adapters(8, 2048, 2048, 8, 16, False, BF16, F32, False, "adapters 8 tokens"),
        # a decode batch of many requests, some without an adapter, ranks of all kinds
        _adapters(61, 2048, 2048, 24, 64, True, BF16, BF16, False, "adapters 61 tokens mixed"),
        # several prompts in one chunk, fp32 activations between blocks
        _adapters(1180, 2048, 2048, 5, 33, True, F32, F32, True, "adapters 1180 tokens"),
        # the longest chunk, three long prompts
        _adapters(8192, 2048, 4096, 3, 64, False, BF16, BF16, True, "adapters 8192 tokens"),
        # one token through a block of the expert's own shape
        _ffn(1, 2048, 768, False, "ffn 1 token"),
        # a verify batch through a wide dense block: bound by the weights' bytes
        _ffn(8, 2048, 8192, False, "ffn 8 tokens"),
        # layer-wise training on a short prompt, sizes that end inside tiles
        _ffn(1180, 2048, 1000, True, "ffn train 1180"),
        # layer-wise training at the longest chunk
        _ffn(8192, 2048, 8192, True, "ffn train 8192"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adapters", "ffn"])
    if op == "norm":
        n, d = _log(rng, 1, 8192), _log(rng, 64, 4096)
        return _norm(n, d, rng.choice([F32, BF16]), rng.choice([F32, BF16]),
                     rng.choice(["none", "channel", "token", "full"]), rng.random() < 0.5, rng.random() < 0.4)
    if op == "adapters":
        n = _log(rng, 1, 8192)
        slots = min(_log(rng, 1, 64), max(1, 65536 // n))
        return _adapters(n, 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512), slots, _log(rng, 1, 128),
                         rng.random() < 0.6, rng.choice([F32, BF16]), rng.choice([F32, BF16]), rng.random() < 0.5)
    n, d, f = _log(rng, 1, 8192), 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 1024)
    back = rng.random() < 0.5
    while n * d * f > 8192 * 2048 * 8192:
        n = max(1, n // 2)
    return _ffn(n, d, f, back)


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return v.mul_(std).add_(mean).to(dtype)


def _inputs(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        s["o"] = _randn(g, n, d, std=0.3, dtype=_TYPES[case["o"]])            # a block's output
        s["res"] = _randn(g, n, d, std=2.0, dtype=_TYPES[case["res"]])        # the residual stream
        s["w"] = _randn(g, d, std=0.2, mean=1.0, dtype=torch.float32)
        s["w_next"] = _randn(g, d, std=0.2, mean=1.0, dtype=torch.float32)
        shape = {"none": None, "channel": (d,), "token": (n, 1), "full": (n, d)}[case["gate"]]
        s["gate"] = None if shape is None else _randn(g, *shape, dtype=torch.bfloat16)
        if case["back"]:
            s["d_res"] = _randn(g, n, d, std=0.1, dtype=_TYPES[case["res"]])  # gradient of the new residual
            s["d_h"] = _randn(g, n, d, std=0.1, dtype=torch.bfloat16)         # gradient of the next block's input
    elif case["op"] == "adapters":
        n, k, r = case["n"], case["slots"], case["rank"]
        s["x"] = _randn(g, n, case["d_in"], dtype=_TYPES[case["x"]])
        s["base"] = _randn(g, n, case["d_out"], dtype=_TYPES[case["out"]])    # the shared block's output
        s["a"] = _randn(g, k, r, case["d_in"], std=case["d_in"] ** -0.5)
        s["b"] = _randn(g, k, case["d_out"], r, std=r ** -0.5)
        h = torch.Generator()
        h.manual_seed(int(seed))
        ranks = [r] * k
        if case["mixed"]:
            ranks = torch.randint(1, r + 1, (k,), generator=h).tolist()
        ids = torch.randint(-1 if case["mixed"] else 0, k, (n,), generator=h)
        s["ranks"], s["scales"] = ranks, [0.5 + i / k for i in range(k)]
        s["ids"] = (ids.sort().values if case["runs"] else ids).to(torch.int32).cuda()
        live = torch.arange(r)[None, :] < torch.tensor(ranks)[:, None]
        s["live"] = live.cuda()                                               # [slots, rank]
        s["scale"] = torch.tensor(s["scales"], dtype=torch.float32).cuda()
    else:
        n, d, f = case["n"], case["d"], case["f"]
        s["x"] = _randn(g, n, d)
        s["wg"] = _randn(g, f, d, std=d ** -0.5)
        s["wu"] = _randn(g, f, d, std=d ** -0.5)
        s["wd"] = _randn(g, d, f, std=f ** -0.5)
        if case["back"]:
            s["dy"] = _randn(g, n, d, std=0.1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "adapters":  # the adapters' handle, loaded once as a server does
        import expert_ffn_gemv_b200 as P

        h = P.Adapters(d_in=case["d_in"], d_out=case["d_out"], max_adapters=case["slots"], max_rank=case["rank"],
                       max_tokens=case["n"])
        for i, r in enumerate(s["ranks"]):
            h.load(i, s["a"][i, :r].contiguous(), s["b"][i, :, :r].contiguous(), s["scales"][i])
        s["handle"] = h
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    o, res, w, wn = s["o"].float(), s["res"].float(), s["w"], s["w_next"]
    q = _rms(o)
    u = o * q * w
    a = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"].float())
    out = {"res": (res + SCALE * (a * u)).to(s["res"].dtype)}
    if c["next"]:
        x = out["res"].float()  # the next norm reads the residual as it is stored
        p = _rms(x)
        out["h"] = (x * p * wn).to(torch.bfloat16)
    if c["back"]:
        dr = s["d_res"].float()
        if c["next"]:
            dh = s["d_h"].float()
            t = dh * wn
            dr = (dr + p * (t - x * (p * p) * (t * x).mean(-1, keepdim=True))).to(s["res"].dtype)
            out["d_res"], out["d_w_next"] = dr, (dh * x * p).sum(0)
            dr = dr.float()
        du = SCALE * dr * a
        t = du * w
        out["d_o"] = (q * (t - o * (q * q) * (t * o).mean(-1, keepdim=True))).to(s["o"].dtype)
        out["d_w"] = (du * o * q).sum(0)
        if s["gate"] is not None:
            dg = SCALE * dr * u * (a * (1.0 - a))
            if c["gate"] == "channel":
                dg = dg.sum(0)
            if c["gate"] == "token":
                dg = dg.sum(-1, keepdim=True)
            out["d_gate"] = dg.to(s["gate"].dtype)
    return out


def _plain_adapters(s):
    n = s["x"].shape[0]
    k, r, d = s["a"].shape
    v = (s["x"].float() @ s["a"].float().reshape(k * r, d).T).reshape(n, k, r)
    mine = s["ids"][:, None] == torch.arange(k, device=s["ids"].device)[None, :]
    v = torch.where(mine[:, :, None] & s["live"][None], v * s["scale"][None, :, None], torch.zeros_like(v))
    b = s["b"].float().permute(0, 2, 1).reshape(k * r, -1)
    return (s["base"].float() + v.reshape(n, k * r) @ b).to(s["base"].dtype)


def _plain_ffn(s):
    x, wg, wu, wd = s["x"].float(), s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u = x @ wg.T, x @ wu.T
    sg = torch.sigmoid(g)
    h = g * sg * u
    out = {"y": (h @ wd.T).to(s["x"].dtype)}
    if s["case"]["back"]:
        dy = s["dy"].float()
        dh = dy @ wd
        dg = dh * u * (sg * (1.0 + g * (1.0 - sg)))
        du = dh * (g * sg)
        grads = {"d_x": dg @ wg + du @ wu, "d_wg": dg.T @ x, "d_wu": du.T @ x, "d_wd": dy.T @ h}
        out.update({key: v.to(s["x"].dtype) for key, v in grads.items()})
    return out


# ------------------------------------------------------------------------------ the package's calls
def _own_norm(s):
    import expert_ffn_gemv_b200 as P

    c = s["case"]
    gate = dict(weight=s["w"], eps=EPS, gate=s["gate"], gate_act="sigmoid", scale=SCALE)
    out, dr = {}, s.get("d_res")
    if c["next"]:
        out["res"], out["h"] = P.norm_out(s["o"], s["res"], next_weight=s["w_next"], next_eps=EPS,
                                          next_dtype=torch.bfloat16, **gate)
    else:
        out["res"] = P.norm_out(s["o"], s["res"], **gate)
    if not c["back"]:
        return out
    if c["next"]:
        dr, out["d_w_next"] = P.norm_in_backward(out["res"], s["w_next"], s["d_h"], eps=EPS, d_residual=dr)
        out["d_res"] = dr
    out["d_o"], out["d_w"], dg = P.norm_out_backward(s["o"], dr, **gate)
    if dg is not None:
        out["d_gate"] = dg
    return out


def _own_adapters(s):
    return s["handle"].apply(s["x"], s["base"], s["ids"])


def _own_ffn(s):
    import expert_ffn_gemv_b200 as P

    w = (s["wg"], s["wu"], s["wd"])
    if not s["case"]["back"]:
        return {"y": P.ffn_forward(s["x"], *w)}
    y, saved = P.ffn_forward(s["x"], *w, save=True)
    dx, dwg, dwu, dwd = P.ffn_backward(s["dy"], s["x"], *w, saved)
    return {"y": y, "d_x": dx, "d_wg": dwg, "d_wu": dwu, "d_wd": dwd}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "adapters": _own_adapters, "ffn": _own_ffn}[op](state)
    return {"norm": _plain_norm, "adapters": _plain_adapters, "ffn": _plain_ffn}[op](state)


# ------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        ob, rb = _BYTES[case["o"]], _BYTES[case["res"]]
        gate = 2 * {"none": 0, "channel": d, "token": n, "full": n * d}[case["gate"]]
        nbytes = n * d * (ob + 2 * rb) + 4 * d + gate
        flops = 8.0 * n * d
        if case["next"]:
            nbytes += 2 * n * d + 4 * d
            flops += 4.0 * n * d
        if case["back"]:  # read d_res, write d_o, the gradients of weight and gate; the next norm: d_h, d_res
            nbytes += n * d * (rb + ob) + 4 * d + gate
            flops += 16.0 * n * d
            if case["next"]:
                nbytes += n * d * (2 + rb) + 4 * d
                flops += 10.0 * n * d
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "adapters":
        n, r = case["n"], case["rank"] / (2.0 if case["mixed"] else 1.0)
        w = 2 * min(case["slots"], n) * r * (case["d_in"] + case["d_out"])
        nbytes = n * (case["d_in"] * _BYTES[case["x"]] + 2 * case["d_out"] * _BYTES[case["out"]] + 4) + w
        return {"bytes": nbytes, "flops": 2.0 * n * r * (case["d_in"] + case["d_out"])}
    n, d, f = case["n"], case["d"], case["f"]
    nbytes, flops = 2 * (3 * d * f + 2 * n * d), 6.0 * n * d * f
    if case["back"]:
        nbytes, flops = nbytes + 2 * (3 * d * f + 2 * n * d), 3 * flops
    return {"bytes": nbytes, "flops": flops}


# --------------------------------------------------------------------------- definitions in 64 bits
def _unit(v):
    """v / sqrt(mean(v^2) + eps), and that root."""
    root = ((v * v).sum(dim=1, keepdim=True) / v.shape[1] + EPS) ** 0.5
    return v / root, root


def _unit_gradient(unit, root, d):
    """Gradient of _unit: the part of d across the unit vector, over the root."""
    return (d - unit * ((d * unit).sum(dim=1, keepdim=True) / unit.shape[1])) / root


def _exact_norm(s):
    c = s["case"]
    o, w, wn = s["o"].double(), s["w"].double(), s["w_next"].double()
    n1, root1 = _unit(o)
    a = torch.ones((), dtype=torch.float64, device=o.device)
    if s["gate"] is not None:
        a = 1.0 / (1.0 + torch.exp(-s["gate"].double()))
    out = {"res": s["res"].double() + SCALE * a * (n1 * w)}
    if c["next"]:
        n2, root2 = _unit(out["res"].to(s["res"].dtype).double())
        out["h"] = n2 * wn
    if c["back"]:
        dr = s["d_res"].double()
        if c["next"]:
            dh = s["d_h"].double()
            dr = dr + _unit_gradient(n2, root2, dh * wn)
            out["d_res"], out["d_w_next"] = dr, (dh * n2).sum(dim=0)
            dr = dr.to(s["res"].dtype).double()
        dz = SCALE * dr
        out["d_o"] = _unit_gradient(n1, root1, dz * a * w)
        out["d_w"] = (dz * a * n1).sum(dim=0)
        if s["gate"] is not None:
            dg = dz * (n1 * w) * a * (1.0 - a)
            out["d_gate"] = {"channel": lambda: dg.sum(dim=0), "token": lambda: dg.sum(dim=1, keepdim=True),
                             "full": lambda: dg}[c["gate"]]()
    return out


def _exact_adapters(s):
    y = s["base"].double()
    ids = s["ids"].cpu()
    for i, r in enumerate(s["ranks"]):
        t = torch.nonzero(ids == i).flatten().to(y.device)
        if t.numel():
            low = torch.einsum("td,rd->tr", s["x"][t].double(), s["a"][i, :r].double())
            y[t] += s["scales"][i] * torch.einsum("tr,or->to", low, s["b"][i, :, :r].double())
    return y


def _exact_ffn(s):
    x, wg, wu, wd = (s[key].double() for key in ("x", "wg", "wu", "wd"))
    g, u = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
    e = torch.exp(-g)
    silu = g / (1.0 + e)
    out = {"y": torch.einsum("tf,df->td", silu * u, wd)}
    if s["case"]["back"]:
        dy = s["dy"].double()
        dh = torch.einsum("td,df->tf", dy, wd)
        slope = 1.0 / (1.0 + e) + g * e / (1.0 + e) ** 2
        dg, du = dh * u * slope, dh * silu
        out["d_x"] = torch.einsum("tf,fd->td", dg, wg) + torch.einsum("tf,fd->td", du, wu)
        out["d_wg"], out["d_wu"] = torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)
        out["d_wd"] = torch.einsum("td,tf->df", dy, silu * u)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "adapters": _exact_adapters, "ffn": _exact_ffn}[case["op"]](s)
