"""A run of layers with their norms, gates, dense blocks and adapters (moe_forward_blocks): the same
bits as the single calls in order, and one layer's experts against the fp64 oracle."""
import numpy as np
import pytest
import torch

import synth
from helpers import (TIE_EPS, TOL_DECODE, TOL_PREFILL, compare_routing, load_layer_device, moe_for, oracle_layer, rel_l2,
                     route_buffers, x_f64)

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
D = 512


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    return P


def randn(*shape, seed, std=1.0, mean=0.0, dtype=F):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


@pytest.fixture(scope="module")
def model(P):
    wl = synth.small_workload(d_model=D, d_ff=256, n_experts=32, top_k=4, n_shared=1, shared_d_ff=256)
    m = moe_for(wl, 3, 512, seed=11)
    for l in range(3):
        load_layer_device(m, l, wl, 11, l)
    ad = P.Adapters(d_in=D, d_out=D, max_adapters=4, max_rank=24, max_tokens=512)
    for i in range(4):
        ad.load(i, randn(8 + 5 * i, D, seed=60 + i, std=D ** -0.5, dtype=BF), randn(D, 8 + 5 * i, seed=70 + i, std=0.1, dtype=BF), 0.5)
    yield wl, m, ad
    ad.close()
    m.close()


def blocks_of(P, ad, mixed=False):
    def ffn(s):
        return (randn(320, D, seed=s, std=D ** -0.5, dtype=BF), randn(320, D, seed=s + 1, std=D ** -0.5, dtype=BF),
                randn(D, 320, seed=s + 2, std=0.05, dtype=BF))

    w = [randn(D, seed=20 + i, std=0.2, mean=1.0) for i in range(8)]
    second = [t.to(BF) for t in w[3:6]] if mixed else w[3:6]  # another type: the norms cannot share a pass
    return [P.Block(norm_in=w[0], norm_out=w[1], gate=w[2], gate_act="sigmoid", scale=0.5, ffn=ffn(40), adapters=ad),
            P.Block(norm_in=second[0], norm_out=second[1], unit_offset=mixed, ffn=ffn(50)),
            P.Block(norm_in=w[6], gate=w[7], scale=-0.25, adapters=ad)]


def by_hand(P, m, blocks, x, ids, out_dtype):
    res, n = x, x.shape[0]
    for l, b in enumerate(blocks):
        a = P.norm_in(res, b.norm_in, eps=b.eps, unit_offset=b.unit_offset, out_dtype=BF)
        o = torch.empty((n, D), device="cuda")
        m.forward(l, a, o)
        if b.ffn:
            P.ffn_forward(a, *b.ffn, add=o, out=o)
        if b.adapters:
            b.adapters.apply(a, o, ids, out=o)
        res = P.norm_out(o, res, weight=b.norm_out, eps=b.eps, unit_offset=b.unit_offset, gate=b.gate, gate_act=b.gate_act,
                         scale=b.scale, out_dtype=out_dtype if l == len(blocks) - 1 else F)
    return res


@pytest.mark.parametrize("n", [1, 8, 40, 300])
@pytest.mark.parametrize("mixed", [False, True])
def test_blocks_are_the_single_calls(P, model, n, mixed):
    wl, m, ad = model
    blocks = blocks_of(P, ad, mixed)
    x = randn(n, D, seed=n, dtype=BF)
    ids = (torch.arange(n) % 5 - 1).to(torch.int32).cuda()
    out = torch.empty((n, D), device="cuda")
    m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
    want = by_hand(P, m, blocks, x, ids, F)
    assert torch.equal(out, want) and torch.isfinite(out).all()
    m.forward_blocks(1, blocks[1:2], x, out)  # a run of one layer, from the middle
    a = P.norm_in(x, blocks[1].norm_in, eps=1e-6, unit_offset=mixed, out_dtype=BF)
    o = torch.empty_like(out)
    m.forward(1, a, o)
    P.ffn_forward(a, *blocks[1].ffn, add=o, out=o)
    assert torch.equal(out, P.norm_out(o, x, weight=blocks[1].norm_out, eps=1e-6, unit_offset=mixed, out_dtype=F))


@pytest.mark.parametrize("n,tol", [(6, TOL_DECODE), (64, TOL_PREFILL)])
def test_experts_between_the_norms_against_the_oracle(P, model, n, tol):
    wl, m, _ = model
    w = randn(D, seed=20, std=0.2, mean=1.0)
    x = randn(n, D, seed=5, std=30.0, dtype=BF)
    out, rb = torch.empty((n, D), device="cuda"), route_buffers(n, wl.top_k, wl.n_experts)
    m.forward_blocks(0, [P.Block(norm_in=w)], x, out, routes=[rb])
    a = P.norm_in(x, w, eps=1e-6, out_dtype=BF)
    xs = x_f64(wl, a.view(torch.int16).cpu().numpy().view(np.uint16))
    ref = oracle_layer(wl, 11, 0).forward(xs)
    bad, _ = compare_routing(rb["idx"].cpu().numpy(), ref["idx"], ref["margin"], wl.n_experts, rb["counts"].cpu().numpy())
    assert bad == 0
    y = out.double().cpu().numpy() - x.double().cpu().numpy()
    # the add to a residual of up to 2^7 rounds by 2^-18 a value: against experts' outputs of norm |y|
    slack = 2.0 ** -18 * np.sqrt(D) / np.linalg.norm(ref["y"], axis=-1).min()
    assert rel_l2(y, ref["y"], ref["margin"] >= TIE_EPS) <= tol + slack


def test_a_long_chain_stays_finite(P, model):
    """The norms keep a residual chain in range: 30 passes over the same layers."""
    wl, m, ad = model
    blocks = blocks_of(P, ad)
    n = 8
    x, ids = randn(n, D, seed=1, std=100.0, dtype=BF), torch.zeros(n, dtype=torch.int32, device="cuda")
    out = torch.empty((n, D), device="cuda")
    for _ in range(30):
        m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
        x = out.to(BF)
    assert torch.isfinite(out).all() and out.abs().max() < 1e5


@pytest.mark.parametrize("n", [4, 40])
def test_captured(P, model, n):
    wl, m, ad = model
    blocks = blocks_of(P, ad)
    x, out = randn(n, D, seed=1, dtype=BF), torch.empty((n, D), device="cuda")
    ids = torch.full((n,), 2, dtype=torch.int32, device="cuda")
    m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
    for k in range(2):
        x.copy_(randn(n, D, seed=7 + k, dtype=BF))
        ids.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, by_hand(P, m, blocks, x, ids, F))


def test_training_step_of_a_layer(P):
    """Norm, dense block, norm with gate and residual, and all their gradients in one run, against the
    chain of the 64-bit definitions on the values as they are stored between the calls."""
    import block_reference as R

    n, f = 70, 264
    x, w1, w2 = randn(n, D, seed=1), randn(D, seed=2, std=0.2, mean=1.0), randn(D, seed=3, std=0.2, mean=1.0)
    gate = randn(n, 1, seed=4, dtype=BF)
    wt = (randn(f, D, seed=5, std=D ** -0.5, dtype=BF), randn(f, D, seed=6, std=D ** -0.5, dtype=BF),
          randn(D, f, seed=7, std=f ** -0.5, dtype=BF))
    dres = randn(n, D, seed=8, std=0.1)
    a = P.norm_in(x, w1, out_dtype=BF)
    o, saved = P.ffn_forward(a, *wt, save=True)
    kw = dict(weight=w2, gate=gate, gate_act="sigmoid", scale=0.5)
    P.norm_out(o, x, **kw)
    do, dw2, dgate = P.norm_out_backward(o, dres, **kw)
    da, dwg, dwu, dwd = P.ffn_backward(do, a, *wt, saved)
    dx, dw1 = P.norm_in_backward(x, w1, da, d_residual=dres)

    p = {"x": x, "w1": w1, "w2": w2, "gate": gate, "wg": wt[0], "wu": wt[1], "wd": wt[2]}
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    aa = p["x"] * torch.rsqrt((p["x"] ** 2).mean(-1, keepdim=True) + 1e-6) * p["w1"]
    h = torch.nn.functional.silu(aa @ p["wg"].T) * (aa @ p["wu"].T)
    oo = h @ p["wd"].T
    res = p["x"] + 0.5 * torch.sigmoid(p["gate"]) * (oo * torch.rsqrt((oo ** 2).mean(-1, keepdim=True) + 1e-6) * p["w2"])
    res.backward(dres.double())
    got = {"x": dx, "w1": dw1, "w2": dw2, "gate": dgate, "wg": dwg, "wu": dwu, "wd": dwd}
    # at most eight roundings to bf16 (2^-8 of a value, independent) lie between the inputs and any gradient,
    # in 2-norm at most sqrt(8) 2^-8 = 1.1e-2
    for k, v in got.items():
        ref = p[k].grad
        assert ((v.double() - ref).norm() / ref.norm()).item() <= 8 ** 0.5 * R.HALF[BF], k


def test_refusals(P, model):
    wl, m, ad = model
    b = blocks_of(P, ad)
    x, out = randn(4, D, seed=1, dtype=BF), torch.empty((4, D), device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(P.MoeError) as e:
        m.forward_blocks(0, b, x, out)
    assert "adapter_ids" in str(e.value)
    with pytest.raises(P.MoeError):
        m.forward_blocks(1, b, x, out, adapter_ids=ids)  # one layer too many
    big = P.Adapters(d_in=D, d_out=D, max_adapters=1, max_rank=1, max_tokens=2)
    with pytest.raises(P.MoeError) as e:
        m.forward_blocks(0, [P.Block(norm_in=b[0].norm_in, adapters=big)], x, out, adapter_ids=ids)
    assert "max_tokens" in str(e.value)
    big.close()
    for bad in (dict(x_in=x.float()), dict(x_out=out[:3]), dict(x_out=out.to(BF)), dict(adapter_ids=ids[:2]), dict(x_in=x.cpu()),
                dict(blocks=[P.Block(norm_in=b[0].norm_in, norm_out=b[1].norm_in.to(BF))]),
                dict(blocks=[P.Block(norm_in=b[0].norm_in[:-1])]), dict(blocks=[P.Block(norm_in=b[0].norm_in, adapters=big)]),
                dict(blocks=[P.Block(norm_in=b[0].norm_in, gate_act="tanh")])):
        kw = {**dict(blocks=b, x_in=x, x_out=out, adapter_ids=ids), **bad}
        with pytest.raises(ValueError):
            m.forward_blocks(0, **kw)


@pytest.mark.parametrize("n", [3, 300])
def test_ids_out_of_range_in_a_run(P, model, n):
    """A run of layers that share a handle takes them as -1 throughout, however far the device has got; the
    next run returns the error before anything of it is launched."""
    wl, m, ad = model
    blocks = blocks_of(P, ad)
    x, out = randn(n, D, seed=1, dtype=BF), torch.empty((n, D), device="cuda")
    ids = (torch.arange(n) % 5 - 1).to(torch.int32).cuda()
    want = torch.empty_like(out)
    m.forward_blocks(0, blocks, x, want, adapter_ids=ids)
    ids[ids == -1] = 77
    for _ in range(5):  # the first layer's report may come before or after the third layer's launch
        m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and ad.check() == P.MOE_ERR_DEVICE_FAULT and ad.check() == P.MOE_OK
    m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
    torch.cuda.synchronize()
    out.fill_(7)
    routes = [{k: v.fill_(-5) for k, v in route_buffers(n, wl.top_k, wl.n_experts).items()} for _ in range(2)]
    with pytest.raises(P.MoeError) as e:  # only the second layer of this run has the adapters
        m.forward_blocks(1, blocks[1:], x, out, adapter_ids=ids, routes=routes)
    assert e.value.status == P.MOE_ERR_DEVICE_FAULT and "adapter id" in str(e.value)
    torch.cuda.synchronize()
    assert (out == 7).all() and all((v == -5).all() for r in routes for v in r.values())
    m.forward_blocks(0, blocks, x, out, adapter_ids=ids)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ad.check() == P.MOE_ERR_DEVICE_FAULT


def test_a_bad_second_layer_is_refused_before_the_first_is_launched(P, model):
    wl, m, ad = model
    n = 9
    w = randn(D, seed=20, std=0.2, mean=1.0)
    x, out = randn(n, D, seed=1, dtype=BF), torch.full((n, D), 7.0, device="cuda")
    mats = [randn(320 * D + 8, seed=30 + i, std=0.05, dtype=BF) for i in range(3)]
    ffn = [t[:320 * D].view(s) for t, s in zip(mats, ((320, D), (320, D), (D, 320)))]
    off = [t[1:320 * D + 1].view(s) for t, s in zip(mats, ((320, D), (320, D), (D, 320)))]  # 2 bytes on
    odd = [t[:12 * D].view(s) for t, s in zip(mats, ((12, D), (12, D), (D, 12)))]
    blocks = [P.Block(norm_in=w, ffn=(off[0], ffn[1], ffn[2])), P.Block(norm_in=w, ffn=(ffn[0], off[1], ffn[2])),
              P.Block(norm_in=w, ffn=(ffn[0], ffn[1], off[2])), P.Block(norm_in=w, ffn=tuple(odd)),
              P.Block(norm_in=w, eps=-1.0), P.Block(norm_in=w, eps=float("nan")), P.Block(norm_in=w, unit_offset=2),
              P.Block(norm_in=w, unit_offset=-1)]
    routes = [{k: v.fill_(-5) for k, v in route_buffers(n, wl.top_k, wl.n_experts).items()} for _ in range(2)]
    for b in blocks:
        with pytest.raises(P.MoeError) as e:
            m.forward_blocks(0, [P.Block(norm_in=w), b], x, out, routes=routes)
        assert e.value.status == P.MOE_ERR_INVALID_ARGUMENT
        torch.cuda.synchronize()
        assert (out == 7).all() and all((v == -5).all() for r in routes for v in r.values()), b
    arr = (P.moe_block * 1)(P.Block(norm_in=w, gate=w, ffn=tuple(ffn)).args(D, x.device))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    run = lambda work: P.lib().moe_forward_blocks(m.h, 0, 1, arr, x.data_ptr(), out.data_ptr(), n, None, work, 1 << 19, 0, None)
    assert run(ws.data_ptr() + 8) == P.MOE_ERR_INVALID_ARGUMENT and run(None) == P.MOE_ERR_INVALID_ARGUMENT
    arr[0].gate_act = 2
    assert run(ws.data_ptr()) == P.MOE_ERR_INVALID_ARGUMENT
    arr[0].gate_act = 1
    torch.cuda.synchronize()
    assert (out == 7).all()
    assert run(ws.data_ptr()) == P.MOE_OK
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
