"""Waits of the block operators that run out: the call's status, and that nothing of it is left behind.

A limit set by hand has the rings' first copies held back for longer than it, so that the waits for them run
out.  The kernels then leave with an error word, once every copy of theirs has landed; the calls after them
are right."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    return P


@pytest.fixture
def limit(P):
    """Sets the rings' limit, in clocks; the default comes back at the end."""
    yield lambda clocks: P.moe_debug_set_ring_spin_limit(clocks)
    P.moe_debug_set_ring_spin_limit(0)


def randn(*shape, seed, std=1.0, mean=0.0, dtype=F):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


# sizes of every instantiation whose blocks are fed by a ring (at 2,048 columns from 1,776 rows on)
@pytest.mark.parametrize("n,d,back", [(2000, 264, False), (2000, 264, True), (1900, 2048, False), (1900, 2048, True),
                                      (2500, 4096, False), (2500, 4096, True), (700, 8192, False)])
@pytest.mark.parametrize("clocks", [20_000, 2_000_000])  # 10 us, 1 ms
def test_norm_rings(P, limit, n, d, back, clocks):
    o, res, w = randn(n, d, seed=1, std=0.5, dtype=BF), randn(n, d, seed=2), randn(d, seed=3, std=0.3, mean=1.0)

    def call():
        if back:
            return P.norm_out_backward(o, res, weight=w, eps=R.EPS)[:2]
        return P.norm_out(o, res, weight=w, eps=R.EPS, next_weight=w, next_eps=R.EPS)

    want = call()
    assert P.block_check() == P.MOE_OK
    limit(clocks)
    for _ in range(3):
        got = call()
        torch.cuda.synchronize()
        status = P.block_check()
        # (a hardware wait may suspend a thread for longer than the shorter limit)
        assert status == P.MOE_ERR_TIMEOUT or (clocks < 2_000_000 and all(torch.equal(a, b) for a, b in zip(got, want)))
        assert P.block_check() == P.MOE_OK  # reported once
    limit(0)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert P.block_check() == P.MOE_OK


@pytest.mark.parametrize("xt,bt", [(BF, BF), (BF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("n,rank", [(5, 16), (300, 33), (2500, 128)])  # clusters, single blocks, both tile sizes
@pytest.mark.parametrize("clocks", [20_000, 2_000_000])
def test_adapter_rings(P, limit, n, rank, xt, bt, clocks):
    h = P.Adapters(d_in=520, d_out=1032, max_adapters=2, max_rank=rank, max_tokens=n)
    for i in range(2):
        h.load(i, randn(rank - i, 520, seed=i, std=0.05, dtype=BF), randn(1032, rank - i, seed=5 + i, std=0.2, dtype=BF), 0.5 + i)
    x, base = randn(n, 520, seed=7, dtype=xt), randn(n, 1032, seed=8, dtype=bt)
    ids = (torch.arange(n) % 3 - 1).to(torch.int32).cuda()
    want = h.apply(x, base, ids)
    torch.cuda.synchronize()
    assert h.check() == P.MOE_OK
    limit(clocks)
    for _ in range(3):
        got = h.apply(x, base, ids)
        torch.cuda.synchronize()
        status = h.check()
        assert status == P.MOE_ERR_TIMEOUT or (clocks < 2_000_000 and torch.equal(got, want))
        assert torch.equal(got[ids == -1], base[ids == -1])  # these wait for nothing
        assert h.check() == P.MOE_OK
    limit(0)
    for _ in range(3):
        assert torch.equal(h.apply(x, base, ids), want)
    torch.cuda.synchronize()
    assert h.check() == P.MOE_OK
    h.close()


def test_check_waits_for_every_stream(P, limit):
    """torch's streams wait for nobody: the check has to."""
    x, w = randn(2000, 1024, seed=1), randn(1024, seed=2)
    side = torch.cuda.Stream()
    P.norm_in(x, w)
    for clocks, status in ((0, P.MOE_OK), (2_000_000, P.MOE_ERR_TIMEOUT), (0, P.MOE_OK)):
        limit(clocks)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)  # 0.2 s
            P.norm_in(x, w)
        assert not side.query()
        assert P.block_check() == status
        assert side.query()


def test_a_run_of_layers_reports_by_its_handle(P, limit):
    """The norm behind the experts waits in a ring; the one before them, whose weight is off a 16-byte boundary,
    has none, so that the experts see sound values."""
    import synth
    from helpers import load_layer_device, moe_for

    wl = synth.small_workload(d_model=512, d_ff=256, n_experts=32, top_k=4, n_shared=1, shared_d_ff=256)
    n = 2000
    m = moe_for(wl, 1, n, seed=3)
    load_layer_device(m, 0, wl, 3, 0)
    w = randn(513, seed=1, std=0.2, mean=1.0)[1:]
    x, out = randn(n, 512, seed=2, dtype=BF), torch.empty((n, 512), device="cuda")
    run = lambda: m.forward_blocks(0, [P.Block(norm_in=w)], x, out)
    run()
    torch.cuda.synchronize()
    assert m.check() == P.MOE_OK
    want = out.clone()
    limit(2_000_000)
    run()
    limit(0)
    torch.cuda.synchronize()
    assert P.block_check() == P.MOE_OK
    with pytest.raises(P.MoeError) as e:
        run()
    assert e.value.status == P.MOE_ERR_TIMEOUT
    run()
    torch.cuda.synchronize()
    assert m.check() == P.MOE_OK and torch.equal(out, want)
    m.close()


def test_the_next_call_reports(P, limit):
    """Once, whichever of the operators it is, and with nothing launched."""
    x, w = randn(2000, 1024, seed=1), randn(1024, seed=2)
    a, m = randn(12, 64, seed=3, dtype=BF), randn(64, 64, seed=4, dtype=BF)
    y, saved = P.ffn_forward(a, m, m, m, save=True)
    out = torch.full((3, 64), 7.0, device="cuda")
    calls = {"norm_in": lambda: P.norm_in(x[:3, :64], w[:64], out=out), "norm_out": lambda: P.norm_out(x[:3, :64], x[:3, :64], out=out),
             "norm_in_backward": lambda: P.norm_in_backward(x, w, x), "norm_out_backward": lambda: P.norm_out_backward(x, x),
             "ffn_forward": lambda: P.ffn_forward(a[:3], m, m, m, out=out), "ffn_backward": lambda: P.ffn_backward(y, a, m, m, m, saved)}
    for name, call in calls.items():
        limit(2_000_000)
        P.norm_in(x, w)
        limit(0)
        torch.cuda.synchronize()
        with pytest.raises(P.MoeError) as e:
            call()
        assert e.value.status == P.MOE_ERR_TIMEOUT and name in str(e.value)
        torch.cuda.synchronize()
        assert (out == 7).all()
    for call in calls.values():
        call()
    assert P.block_check() == P.MOE_OK


def test_first_call_inside_a_capture():
    """The page of error words is pinned by the first call that may wait, which may be one that is captured."""
    import subprocess
    import sys
    from pathlib import Path

    code = """
import torch
import expert_ffn_gemv_b200 as P
x, w = torch.randn(2000, 1024, device="cuda"), torch.randn(1024, device="cuda")
a, m = torch.randn(40, 64, device="cuda").bfloat16(), (torch.randn(64, 64, device="cuda") / 8).bfloat16()
torch.cuda.synchronize()
for call in (lambda: P.norm_in(x, w), lambda: P.ffn_forward(a, m, m, m)):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    graph.replay()
    assert torch.equal(y, call())
assert P.block_check() == P.MOE_OK
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
