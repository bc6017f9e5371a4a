"""Low-rank adapters of many requests against their definition in 64 bits."""
import ctypes as C

import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    return P


def rng(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def make(P, d_in, d_out, ranks, max_tokens, seed=0, slots=None, host=False):
    """A handle and what its slots hold."""
    h = P.Adapters(d_in=d_in, d_out=d_out, max_adapters=slots or len(ranks), max_rank=max(max(ranks), 1), max_tokens=max_tokens)
    a, b, sc = [], [], []
    for i, r in enumerate(ranks):
        if r == 0:
            a.append(None), b.append(None), sc.append(0.0)
            continue
        g = rng(100 * seed + i)
        a.append((torch.randn(r, d_in, generator=g) * d_in ** -0.5).to(BF))
        b.append((torch.randn(d_out, r, generator=g) * r ** -0.5).to(BF))
        sc.append(0.5 + i)
        if host:
            h.load(i, a[-1], b[-1], sc[-1])
        else:
            h.load(i, a[-1].cuda(), b[-1].cuda(), sc[-1])
    return h, a, b, sc


def data(n, d_in, d_out, xt, bt, seed=1):
    g = rng(seed)
    return torch.randn(n, d_in, generator=g).to(xt).cuda(), torch.randn(n, d_out, generator=g).to(bt).cuda()


def check(x, base, ids, a, b, sc, out, rank):
    ref, size = R.adapters(x, base, ids, a, b, sc)
    R.near(out, ref, R.adapters_tolerance(ref, size, base, x.shape[1], rank, out.dtype), "out")


@pytest.mark.parametrize("xt,bt", [(BF, BF), (BF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("n", [1, 8, 17, 61, 256, 257, 1100])
def test_tokens_and_types(P, n, xt, bt):
    ranks = [16, 1, 33, 64, 7]
    h, a, b, sc = make(P, 512, 264, ranks, 1100)
    ids = torch.randint(-1, len(ranks), (n,), generator=rng(n)).to(torch.int32).cuda()
    x, base = data(n, 512, 264, xt, bt)
    out = h.apply(x, base, ids)
    check(x, base, ids, a, b, sc, out, 64)
    assert torch.equal(out, h.apply(x, base, ids))
    none = ids == -1
    assert torch.equal(out[none], base[none])
    assert h.check() == P.MOE_OK
    # in place: the same bits
    buf = base.clone()
    assert h.apply(x, buf, ids, out=buf) is buf and torch.equal(buf, out)
    h.close()


@pytest.mark.parametrize("d_in,d_out,rank", [(8, 8, 1), (8, 40, 128), (40, 8, 16), (2048, 2048, 128), (1032, 4096, 65),
                                             (4096, 1000, 17)])
@pytest.mark.parametrize("n", [3, 40, 1500])
def test_sizes(P, d_in, d_out, rank, n):
    h, a, b, sc = make(P, d_in, d_out, [rank, max(1, rank // 2)], 1500, seed=3)
    ids = (torch.arange(n) % 3 - 1).to(torch.int32).cuda()
    for xt, bt in ((BF, BF), (F, F)):
        x, base = data(n, d_in, d_out, xt, bt)
        check(x, base, ids, a, b, sc, h.apply(x, base, ids), rank)
    h.close()


def test_one_adapter_runs_and_all_without(P):
    h, a, b, sc = make(P, 256, 256, [8, 24], 3000)
    x, base = data(3000, 256, 256, BF, BF)
    for ids in (torch.zeros(3000), torch.full((3000,), -1), torch.arange(3000) // 1700, torch.full((3000,), 1)):
        ids = ids.to(torch.int32).cuda()
        out = h.apply(x, base, ids)
        check(x, base, ids, a, b, sc, out, 24)
        # a token's result does not depend on its company
        few = h.apply(x[1690:1710].contiguous(), base[1690:1710].contiguous(), ids[1690:1710].contiguous())
        ref, size = R.adapters(x[1690:1710], base[1690:1710], ids[1690:1710], a, b, sc)
        R.near(few, ref, R.adapters_tolerance(ref, size, base[1690:1710], 256, 24, BF), "few")
    h.close()


@pytest.mark.parametrize("xt,bt", [(BF, BF), (BF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("rank", [3, 32, 48, 128])
def test_long_prompts(P, xt, bt, rank):
    """Sizes of the widest tiles, in place too, ragged groups, some tokens without an adapter."""
    n = 2500
    h, a, b, sc = make(P, 264, 1032, [rank, max(1, rank - 5), 1], n, seed=6)
    ids = (torch.randint(-1, 3, (n,), generator=rng(8)).sort().values).to(torch.int32).cuda()
    x, base = data(n, 264, 1032, xt, bt)
    out = h.apply(x, base, ids)
    check(x, base, ids, a, b, sc, out, rank)
    buf = base.clone()
    h.apply(x, buf, ids, out=buf)
    assert torch.equal(buf, out)
    # the tokens' order is of no account
    order = torch.randperm(n, generator=rng(9)).cuda()
    assert torch.equal(h.apply(x[order].contiguous(), base[order].contiguous(), ids[order].contiguous()), out[order])
    h.close()


def test_many_slots_one_token_each(P):
    n = 300
    h, a, b, sc = make(P, 128, 128, [1 + i % 20 for i in range(n)], 512)
    x, base = data(n, 128, 128, BF, F)
    ids = torch.randperm(n, generator=rng(5)).to(torch.int32).cuda()
    check(x, base, ids, a, b, sc, h.apply(x, base, ids), 20)
    check(x[:200], base[:200], ids[:200], a, b, sc, h.apply(x[:200], base[:200], ids[:200]), 20)
    h.close()


@pytest.mark.parametrize("xt,bt", [(BF, BF), (BF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("n,rank", [(127, 20), (128, 64), (129, 20), (129, 64), (4700, 16), (5001, 16), (8192, 32), (8191, 33)])
def test_where_the_forms_change(P, n, rank, xt, bt):
    """Both sides of the sizes at which ids are counted and tiles get wider; ids in any order."""
    h, a, b, sc = make(P, 136, 72, [rank, 1, rank // 2], n, seed=4, slots=5)
    ids = torch.randint(-1, 3, (n,), generator=rng(n)).to(torch.int32).cuda()
    x, base = data(n, 136, 72, xt, bt)
    out = h.apply(x, base, ids)
    check(x, base, ids, a, b, sc, out, rank)
    assert torch.equal(out, h.apply(x, base, ids)) and h.check() == P.MOE_OK
    buf = base.clone()
    assert torch.equal(h.apply(x, buf, ids, out=buf), out)
    h.close()


@pytest.mark.parametrize("host", [False, True])
def test_replacing_and_emptying_a_slot(P, host):
    h, a, b, sc = make(P, 128, 64, [64, 8], 8, host=host)
    x, base = data(4, 128, 64, BF, F)
    ids = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    check(x, base, ids, a, b, sc, h.apply(x, base, ids), 64)
    _, a2, b2, _ = make(P, 128, 64, [3, 8], 8, seed=9)
    h.load(0, a2[0] if host else a2[0].cuda(), b2[0] if host else b2[0].cuda(), -1.5)
    a[0], b[0], sc[0] = a2[0], b2[0], -1.5  # a smaller rank where a larger one was
    check(x, base, ids, a, b, sc, h.apply(x, base, ids), 64)
    h.load(1, None, None)
    a[1] = None
    out = h.apply(x, base, ids)
    check(x, base, ids, a, b, sc, out, 64)
    torch.cuda.synchronize()
    assert h.check() == P.MOE_ERR_DEVICE_FAULT  # tokens asked for an empty slot
    assert h.check() == P.MOE_OK
    h.close()


@pytest.mark.parametrize("n", [5, 300])
def test_ids_out_of_range(P, n):
    h, a, b, sc = make(P, 64, 64, [4, 4, 0], 512)
    x, base = data(n, 64, 64, BF, BF)
    ids = torch.zeros(n, dtype=torch.int32)
    bad = [3, -2, 2 ** 31 - 1, -2 ** 31]
    ids[:4] = torch.tensor(bad, dtype=torch.int32)
    ids = ids.cuda()
    out = h.apply(x, base, ids)
    torch.cuda.synchronize()
    assert torch.equal(out[:4], base[:4])
    check(x, base, ids, a, b, sc, out, 4)
    with pytest.raises(P.MoeError) as e:  # reported once, by the next call
        h.apply(x, base, ids)
    assert e.value.status == P.MOE_ERR_DEVICE_FAULT and "id" in str(e.value)
    buf = base.clone()
    h.apply(x, buf, ids, out=buf)
    torch.cuda.synchronize()
    assert torch.equal(buf, out) and h.check() == P.MOE_ERR_DEVICE_FAULT
    h.close()


def test_values_that_are_not_finite_stay_in_their_row(P):
    h, a, b, sc = make(P, 64, 64, [5, 5], 64)
    h.load(1, torch.full((5, 64), float("nan"), dtype=BF), torch.full((64, 5), float("inf"), dtype=BF), 1.0)
    x, base = data(20, 64, 64, F, F)
    ids = torch.zeros(20, dtype=torch.int32)
    ids[3] = 1
    x[4, 9] = float("nan")
    x[5, 2] = float("inf")
    x[6, 2] = 3.4e38
    out = h.apply(x, base, ids.cuda())
    ref, size = R.adapters(x, base, ids, a[:1], b[:1], sc[:1])
    rows = [t for t in range(20) if t not in (3, 4, 5, 6)]
    R.near(out[rows], ref[rows], R.adapters_tolerance(ref, size, base, 64, 5, F)[rows], "the other rows")
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all()
    assert not torch.isfinite(out[5]).any()
    assert not torch.isnan(out[6]).all()
    h.close()


def test_strided_rows_and_rows_behind_the_last(P):
    h, a, b, sc = make(P, 64, 128, [9, 2], 64)
    x, base = data(20, 96, 160, BF, F)
    x, base = x[:, 16:80], base[:, 8:136]
    ids = (torch.arange(20) % 2).to(torch.int32).cuda()
    buf = torch.full((24, 200), 7.0, device="cuda")
    out = h.apply(x, base, ids, out=buf[:20, 4:132])
    check(x, base, ids, a, b, sc, out, 9)
    assert (buf[20:] == 7).all() and (buf[:, :4] == 7).all() and (buf[:, 132:] == 7).all()
    h.close()


@pytest.mark.parametrize("n", [12, 500])
def test_graph_and_stream(P, n):
    """A replay reads the ids, the inputs and the slots as they are then."""
    h, a, b, sc = make(P, 256, 256, [16, 32], 512)
    x, base = data(n, 256, 256, BF, BF)
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    out = h.apply(x, base, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        h.apply(x, base, ids, out=out)
    torch.cuda.synchronize()
    for k in range(2):
        ids.copy_((torch.arange(n) % 3 - 1 + k).clamp(-1, 1).to(torch.int32))
        if k:
            _, a2, b2, _ = make(P, 256, 256, [8, 32], 8, seed=4)
            h.load(0, a2[0].cuda(), b2[0].cuda(), 2.0)
            a[0], b[0], sc[0] = a2[0], b2[0], 2.0
        graph.replay()
        torch.cuda.synchronize()
        check(x, base, ids, a, b, sc, out, 32)
    h.close()


def test_two_streams_and_two_graphs_at_once(P):
    """Nothing of a call is kept in the handle: calls may overlap."""
    n = 700
    h, a, b, sc = make(P, 512, 512, [16, 48, 5], n)
    sets = []
    for k in range(2):
        x, base = data(n, 512, 512, BF, F, seed=20 + k)
        ids = torch.randint(-1, 3, (n,), generator=rng(30 + k)).to(torch.int32).cuda()
        sets.append((x, base, ids, h.apply(x, base, ids)))
    streams = [torch.cuda.Stream() for _ in sets]
    graphs, outs = [], []
    for s, (x, base, ids, _) in zip(streams, sets):
        s.wait_stream(torch.cuda.current_stream())
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(base)
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                h.apply(x, base, ids, out=out)
        graphs.append(g), outs.append(out)
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    for s, (x, base, ids, _), out in zip(streams, sets, outs):
        with torch.cuda.stream(s):
            for _ in range(20):
                h.apply(x, base, ids, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[3]) for o, want in zip(outs, sets))
    h.close()


def test_refusals(P):
    h, *_ = make(P, 64, 64, [4], 16)
    x, base = data(4, 64, 64, BF, BF)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(x=x[:, :56]), dict(x=x.half()), dict(x=x.cpu()), dict(x=x.T.contiguous().T), dict(ids=ids.long()),
                dict(ids=ids[:3]), dict(base=base[:3]), dict(out=base.float()), dict(out=x), dict(x=x[:0], base=base[:0], ids=ids[:0])):
        with pytest.raises(ValueError):
            h.apply(**{**dict(x=x, base=base, ids=ids), **bad})
    wide = torch.zeros(4, 100, dtype=BF, device="cuda")
    for off in (wide[:, 4:68], wide[:, 1:65]):  # rows or strides off a 16-byte boundary
        with pytest.raises(P.MoeError) as e:
            h.apply(off, base, ids)
        assert e.value.status == P.MOE_ERR_INVALID_ARGUMENT and "16" in str(e.value)
    both = torch.zeros(4, 128, dtype=BF, device="cuda")  # out is base with other rows than base's
    assert P.lib().moe_adapters_apply(h.h, x.data_ptr(), P.MOE_BF16, 64, both.data_ptr(), 64, both.data_ptr(), 128, P.MOE_BF16,
                                      ids.data_ptr(), 4, None) == P.MOE_ERR_INVALID_ARGUMENT
    many, mbase = data(17, 64, 64, BF, BF)
    with pytest.raises(P.MoeError):
        h.apply(many, mbase, torch.zeros(17, dtype=torch.int32, device="cuda"))
    g = torch.zeros(5, 64, dtype=BF)
    for slot, a, b in ((1, g[:4], g[:4].T.contiguous()), (-1, g[:4], g[:4].T.contiguous()), (0, g, g.T.contiguous())):
        with pytest.raises(P.MoeError):
            h.load(slot, a, b)
    with pytest.raises(ValueError):
        h.load(0, g[:4], g[:4])
    for bad in (dict(d_in=12), dict(d_out=0), dict(max_rank=129), dict(max_rank=0), dict(max_adapters=0), dict(max_tokens=0),
                dict(max_tokens=8193), dict(device=999)):
        with pytest.raises(P.MoeError) as e:
            P.Adapters(**{**dict(d_in=64, d_out=64, max_adapters=1, max_rank=4, max_tokens=8), **bad})
        assert e.value.status == P.MOE_ERR_INVALID_ARGUMENT
    assert h.device_bytes() > 0
    h.close()
