"""What the block operators refuse before anything is launched (no GPU needed): the C calls return
MOE_ERR_INVALID_ARGUMENT or MOE_ERR_UNSUPPORTED, the wrappers raise ValueError.  And the 64-bit
gradients that the GPU tests compare with, against differences."""
import ctypes as C

import pytest
import torch

import block_reference as R


@pytest.fixture(scope="module")
def P():
    from expert_ffn_gemv_b200 import build

    build.build()
    import expert_ffn_gemv_b200 as P

    return P


BAD, UNSUP = 1, 5


def norm_out_args(P, **kw):
    a = P.moe_norm_out_args(n_tokens=2, d_model=64, o=64, residual=64, res_out=64, o_stride=64, res_stride=64, res_out_stride=64,
                            eps=1e-6, next_eps=1e-6, scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(struct_size=8), BAD), (dict(n_tokens=0), BAD), (dict(d_model=0), BAD), (dict(o=None), BAD), (dict(residual=None), BAD),
    (dict(res_out=None), BAD), (dict(o_dtype=2), BAD), (dict(o_stride=63), BAD), (dict(res_stride=0), BAD), (dict(o=66), BAD),
    (dict(weight=64, eps=-1.0), BAD), (dict(weight=64, eps=float("nan")), BAD), (dict(weight=62), BAD), (dict(weight=64, w_dtype=7), BAD),
    (dict(h=64, h_stride=64), BAD), (dict(next_weight=64), BAD), (dict(gate_kind=1), BAD), (dict(gate=64), BAD),
    (dict(gate=64, gate_kind=4), BAD), (dict(gate=64, gate_kind=3, gate_stride=63), BAD), (dict(gate=64, gate_kind=2, gate_act=2), BAD),
    (dict(gate=64, gate_kind=2), BAD), (dict(unit_offset=2), BAD),
    (dict(d_model=8193, o_stride=8193, res_stride=8193, res_out_stride=8193), UNSUP)])
def test_norm_out(P, bad, status):
    assert P.lib().moe_norm_out(C.byref(norm_out_args(P, **bad)), None) == status


def test_norm_out_null(P):
    assert P.lib().moe_norm_out(None, None) == BAD


@pytest.mark.parametrize("i,v,status", [(0, None, BAD), (1, 3, BAD), (2, 63, BAD), (3, None, BAD), (5, -1.0, BAD), (6, 3, BAD),
                                        (7, None, BAD), (9, 1, BAD), (10, 0, BAD), (11, 0, BAD), (11, 9000, BAD)])
def test_norm_in(P, i, v, status):
    a = [64, 0, 64, 64, 0, 1e-6, 0, 64, 0, 64, 2, 64, None]
    a[i] = v
    assert P.lib().moe_norm_in(*a) == status
    assert P.lib().moe_norm_in(64, 0, 9000, 64, 0, 1e-6, 0, 64, 0, 9000, 2, 9000, None) == UNSUP


@pytest.mark.parametrize("bad", [dict(struct_size=0), dict(n_tokens=0), dict(x=None), dict(weight=None), dict(dh=None), dict(dx=None),
                                 dict(x_stride=63), dict(dres=64), dict(eps=-1.0), dict(dx_dtype=5), dict(unit_offset=-1)])
def test_norm_in_backward(P, bad):
    a = P.moe_norm_in_bwd_args(n_tokens=2, d_model=64, x=64, weight=64, dh=64, dx=64, x_stride=64, dh_stride=64, dx_stride=64)
    for k, v in bad.items():
        setattr(a, k, v)
    assert P.lib().moe_norm_in_backward(C.byref(a), None) == BAD


@pytest.mark.parametrize("bad", [dict(struct_size=0), dict(n_tokens=0), dict(o=None), dict(dres=None), dict(d_o=None), dict(dweight=64),
                                 dict(dgate=64), dict(gate=64), dict(gate=64, gate_kind=3, gate_stride=64, dgate=64, dgate_stride=3)])
def test_norm_out_backward(P, bad):
    a = P.moe_norm_out_bwd_args(n_tokens=2, d_model=64, o=64, dres=64, d_o=64, o_stride=64, dres_stride=64, do_stride=64)
    for k, v in bad.items():
        setattr(a, k, v)
    assert P.lib().moe_norm_out_backward(C.byref(a), None) == BAD


FFN = dict(n_tokens=2, d_model=64, d_ff=32, x=64, w_gate=64, w_up=64, w_down=64, y=64, workspace=64, workspace_bytes=1 << 20,
           x_stride=64, y_stride=64)


@pytest.mark.parametrize("bad", [dict(struct_size=4), dict(n_tokens=0), dict(n_tokens=(1 << 20) + 1), dict(d_model=60), dict(d_ff=12), dict(d_ff=0),
                                 dict(d_model=65544), dict(x=None), dict(x=72), dict(w_gate=None), dict(w_up=None), dict(w_down=66),
                                 dict(y=None), dict(y_dtype=3), dict(x_stride=68), dict(x_stride=56), dict(add=64, add_stride=60),
                                 dict(add=64, add_stride=64, add_dtype=9), dict(save_gate=64), dict(workspace=None),
                                 dict(workspace_bytes=100), dict(workspace=40)])
def test_ffn_forward(P, bad):
    a = P.moe_ffn_args(**FFN)
    for k, v in bad.items():
        setattr(a, k, v)
    assert P.lib().moe_ffn_forward(C.byref(a), None) == BAD


@pytest.mark.parametrize("bad", [dict(struct_size=4), dict(n_tokens=0), dict(dy=None), dict(x=8), dict(save_gate=None), dict(save_up=None),
                                 dict(dx=None, dw_gate=None, dw_up=None, dw_down=None), dict(dw_gate=None), dict(dw_down=72),
                                 dict(dx_stride=8), dict(dy_stride=66), dict(workspace_bytes=300)])
def test_ffn_backward(P, bad):
    a = P.moe_ffn_bwd_args(n_tokens=2, d_model=64, d_ff=32, dy=64, x=64, w_gate=64, w_up=64, w_down=64, save_gate=64, save_up=64,
                           dx=64, dw_gate=64, dw_up=64, dw_down=64, workspace=64, workspace_bytes=1 << 20, dy_stride=64, x_stride=64,
                           dx_stride=64)
    for k, v in bad.items():
        setattr(a, k, v)
    assert P.lib().moe_ffn_backward(C.byref(a), None) == BAD


def test_workspaces(P):
    L = P.lib()
    # h; h, dg, du
    assert L.moe_ffn_workspace(3, 64, 40, 0) == 256 and L.moe_ffn_workspace(3, 64, 40, 1) == 768
    # the pieces of a split product come on top: 64 tiles, 2 x 65,536 deep
    assert L.moe_ffn_workspace(8192, 64, 65536, 1) == 3 * 8192 * 65536 * 2
    assert L.moe_ffn_workspace(0, 64, 40, 0) == 0 and L.moe_ffn_workspace(3, 60, 40, 0) == 0
    assert L.moe_norm_workspace(0, 64) == 0 and L.moe_norm_workspace(4, 9000) == 0
    assert L.moe_blocks_workspace(None, None, 1, 1) == 0


def test_handles(P):
    L = P.lib()
    h = C.c_void_p()
    assert L.moe_adapters_create(None, C.byref(h)) == BAD and not h.value
    assert L.moe_adapters_create(C.byref(P.moe_adapters_config(64, 64, 1, 200, 8, 0)), C.byref(h)) == BAD
    assert L.moe_adapters_apply(None, 64, 0, 64, 64, 64, 64, 64, 0, 64, 1, None) == BAD
    assert L.moe_adapters_load(None, 0, None, None, 0, 1.0, None) == BAD and L.moe_adapters_check(None) == BAD
    assert L.moe_adapters_destroy(None) == 0 and L.moe_adapters_last_error(None) == b"no handle"
    assert L.moe_adapters_device_bytes(None) == 0
    assert L.moe_forward_blocks(None, 0, 1, None, None, None, 1, None, None, 0, None, None) == BAD


def test_wrappers_refuse_host_tensors(P):
    x, w = torch.zeros(2, 64), torch.zeros(64)
    m = torch.zeros(32, 64, dtype=torch.bfloat16)
    for call in (lambda: P.norm_in(x, w), lambda: P.norm_out(x, x, weight=w), lambda: P.norm_in_backward(x, w, x),
                 lambda: P.norm_out_backward(x, x), lambda: P.ffn_forward(m, m, m, m.T.contiguous())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        P.no_such_name


@pytest.mark.parametrize("gate", [None, (7,), (3, 1), (3, 7)])
@pytest.mark.parametrize("kind", ["linear", "sigmoid"])
def test_reference_norm_gradients(gate, kind):
    torch.manual_seed(0)
    o, res, w, wn = torch.randn(3, 7), torch.randn(3, 7), torch.randn(7), torch.randn(7)
    g = None if gate is None else torch.randn(gate)
    dres, dh = torch.randn(3, 7), torch.randn(3, 7)
    v = {"o": o, "w": w, "wn": wn, "res": res, **({} if g is None else {"g": g})}
    v = {k: t.double() for k, t in v.items()}

    def loss(v):
        out, _ = R.norm_out(v["o"], v["res"], v["w"], v.get("g"), kind, 0.7)
        return (out * dres.double()).sum() + (R.norm_in(out, v["wn"]) * dh.double()).sum()

    out, _ = R.norm_out(o, res, w, g, kind, 0.7)
    dr, dwn, _, _ = R.norm_in_backward(out, wn, dh, dres)
    d = R.norm_out_backward(o, dr, w, g, kind, 0.7)
    grads = {"o": d["d_o"][0], "w": d["d_w"][0], "wn": dwn, "res": dr, **({} if g is None else {"g": d["d_gate"][0]})}
    differences(loss, v, grads)


def test_reference_ffn_gradients():
    torch.manual_seed(0)
    v = {"x": torch.randn(3, 8), "wg": torch.randn(5, 8), "wu": torch.randn(5, 8), "wd": torch.randn(8, 5)}
    v = {k: t.double() for k, t in v.items()}
    dy = torch.randn(3, 8).double()
    r = R.ffn(v["x"], v["wg"], v["wu"], v["wd"], dy)
    differences(lambda v: (R.ffn(v["x"], v["wg"], v["wu"], v["wd"])["y"] * dy).sum(), v,
                {"x": r["dx"], "wg": r["dwg"], "wu": r["dwu"], "wd": r["dwd"]})


def differences(loss, v, grads):
    """Central differences at e = 1e-5: e^2 and 1e-16 / e are both below 1e-9 of values of order 1..100."""
    e = 1e-5
    for k, g in grads.items():
        got = torch.empty_like(v[k]).reshape(-1)
        for i in range(v[k].numel()):
            up, down = dict(v), dict(v)
            up[k], down[k] = v[k].clone(), v[k].clone()
            up[k].reshape(-1)[i] += e
            down[k].reshape(-1)[i] -= e
            got[i] = (loss(up) - loss(down)) / (2 * e)
        assert torch.allclose(got.reshape(v[k].shape), g, rtol=1e-7, atol=1e-7), k


def test_wrappers_refuse_tensors_that_require_grad(P):
    """Nothing is recorded for autograd: without a word a graph through them would train nothing.  (Host tensors:
    under no_grad the same calls get as far as their device.)"""
    from expert_ffn_gemv_b200 import block

    def x(grad):
        return torch.zeros(2, 64, requires_grad=grad)

    def w(grad):
        return torch.zeros(64, requires_grad=grad)

    def m(grad):
        return torch.zeros(64, 64, dtype=torch.bfloat16, requires_grad=grad)

    calls = {
        "x": [lambda g: P.norm_in(x(g), w(False)), lambda g: P.norm_in_backward(x(g), w(False), x(False)), lambda g: P.ffn_forward(m(g), m(False), m(False), m(False))],
        "weight": [lambda g: P.norm_in(x(False), w(g))],
        "o": [lambda g: P.norm_out(x(g), x(False)), lambda g: P.norm_out_backward(x(g), x(False))],
        "residual": [lambda g: P.norm_out(x(False), x(g))],
        "w_up": [lambda g: P.ffn_forward(m(False), m(False), m(g), m(False)), lambda g: P.ffn_backward(m(False), m(False), m(False), m(g), m(False), (m(False), m(False)))],
        "x_in": [lambda g: block.matrix(x(g), "x_in", torch.device("cuda", 0), (None, 64))],
        "norm_in": [lambda g: block.vector(w(g), "norm_in", torch.device("cuda", 0), 64)],
    }
    for name, some in calls.items():
        for call in some:
            with pytest.raises(ValueError, match=f"^{name}: requires grad"):
                call(True)
            with torch.no_grad(), pytest.raises(ValueError, match="cuda|CUDA"):
                call(True)
            with pytest.raises(ValueError, match="cuda|CUDA"):
                call(False)


def test_ring_limit(P):
    """Copies are held back for four times as long: no longer than half a second."""
    for cycles in (200_000_001, 1 << 62, (1 << 64) - 1):
        assert P.moe_debug_set_ring_spin_limit(cycles) == BAD
    assert P.moe_debug_set_ring_spin_limit(200_000_000) == P.MOE_OK and P.moe_debug_set_ring_spin_limit(0) == P.MOE_OK


def test_outputs_in_an_inputs_place(P):
    """With another type or row stride than the input's, rows would be written before they are read.  (Pointers of
    their own everywhere else; d_model 9000 has the sound calls end as unsupported, before any launch.)"""
    L, d = P.lib(), 9000
    ld = dict(o_stride=d, res_stride=d, res_out_stride=d, h_stride=d)
    same = dict(n_tokens=2, d_model=d, o=1 << 20, residual=2 << 20, res_out=3 << 20, next_weight=4 << 20, h=5 << 20, eps=1e-6,
                next_eps=1e-6, scale=1.0, **ld)
    for kw, status in [(dict(), UNSUP), (dict(res_out=2 << 20), UNSUP), (dict(res_out=1 << 20), UNSUP), (dict(h=1 << 20), UNSUP),
                       (dict(res_out=2 << 20, res_out_dtype=1), BAD), (dict(res_out=2 << 20, res_dtype=1), BAD),
                       (dict(res_out=2 << 20, res_out_stride=d + 8), BAD), (dict(res_out=1 << 20, o_dtype=1), BAD),
                       (dict(h=1 << 20, h_dtype=1), BAD), (dict(h=1 << 20, h_stride=d + 1), BAD), (dict(h=3 << 20), BAD),
                       (dict(res_out=2 << 20, res_out_stride=d + 8, n_tokens=1), UNSUP)]:
        assert L.moe_norm_out(C.byref(P.moe_norm_out_args(**{**same, **kw})), None) == status, kw
    for x_dt, h_dt, h_ld, status in [(0, 0, d, UNSUP), (0, 1, d, BAD), (1, 0, d, BAD), (0, 0, d + 4, BAD)]:
        assert L.moe_norm_in(64, x_dt, d, 1 << 20, 0, 1e-6, 0, 64, h_dt, h_ld, 2, d, None) == status
    same = dict(n_tokens=2, d_model=d, x=64, weight=1 << 20, dh=2 << 20, dres=3 << 20, dx=3 << 20, x_stride=d, dh_stride=d,
                dres_stride=d, dx_stride=d)
    for kw, status in [(dict(), UNSUP), (dict(dx_dtype=1), BAD), (dict(dres_stride=d + 1), BAD), (dict(dx=4 << 20, dx_dtype=1), UNSUP)]:
        assert L.moe_norm_in_backward(C.byref(P.moe_norm_in_bwd_args(**{**same, **kw})), None) == status, kw
    for kw in (dict(add_dtype=1), dict(y_dtype=1), dict(add_stride=72)):
        a = P.moe_ffn_args(**{**FFN, **dict(add=1 << 20, y=1 << 20, add_stride=64), **kw})
        assert L.moe_ffn_forward(C.byref(a), None) == BAD, kw
