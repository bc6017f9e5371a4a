"""Torch wrappers of the block operators (include/moe.h): the norms before and after a block, low-rank
adapters of many requests, and the dense gated feed-forward block.

Argument checks and marshalling only.  Tensors are CUDA tensors of one device, matrices 2-D with unit
stride in their last dimension (rows may be strided); the work goes to that device's current stream.
Bad tensors raise ``ValueError``, a status other than ok raises ``MoeError``.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

import expert_ffn_gemv_b200 as P

TYPES = {P.MOE_F32: torch.float32, P.MOE_BF16: torch.bfloat16}
CODES = {v: k for k, v in TYPES.items()}
_ACTS = {"linear": P.MOE_GATE_LINEAR, "sigmoid": P.MOE_GATE_SIGMOID}
_lib = P.lib()


def _bad(name, what):
    raise ValueError(f"{name}: {what}")


def matrix(t, name, dev, shape, dtype=None, dense=False):
    """Checks a 2-D tensor (None in `shape`: any size, but not 0) and returns its row stride."""
    if t.dim() != 2 or (shape[0] is not None and t.shape[0] != shape[0]) or (shape[1] is not None and t.shape[1] != shape[1]):
        _bad(name, f"shape {tuple(t.shape)}, expected {shape}")
    if t.numel() == 0:
        _bad(name, "is empty")
    if t.device != dev or dev.type != "cuda":
        _bad(name, f"on {t.device}, expected a CUDA tensor on {dev}")
    if t.dtype not in CODES if dtype is None else t.dtype != dtype:
        _bad(name, f"dtype {t.dtype}" + (f", expected {dtype}" if dtype else " is not float32 or bfloat16"))
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if (t.stride(1) != 1 and cols > 1) or ld < cols or (dense and ld != cols):
        _bad(name, f"strides {t.stride()}" + (": must be contiguous" if dense else ": rows must be contiguous"))
    return ld


def vector(t, name, dev, n, dtype=None):
    if t.dim() != 1 or t.shape[0] != n:
        _bad(name, f"shape {tuple(t.shape)}, expected ({n},)")
    if t.device != dev:
        _bad(name, f"on {t.device}, expected {dev}")
    if t.dtype not in CODES if dtype is None else t.dtype != dtype:
        _bad(name, f"dtype {t.dtype}")
    if t.stride(0) != 1 and n > 1:
        _bad(name, "must be contiguous")


def _run(dev, what, call):
    """Runs call(stream) with the tensors' device current."""
    if torch.cuda.current_device() == dev.index:
        st = call(torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = call(torch.cuda.current_stream().cuda_stream)
    if st != P.MOE_OK:
        raise P.MoeError(st, what)


def _overlap(a, b):
    """Whether two tensors share memory (by the address ranges they span)."""
    def span(t):
        lo = t.data_ptr()
        return lo, lo + (sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _no_overlap(out, name, inputs, may=()):
    """An output may share memory with the tensors in `may` (as a whole: same start, strides and type)
    and with no other of `inputs`."""
    for t in inputs:
        if t is None or not _overlap(out, t):
            continue
        if any(t is m for m in may) and (out.data_ptr(), out.stride(), out.dtype) == (t.data_ptr(), t.stride(), t.dtype):
            continue
        _bad(name, "overlaps another tensor of the call")


# ------------------------------------------------------------------------------------------ norms
def norm_in(x, weight, *, eps=1e-6, unit_offset=False, out=None, out_dtype=None):
    """Norm before a block (``moe_norm_in``): x / sqrt(mean(x^2) + eps) * (weight + unit_offset).

    x [n, d]; weight [d]; the result has x's type unless `out` or `out_dtype` says otherwise.  `out` may
    be x."""
    dev = x.device
    ld = matrix(x, "x", dev, (None, None))
    n, d = x.shape
    vector(weight, "weight", dev, d)
    if out is None:
        out = torch.empty((n, d), dtype=out_dtype or x.dtype, device=dev)
        old = d
        if out.dtype not in CODES:
            _bad("out_dtype", f"{out.dtype}")
    else:
        old = matrix(out, "out", dev, (n, d), out_dtype)
        _no_overlap(out, "out", (x, weight), may=(x,))
    _run(dev, "moe_norm_in", lambda st: _lib.moe_norm_in(
        x.data_ptr(), CODES[x.dtype], ld, weight.data_ptr(), CODES[weight.dtype], eps, int(unit_offset), out.data_ptr(),
        CODES[out.dtype], old, n, d, st))
    return out


def _gate(gate, name, dev, n, d):
    """(kind, dtype code, pointer, row stride) of a gate: None, [d], [n, 1] or [n, d]."""
    if gate is None:
        return P.MOE_GATE_NONE, 0, None, 0
    if gate.dim() == 1:
        vector(gate, name, dev, d)
        return P.MOE_GATE_CHANNEL, CODES[gate.dtype], gate.data_ptr(), 0
    if gate.dim() == 2 and gate.shape[1] == 1:
        ld = matrix(gate, name, dev, (n, 1))
        return P.MOE_GATE_TOKEN, CODES[gate.dtype], gate.data_ptr(), ld
    ld = matrix(gate, name, dev, (n, d))
    return P.MOE_GATE_FULL, CODES[gate.dtype], gate.data_ptr(), ld


def _act(gate_act):
    if gate_act not in _ACTS:
        raise ValueError(f"gate_act: {gate_act!r}, expected one of {sorted(_ACTS)}")
    return _ACTS[gate_act]


def norm_out(o, residual, *, weight=None, eps=1e-6, unit_offset=False, gate=None, gate_act="linear", scale=1.0,
             next_weight=None, next_eps=1e-6, next_dtype=None, out=None, out_dtype=None, next_out=None):
    """Norm after a block, gate, residual (``moe_norm_out``):

        res = residual + scale * act(gate) * (o / sqrt(mean(o^2) + eps) * (weight + unit_offset))

    o, residual [n, d]; weight [d] or None (no norm); gate None, [d], [n, 1] or [n, d].  Returns res (the
    residual's type, `out_dtype` or `out`, which may be o or residual).  With `next_weight` the next
    block's input norm is taken in the same pass and (res, h) is returned, h = norm_in(res, next_weight)
    in `next_dtype` (default: o's type) or in `next_out`, which may be o; both weights have one type."""
    dev = o.device
    o_ld = matrix(o, "o", dev, (None, None))
    n, d = o.shape
    r_ld = matrix(residual, "residual", dev, (n, d))
    wt = None
    for w, name in ((weight, "weight"), (next_weight, "next_weight")):
        if w is not None:
            vector(w, name, dev, d, wt)
            wt = w.dtype
    kind, g_code, g_ptr, g_ld = _gate(gate, "gate", dev, n, d)
    ins = (o, residual, weight, gate, next_weight)
    if out is None:
        out, out_ld = torch.empty((n, d), dtype=out_dtype or residual.dtype, device=dev), d
        if out.dtype not in CODES:
            _bad("out_dtype", f"{out.dtype}")
    else:
        out_ld = matrix(out, "out", dev, (n, d), out_dtype)
        _no_overlap(out, "out", ins, may=(o, residual))
    h, h_ld, h_code, h_ptr, nw_ptr = None, 0, 0, None, None
    if next_weight is not None:
        if next_out is None:
            h, h_ld = torch.empty((n, d), dtype=next_dtype or o.dtype, device=dev), d
            if h.dtype not in CODES:
                _bad("next_dtype", f"{h.dtype}")
        else:
            h = next_out
            h_ld = matrix(h, "next_out", dev, (n, d), next_dtype)
            _no_overlap(h, "next_out", ins + (out,), may=(o,))
        h_code, h_ptr, nw_ptr = CODES[h.dtype], h.data_ptr(), next_weight.data_ptr()
    elif next_out is not None:
        _bad("next_out", "given without next_weight")
    a = P.moe_norm_out_args(
        n, d, CODES[o.dtype], CODES[residual.dtype], CODES[out.dtype], CODES[wt] if wt else 0, g_code, h_code, kind,
        _act(gate_act), int(unit_offset), eps, next_eps, scale, o.data_ptr(), residual.data_ptr(),
        None if weight is None else weight.data_ptr(), g_ptr, out.data_ptr(), nw_ptr, h_ptr, o_ld, r_ld, g_ld, out_ld, h_ld)
    _run(dev, "moe_norm_out", lambda st: _lib.moe_norm_out(C.byref(a), st))
    return out if h is None else (out, h)


def _norm_ws(dev, n, d):
    if torch.cuda.current_device() == dev.index:
        nbytes = _lib.moe_norm_workspace(n, d)
    else:
        with torch.cuda.device(dev):
            nbytes = _lib.moe_norm_workspace(n, d)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


def norm_in_backward(x, weight, dh, *, eps=1e-6, unit_offset=False, d_residual=None):
    """Gradients of ``norm_in``: (dx, dweight) from dh; d_residual (or None) is added to dx and gives it
    its type (else x's)."""
    dev = x.device
    x_ld = matrix(x, "x", dev, (None, None))
    n, d = x.shape
    vector(weight, "weight", dev, d)
    dh_ld = matrix(dh, "dh", dev, (n, d))
    r_ld, r_code, r_ptr = 0, 0, None
    if d_residual is not None:
        r_ld = matrix(d_residual, "d_residual", dev, (n, d))
        r_code, r_ptr = CODES[d_residual.dtype], d_residual.data_ptr()
    dx = torch.empty((n, d), dtype=x.dtype if d_residual is None else d_residual.dtype, device=dev)
    dw = torch.empty_like(weight)
    ws = _norm_ws(dev, n, d)
    a = P.moe_norm_in_bwd_args(n, d, CODES[x.dtype], CODES[weight.dtype], CODES[dh.dtype], r_code, CODES[dx.dtype],
                               int(unit_offset), eps, x.data_ptr(), weight.data_ptr(), dh.data_ptr(), r_ptr,
                               dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel(), x_ld, dh_ld, r_ld, d)
    _run(dev, "moe_norm_in_backward", lambda st: _lib.moe_norm_in_backward(C.byref(a), st))
    return dx, dw


def norm_out_backward(o, d_res, *, weight=None, eps=1e-6, unit_offset=False, gate=None, gate_act="linear", scale=1.0):
    """Gradients of ``norm_out`` from d_res, the gradient of its result (which is the residual's gradient
    too): (d_o, dweight, dgate), None for what was None; each in its tensor's type and shape."""
    dev = o.device
    o_ld = matrix(o, "o", dev, (None, None))
    n, d = o.shape
    r_ld = matrix(d_res, "d_res", dev, (n, d))
    if weight is not None:
        vector(weight, "weight", dev, d)
    kind, g_code, g_ptr, g_ld = _gate(gate, "gate", dev, n, d)
    d_o = torch.empty((n, d), dtype=o.dtype, device=dev)
    dw = None if weight is None else torch.empty_like(weight)
    dg = None if gate is None else torch.empty(gate.shape, dtype=gate.dtype, device=dev)
    ws = _norm_ws(dev, n, d)
    a = P.moe_norm_out_bwd_args(
        n, d, CODES[o.dtype], 0 if weight is None else CODES[weight.dtype], g_code, CODES[d_res.dtype], kind,
        _act(gate_act), int(unit_offset), eps, scale, o.data_ptr(), None if weight is None else weight.data_ptr(), g_ptr,
        d_res.data_ptr(), d_o.data_ptr(), None if dw is None else dw.data_ptr(), None if dg is None else dg.data_ptr(),
        ws.data_ptr(), ws.numel(), o_ld, g_ld, r_ld, d, 0 if dg is None else dg.shape[-1])
    _run(dev, "moe_norm_out_backward", lambda st: _lib.moe_norm_out_backward(C.byref(a), st))
    return d_o, dw, dg


# --------------------------------------------------------------------------------------- adapters
class Adapters:
    """Low-rank adapters of many requests beside a shared projection or block (``moe_adapters_*``):
    out_t = base_t + scale_i B_i (A_i x_t), i = ids[t]; -1: no adapter.  One handle serves one stream at
    a time."""

    def __init__(self, *, d_in, d_out, max_adapters, max_rank, max_tokens=8, device=0):
        self.h = None
        self.device = torch.device("cuda", device)
        self.d_in, self.d_out, self.max_adapters, self.max_rank = d_in, d_out, max_adapters, max_rank
        h = C.c_void_p()
        st = _lib.moe_adapters_create(C.byref(P.moe_adapters_config(d_in, d_out, max_adapters, max_rank, max_tokens, device)),
                                      C.byref(h))
        if st != P.MOE_OK:
            raise P.MoeError(st, "moe_adapters_create")
        self.h = h

    def _check(self, st, what):
        if st != P.MOE_OK:
            raise P.MoeError(st, f"{what}: {_lib.moe_adapters_last_error(self.h).decode()}")

    def load(self, slot, a, b, scale=1.0):
        """Puts an adapter into `slot`: a [rank, d_in], b [d_out, rank], bf16, contiguous, on the handle's
        device or in host memory; a = b = None empties the slot."""
        rank = 0
        if a is not None or b is not None:
            rank = a.shape[0] if a.dim() == 2 else -1
            for t, name, shape in ((a, "a", (rank, self.d_in)), (b, "b", (self.d_out, rank))):
                if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
                    _bad(name, f"{t.dtype} {tuple(t.shape)}, expected contiguous bfloat16 {shape}")
                if t.device.type != "cpu" and t.device != self.device:
                    _bad(name, f"on {t.device}, expected {self.device} or the host")
        with torch.cuda.device(self.device):
            self._check(_lib.moe_adapters_load(self.h, slot, P._ptr(a), P._ptr(b), rank, scale,
                                               torch.cuda.current_stream().cuda_stream), "moe_adapters_load")

    def apply(self, x, base, ids, out=None):
        """x [n, d_in]; base [n, d_out]; ids int32 [n]; returns out (base's type; may be base itself)."""
        dev = self.device
        x_ld = matrix(x, "x", dev, (None, self.d_in))
        n = x.shape[0]
        b_ld = matrix(base, "base", dev, (n, self.d_out))
        vector(ids, "ids", dev, n, torch.int32)
        if out is None:
            out, o_ld = torch.empty((n, self.d_out), dtype=base.dtype, device=dev), self.d_out
        else:
            o_ld = matrix(out, "out", dev, (n, self.d_out), base.dtype)
            _no_overlap(out, "out", (x, base, ids), may=(base,))
        st = _lib.moe_adapters_apply(self.h, x.data_ptr(), CODES[x.dtype], x_ld, base.data_ptr(), b_ld, out.data_ptr(), o_ld,
                                     CODES[out.dtype], ids.data_ptr(), n, torch.cuda.current_stream(dev).cuda_stream)
        if st != P.MOE_OK:
            self._check(st, "moe_adapters_apply")
        return out

    def check(self) -> int:
        return _lib.moe_adapters_check(self.h)

    def device_bytes(self) -> int:
        return _lib.moe_adapters_device_bytes(self.h)

    def close(self):
        if getattr(self, "h", None):
            _lib.moe_adapters_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------------------------ dense block
def _ffn_weights(x, w_gate, w_up, w_down):
    dev = x.device
    bf16 = torch.bfloat16
    ld = matrix(x, "x", dev, (None, None), bf16)
    n, d = x.shape
    matrix(w_gate, "w_gate", dev, (None, d), bf16, dense=True)
    f = w_gate.shape[0]
    matrix(w_up, "w_up", dev, (f, d), bf16, dense=True)
    matrix(w_down, "w_down", dev, (d, f), bf16, dense=True)
    return dev, n, d, f, ld


def _ffn_ws(dev, n, d, f, backward):
    nbytes = _lib.moe_ffn_workspace(n, d, f, backward)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev), nbytes


def ffn_forward(x, w_gate, w_up, w_down, *, add=None, out=None, out_dtype=None, save=False):
    """Dense gated block (``moe_ffn_forward``): w_down (silu(w_gate x) * (w_up x)) (+ add).

    x [n, d] bf16; w_gate, w_up [f, d], w_down [d, f] bf16.  The result is bf16, `out_dtype` or `out` (which
    may be `add`).  With save=True returns (y, saved) for ``ffn_backward``."""
    dev, n, d, f, x_ld = _ffn_weights(x, w_gate, w_up, w_down)
    a_ld, a_code, a_ptr = 0, 0, None
    if add is not None:
        a_ld = matrix(add, "add", dev, (n, d))
        a_code, a_ptr = CODES[add.dtype], add.data_ptr()
    if out is None:
        out, y_ld = torch.empty((n, d), dtype=out_dtype or torch.bfloat16, device=dev), d
        if out.dtype not in CODES:
            _bad("out_dtype", f"{out.dtype}")
    else:
        y_ld = matrix(out, "out", dev, (n, d), out_dtype)
        _no_overlap(out, "out", (x, w_gate, w_up, w_down, add), may=(add,))
    saved = tuple(torch.empty((n, f), dtype=torch.float32, device=dev) if save else None for _ in range(2))
    ws, nbytes = _ffn_ws(dev, n, d, f, 0)
    a = P.moe_ffn_args(n, d, f, a_code, CODES[out.dtype], x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                       w_down.data_ptr(), a_ptr, out.data_ptr(), P._ptr(saved[0]), P._ptr(saved[1]), ws.data_ptr(),
                       nbytes, x_ld, a_ld, y_ld)
    _run(dev, "moe_ffn_forward", lambda st: _lib.moe_ffn_forward(C.byref(a), st))
    return (out, saved) if save else out


def ffn_backward(dy, x, w_gate, w_up, w_down, saved, *, need_dx=True, need_dw=True):
    """Gradients of ``ffn_forward`` (``moe_ffn_backward``): (dx, dw_gate, dw_up, dw_down) in bf16 from dy
    [n, d] bf16 and what the forward saved; None where not needed."""
    dev, n, d, f, x_ld = _ffn_weights(x, w_gate, w_up, w_down)
    dy_ld = matrix(dy, "dy", dev, (n, d), torch.bfloat16)
    for t, name in zip(saved, ("saved gate", "saved up")):
        matrix(t, name, dev, (n, f), torch.float32, dense=True)
    if not need_dx and not need_dw:
        raise ValueError("nothing to compute")
    dx = torch.empty((n, d), dtype=torch.bfloat16, device=dev) if need_dx else None
    dw = [torch.empty_like(w) if need_dw else None for w in (w_gate, w_up, w_down)]
    ws, nbytes = _ffn_ws(dev, n, d, f, 1)
    a = P.moe_ffn_bwd_args(n, d, f, dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                           saved[0].data_ptr(), saved[1].data_ptr(), P._ptr(dx), *[P._ptr(w) for w in dw], ws.data_ptr(),
                           nbytes, dy_ld, x_ld, d)
    _run(dev, "moe_ffn_backward", lambda st: _lib.moe_ffn_backward(C.byref(a), st))
    return (dx, *dw)


def ffn_check() -> int:
    """Waits for the current device; MOE_ERR_TIMEOUT if a wait of the dense block's kernels ran out."""
    return _lib.moe_ffn_check()


# -------------------------------------------------------------------------------------- one block
@dataclass
class Block:
    """What stands around and beside one layer's routed experts (``moe_block``), for
    ``MoE.forward_blocks``: the norms' weights [d], a gate [d], the residual scale, the dense block's
    weights (w_gate, w_up, w_down), and adapters."""
    norm_in: torch.Tensor
    norm_out: torch.Tensor | None = None
    gate: torch.Tensor | None = None
    gate_act: str = "linear"
    scale: float = 1.0
    eps: float = 1e-6
    unit_offset: bool = False
    ffn: tuple | None = None
    adapters: Adapters | None = None

    def args(self, d, dev):
        t = self.norm_in.dtype
        for v, name in ((self.norm_in, "norm_in"), (self.norm_out, "norm_out"), (self.gate, "gate")):
            if v is not None:
                vector(v, name, dev, d, t if t in CODES else None)
        f = 0
        if self.ffn is not None:
            wg, wu, wd = self.ffn
            matrix(wg, "ffn gate", dev, (None, d), torch.bfloat16, dense=True)
            f = wg.shape[0]
            matrix(wu, "ffn up", dev, (f, d), torch.bfloat16, dense=True)
            matrix(wd, "ffn down", dev, (d, f), torch.bfloat16, dense=True)
        if self.adapters is not None and (self.adapters.d_in != d or self.adapters.d_out != d or self.adapters.device != dev):
            _bad("adapters", f"d_in and d_out must be {d}, on {dev}")
        if t not in CODES:
            _bad("norm_in", f"dtype {t}")
        if self.adapters is not None and self.adapters.h is None:
            _bad("adapters", "closed")
        ffn = self.ffn or (None, None, None)
        return P.moe_block(CODES[t], self.norm_in.data_ptr(), P._ptr(self.norm_out), P._ptr(self.gate), self.eps,
                           self.eps, self.scale, _act(self.gate_act), int(self.unit_offset), f, *[P._ptr(w) for w in ffn],
                           None if self.adapters is None else self.adapters.h)
