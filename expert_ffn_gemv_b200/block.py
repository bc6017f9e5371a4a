"""Torch wrappers of the block operators (include/moe.h): the norms before and after a block, low-rank
adapters of many requests, and the dense gated feed-forward block.

Argument checks and marshalling only.  Tensors are CUDA tensors of one device, matrices 2-D with unit
stride in their last dimension (rows may be strided); the work goes to that device's current stream.
Bad tensors raise ``ValueError``, a status other than ok raises ``MoeError``.  Nothing here is recorded for
autograd, so that tensors that require grad are refused outside ``torch.no_grad()``: the gradients of the norms
and the dense block come from the ``_backward`` functions, the adapters have none.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
from dataclasses import dataclass

import torch

import expert_ffn_gemv_b200 as P
from expert_ffn_gemv_b200 import build

TYPES = {P.MOE_F32: torch.float32, P.MOE_BF16: torch.bfloat16}
CODES = {v: k for k, v in TYPES.items()}
_ACTS = {"linear": P.MOE_GATE_LINEAR, "sigmoid": P.MOE_GATE_SIGMOID}
_lib = P.lib()


def _load_ext(path=build.EXT):
    """The binding (csrc/bind.cpp), bound to the loaded library; raises if it was not built, or not for the torch
    and Python that run."""
    if not path.exists():
        raise RuntimeError(f"{path} is missing: build it with `python -m expert_ffn_gemv_b200.build`")
    was, target = build.ext_built_for(path), build.ext_target()
    if was != target:
        raise RuntimeError(f"{path} was built for {was}, not for {target}: build it again with "
                           "`python -m expert_ffn_gemv_b200.build`")
    spec = importlib.util.spec_from_file_location("_block_ext", path)
    ext = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ext)
    ext.bind(P.MoeError, {n: C.cast(getattr(_lib, n), C.c_void_p).value for n in P.EXPORTED})
    return ext


_ext = _load_ext()


def _bad(name, what):
    raise ValueError(f"{name}: {what}")


def _code(dtype, name):
    """-1 for None"""
    if dtype is None:
        return -1
    if dtype not in CODES:
        _bad(name, f"{dtype} is not float32 or bfloat16")
    return CODES[dtype]


def _act(gate_act):
    if gate_act not in _ACTS:
        _bad("gate_act", f"{gate_act!r}, expected one of {sorted(_ACTS)}")
    return _ACTS[gate_act]


def _no_grad(t, name):
    if t.requires_grad and torch.is_grad_enabled():
        _bad(name, "requires grad, but the call leaves nothing for autograd: make it under torch.no_grad()")


def matrix(t, name, dev, shape, dtype=None, dense=False):
    """Checks a 2-D tensor (None in `shape`: any size, but not 0) and returns its row stride."""
    _no_grad(t, name)
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
    _no_grad(t, name)
    if t.dim() != 1 or t.shape[0] != n:
        _bad(name, f"shape {tuple(t.shape)}, expected ({n},)")
    if t.device != dev:
        _bad(name, f"on {t.device}, expected {dev}")
    if t.dtype not in CODES if dtype is None else t.dtype != dtype:
        _bad(name, f"dtype {t.dtype}")
    if t.stride(0) != 1 and n > 1:
        _bad(name, "must be contiguous")


# ------------------------------------------------------------------------------------------ norms
def norm_in(x, weight, *, eps=1e-6, unit_offset=False, out=None, out_dtype=None):
    """Norm before a block (``moe_norm_in``): x / sqrt(mean(x^2) + eps) * (weight + unit_offset).

    x [n, d]; weight [d]; the result has x's type unless `out` or `out_dtype` says otherwise.  `out` may
    be x."""
    return _ext.norm_in(x, weight, eps, unit_offset, out, _code(out_dtype, "out_dtype"))


def norm_out(o, residual, *, weight=None, eps=1e-6, unit_offset=False, gate=None, gate_act="linear", scale=1.0,
             next_weight=None, next_eps=1e-6, next_dtype=None, out=None, out_dtype=None, next_out=None):
    """Norm after a block, gate, residual (``moe_norm_out``):

        res = residual + scale * act(gate) * (o / sqrt(mean(o^2) + eps) * (weight + unit_offset))

    o, residual [n, d]; weight [d] or None (no norm); gate None, [d], [n, 1] or [n, d].  Returns res (the
    residual's type, `out_dtype` or `out`, which may be o or residual).  With `next_weight` the next
    block's input norm is taken in the same pass and (res, h) is returned, h = norm_in(res, next_weight)
    in `next_dtype` (default: o's type) or in `next_out`, which may be o; both weights have one type."""
    return _ext.norm_out(o, residual, weight, eps, unit_offset, gate, _act(gate_act), scale, next_weight, next_eps,
                         _code(next_dtype, "next_dtype"), out, _code(out_dtype, "out_dtype"), next_out)


def norm_in_backward(x, weight, dh, *, eps=1e-6, unit_offset=False, d_residual=None):
    """Gradients of ``norm_in``: (dx, dweight) from dh; d_residual (or None) is added to dx and gives it
    its type (else x's)."""
    return _ext.norm_in_backward(x, weight, dh, eps, unit_offset, d_residual)


def norm_out_backward(o, d_res, *, weight=None, eps=1e-6, unit_offset=False, gate=None, gate_act="linear", scale=1.0):
    """Gradients of ``norm_out`` from d_res, the gradient of its result (which is the residual's gradient
    too): (d_o, dweight, dgate), None for what was None; each in its tensor's type and shape."""
    return _ext.norm_out_backward(o, d_res, weight, eps, unit_offset, gate, _act(gate_act), scale)


# --------------------------------------------------------------------------------------- adapters
class Adapters:
    """Low-rank adapters of many requests beside a shared projection or block (``moe_adapters_*``):
    out_t = base_t + scale_i B_i (A_i x_t), i = ids[t]; -1: no adapter.  Calls of ``apply`` may run at once
    on several streams and in captured graphs."""

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
        if (a is None) != (b is None):
            _bad("a, b", "one is missing")
        if a is not None:
            rank = a.shape[0] if a.dim() == 2 else -1
            for t, name, shape in ((a, "a", (rank, self.d_in)), (b, "b", (self.d_out, rank))):
                if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
                    _bad(name, f"{t.dtype} {tuple(t.shape)}, expected contiguous bfloat16 {shape}")
                if t.device.type != "cpu" and t.device != self.device:
                    _bad(name, f"on {t.device}, expected {self.device} or the host")
        self._check(_lib.moe_adapters_load(self.h, slot, P._ptr(a), P._ptr(b), rank, scale,
                                           torch.cuda.current_stream(self.device).cuda_stream), "moe_adapters_load")

    def apply(self, x, base, ids, out=None):
        """x [n, d_in]; base [n, d_out]; ids int32 [n]; returns out (base's type; may be base itself)."""
        if self.h is None:
            _bad("adapters", "closed")
        return _ext.adapters_apply(self.h.value, self.device.index, self.d_in, self.d_out, x, base, ids, out)

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
def ffn_forward(x, w_gate, w_up, w_down, *, add=None, out=None, out_dtype=None, save=False):
    """Dense gated block (``moe_ffn_forward``): w_down (silu(w_gate x) * (w_up x)) (+ add).

    x [n, d] bf16; w_gate, w_up [f, d], w_down [d, f] bf16, contiguous.  The result is bf16, `out_dtype` or
    `out` (which may be `add`).  With save=True returns (y, saved) for ``ffn_backward``."""
    r = _ext.ffn_forward(x, w_gate, w_up, w_down, add, out, _code(out_dtype, "out_dtype"), save)
    return (r[0], r[1:]) if save else r


def ffn_backward(dy, x, w_gate, w_up, w_down, saved, *, need_dx=True, need_dw=True):
    """Gradients of ``ffn_forward`` (``moe_ffn_backward``): (dx, dw_gate, dw_up, dw_down) in bf16 from dy
    [n, d] bf16 and what the forward saved; None where not needed."""
    g, u = saved
    return _ext.ffn_backward(dy, x, w_gate, w_up, w_down, g, u, need_dx, need_dw)


def block_check() -> int:
    """Waits for the current device, all its streams; MOE_ERR_TIMEOUT if a wait of the norms' or the dense block's
    kernels ran out there (without it, the next call of one of them raises that)."""
    return _lib.moe_block_check()


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
