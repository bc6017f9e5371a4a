"""Python binding of the B200 routed-MoE FFN library (include/moe.h).

Argument marshalling only: every step of the computation runs in the CUDA kernels of
``_lib/libmoe_b200.so``.  The functions carry the C names (``moe_create``,
``moe_load_layer``, ``moe_forward``, ``moe_forward_stack``, ``moe_check``,
``moe_destroy``); ``MoE`` wraps them for torch tensors (device memory and the current
stream come from PyTorch).  Importing this package raises if the library has not been
built (``python -m expert_ffn_gemv_b200.build``): there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
from pathlib import Path

import os

# MOE_B200_LIB may point at another build of the same library (e.g. a tuning variant)
_LIB_PATH = Path(os.environ.get("MOE_B200_LIB") or Path(__file__).resolve().parent / "_lib" / "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARGUMENT = 1
MOE_ERR_OUT_OF_MEMORY = 2
MOE_ERR_CUDA = 3
MOE_ERR_NOT_LOADED = 4
MOE_ERR_UNSUPPORTED = 5
MOE_ERR_TIMEOUT = 6
MOE_ERR_DEVICE_FAULT = 7

MOE_FMT_Q2_32 = 0
MOE_FMT_CB35_32 = 1
MOE_FMT_NVFP4_16 = 2
MOE_F32 = 0
MOE_BF16 = 1
MOE_BIAS_LOGIT = 0
MOE_BIAS_SELECT = 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
MOE_GATE_LINEAR, MOE_GATE_SIGMOID = 0, 1

DECODE_MAX_TOKENS = 8


class moe_config(C.Structure):
    _fields_ = [
        ("struct_size", C.c_uint32), ("n_layers", C.c_int32), ("d_model", C.c_int32),
        ("d_ff", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
        ("n_shared", C.c_int32), ("shared_d_ff", C.c_int32), ("fmt", C.c_int32),
        ("act_dtype", C.c_int32), ("router_dtype", C.c_int32), ("out_dtype", C.c_int32),
        ("max_tokens", C.c_int32), ("codebook_grid", C.c_void_p), ("device", C.c_int32),
        ("bias_mode", C.c_int32), ("shared_gate", C.c_int32),
    ]


class moe_layer_weights(C.Structure):
    _fields_ = [("router_w", C.c_void_p), ("router_bias", C.c_void_p),
                ("expert_blocks", C.c_void_p), ("shared_blocks", C.c_void_p), ("shared_gate_w", C.c_void_p)]


class moe_route_out(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("expert_counts", C.c_void_p)]


def _struct(name, *groups):
    """A ctypes structure whose first field, struct_size, fills itself."""
    fields = [("struct_size", C.c_uint32)] + [(f, t) for t, names in groups for f in names.split()]

    def init(self, *a, **k):
        C.Structure.__init__(self, C.sizeof(type(self)), *a, **k)

    return type(name, (C.Structure,), {"_fields_": fields, "__init__": init})


moe_norm_out_args = _struct(
    "moe_norm_out_args",
    (C.c_int32, "n_tokens d_model o_dtype res_dtype res_out_dtype w_dtype gate_dtype h_dtype gate_kind gate_act unit_offset"),
    (C.c_float, "eps next_eps scale"),
    (C.c_void_p, "o residual weight gate res_out next_weight h"),
    (C.c_int64, "o_stride res_stride gate_stride res_out_stride h_stride"))
moe_norm_in_bwd_args = _struct(
    "moe_norm_in_bwd_args",
    (C.c_int32, "n_tokens d_model x_dtype w_dtype dh_dtype dres_dtype dx_dtype unit_offset"),
    (C.c_float, "eps"),
    (C.c_void_p, "x weight dh dres dx dweight workspace"),
    (C.c_uint64, "workspace_bytes"),
    (C.c_int64, "x_stride dh_stride dres_stride dx_stride"))
moe_norm_out_bwd_args = _struct(
    "moe_norm_out_bwd_args",
    (C.c_int32, "n_tokens d_model o_dtype w_dtype gate_dtype dres_dtype gate_kind gate_act unit_offset"),
    (C.c_float, "eps scale"),
    (C.c_void_p, "o weight gate dres d_o dweight dgate workspace"),
    (C.c_uint64, "workspace_bytes"),
    (C.c_int64, "o_stride gate_stride dres_stride do_stride dgate_stride"))
moe_adapters_config = _struct(
    "moe_adapters_config", (C.c_int32, "d_in d_out max_adapters max_rank max_tokens device"))
moe_ffn_args = _struct(
    "moe_ffn_args",
    (C.c_int32, "n_tokens d_model d_ff add_dtype y_dtype"),
    (C.c_void_p, "x w_gate w_up w_down add y save_gate save_up workspace"),
    (C.c_uint64, "workspace_bytes"),
    (C.c_int64, "x_stride add_stride y_stride"))
moe_ffn_bwd_args = _struct(
    "moe_ffn_bwd_args",
    (C.c_int32, "n_tokens d_model d_ff"),
    (C.c_void_p, "dy x w_gate w_up w_down save_gate save_up dx dw_gate dw_up dw_down workspace"),
    (C.c_uint64, "workspace_bytes"),
    (C.c_int64, "dy_stride x_stride dx_stride"))
moe_block = _struct(
    "moe_block",
    (C.c_int32, "norm_dtype"),
    (C.c_void_p, "norm_in_w norm_out_w gate"),
    (C.c_float, "norm_in_eps norm_out_eps scale"),
    (C.c_int32, "gate_act unit_offset ffn_d_ff"),
    (C.c_void_p, "ffn_gate ffn_up ffn_down adapters"))


EXPORTED = [
    "moe_create", "moe_load_layer", "moe_forward", "moe_forward_stack", "moe_check", "moe_destroy",
    "moe_status_string", "moe_last_error", "moe_device_bytes", "moe_debug_set_spin_limit",
    "moe_debug_set_alloc_cap", "moe_debug_set_ring_spin_limit", "moe_debug_wait_test", "moe_profile_enable", "moe_profile_read",
    "moe_route_noalloc",
    "moe_norm_in", "moe_norm_out", "moe_norm_workspace", "moe_norm_in_backward", "moe_norm_out_backward",
    "moe_adapters_create", "moe_adapters_load", "moe_adapters_apply", "moe_adapters_check", "moe_adapters_destroy",
    "moe_adapters_last_error", "moe_adapters_device_bytes",
    "moe_ffn_workspace", "moe_ffn_forward", "moe_ffn_backward", "moe_block_check",
    "moe_blocks_workspace", "moe_forward_blocks",
]

_lib = None


def library_path() -> Path:
    return _LIB_PATH


def lib() -> C.CDLL:
    """Load the CUDA library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not _LIB_PATH.exists():
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m expert_ffn_gemv_b200.build`")
        L = C.CDLL(str(_LIB_PATH))
        P, I, U64 = C.c_void_p, C.c_int32, C.c_uint64
        L.moe_create.argtypes = [C.POINTER(moe_config), C.POINTER(P)]
        L.moe_load_layer.argtypes = [P, I, C.POINTER(moe_layer_weights), P]
        L.moe_forward.argtypes = [P, I, P, P, I, P, C.POINTER(moe_route_out)]
        L.moe_forward_stack.argtypes = [P, I, I, P, P, I, P, C.POINTER(moe_route_out), P]
        L.moe_check.argtypes = [P]
        L.moe_destroy.argtypes = [P]
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = C.c_char_p
        L.moe_last_error.argtypes = [P]
        L.moe_last_error.restype = C.c_char_p
        L.moe_device_bytes.argtypes = [P]
        L.moe_device_bytes.restype = U64
        L.moe_debug_set_spin_limit.argtypes = [P, U64]
        L.moe_debug_set_alloc_cap.argtypes = [P, U64]
        L.moe_debug_set_ring_spin_limit.argtypes = [U64]
        L.moe_debug_wait_test.argtypes = [P, P]
        L.moe_profile_enable.argtypes = [P, I]
        L.moe_profile_read.argtypes = [P, I, C.POINTER(C.c_float), C.POINTER(I)]
        L.moe_route_noalloc.argtypes = [P, I, P, I, I, I, P, I, I, P, P, P]
        I64, F = C.c_int64, C.c_float
        L.moe_norm_in.argtypes = [P, I, I64, P, I, F, I, P, I, I64, I, I, P]
        for name in ("moe_norm_out", "moe_norm_in_backward", "moe_norm_out_backward", "moe_ffn_forward",
                     "moe_ffn_backward"):
            getattr(L, name).argtypes = [P, P]
        L.moe_norm_workspace.argtypes = [I, I]
        L.moe_norm_workspace.restype = U64
        L.moe_adapters_create.argtypes = [P, C.POINTER(P)]
        L.moe_adapters_load.argtypes = [P, I, P, P, I, F, P]
        L.moe_adapters_apply.argtypes = [P, P, I, I64, P, I64, P, I64, I, P, I, P]
        L.moe_adapters_check.argtypes = [P]
        L.moe_adapters_destroy.argtypes = [P]
        L.moe_adapters_last_error.argtypes = [P]
        L.moe_adapters_last_error.restype = C.c_char_p
        L.moe_adapters_device_bytes.argtypes = [P]
        L.moe_adapters_device_bytes.restype = U64
        L.moe_ffn_workspace.argtypes = [I, I, I, I]
        L.moe_ffn_workspace.restype = U64
        L.moe_block_check.argtypes = []
        L.moe_blocks_workspace.argtypes = [P, P, I, I]
        L.moe_blocks_workspace.restype = U64
        L.moe_forward_blocks.argtypes = [P, I, I, P, P, P, I, P, P, U64, P, C.POINTER(moe_route_out)]
        for name in ("moe_norm_in", "moe_norm_out", "moe_norm_in_backward", "moe_norm_out_backward",
                     "moe_adapters_create", "moe_adapters_load", "moe_adapters_apply", "moe_adapters_check",
                     "moe_adapters_destroy", "moe_ffn_forward", "moe_ffn_backward", "moe_block_check",
                     "moe_forward_blocks"):
            getattr(L, name).restype = I
        for name in ("moe_create", "moe_load_layer", "moe_forward", "moe_forward_stack", "moe_check",
                     "moe_destroy", "moe_debug_set_spin_limit", "moe_debug_set_alloc_cap",
                     "moe_debug_set_ring_spin_limit", "moe_debug_wait_test", "moe_profile_enable", "moe_profile_read", "moe_route_noalloc"):
            getattr(L, name).restype = I
        _lib = L
    return _lib


class MoeError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{lib().moe_status_string(status).decode()} ({status}): {detail}")


# ----------------------------------------------------------------------------------- C names
def moe_create(cfg: moe_config) -> C.c_void_p:
    h = C.c_void_p()
    st = lib().moe_create(C.byref(cfg), C.byref(h))
    if st != MOE_OK:
        raise MoeError(st, "moe_create")
    return h


def moe_load_layer(h, layer: int, w: moe_layer_weights, stream) -> int:
    return lib().moe_load_layer(h, layer, C.byref(w), stream)


def moe_forward(h, layer: int, x: int, y: int, n_tokens: int, stream, route: moe_route_out | None = None) -> int:
    return lib().moe_forward(h, layer, x, y, n_tokens, stream, None if route is None else C.byref(route))


def moe_forward_stack(h, first_layer: int, n_layers: int, x_in: int, x_out: int, n_tokens: int, stream,
                      per_layer_route=None, x_trace: int | None = None) -> int:
    return lib().moe_forward_stack(h, first_layer, n_layers, x_in, x_out, n_tokens, stream, per_layer_route,
                                   x_trace)


def moe_check(h) -> int:
    return lib().moe_check(h)


def moe_destroy(h) -> int:
    return lib().moe_destroy(h)


def moe_last_error(h) -> str:
    return lib().moe_last_error(h).decode()


def moe_device_bytes(h) -> int:
    return lib().moe_device_bytes(h)


def moe_debug_set_spin_limit(h, cycles: int) -> int:
    return lib().moe_debug_set_spin_limit(h, cycles)


def moe_debug_set_alloc_cap(h, nbytes: int) -> int:
    return lib().moe_debug_set_alloc_cap(h, nbytes)


def moe_debug_set_ring_spin_limit(cycles: int) -> int:
    return lib().moe_debug_set_ring_spin_limit(cycles)


def moe_debug_wait_test(h, stream) -> int:
    return lib().moe_debug_wait_test(h, stream)


def moe_profile_enable(h, on) -> int:
    """on: False/0 = off, True = all kernel classes, or a bit mask of classes."""
    mask = 0x7 if on is True else int(on)
    return lib().moe_profile_enable(h, mask)


def moe_profile_read(h, kind: int):
    """(status, total_ms, launches) of kernel class ``kind`` in the most recent call."""
    ms = C.c_float()
    n = C.c_int32()
    st = lib().moe_profile_read(h, kind, C.byref(ms), C.byref(n))
    return st, ms.value, n.value


PROF_ROUTE, PROF_GATEUP, PROF_DOWN = 0, 1, 2


def moe_route_noalloc(router_w: int, router_dtype: int, router_bias: int | None, n_experts: int, d_model: int,
                      top_k: int, x: int, x_dtype: int, n_tokens: int, topk_idx: int, topk_w: int, stream) -> int:
    """Handle-less routing that allocates no device memory (device pointers; see include/moe.h)."""
    return lib().moe_route_noalloc(router_w, router_dtype, router_bias, n_experts, d_model, top_k, x, x_dtype,
                                   n_tokens, topk_idx, topk_w, stream)


# ----------------------------------------------------------------------------------- torch wrapper
def _ptr(t) -> int | None:
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if hasattr(t, "ctypes"):  # numpy (host memory)
        return t.ctypes.data
    return int(t)


def _stream():
    import torch

    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


class MoE:
    """A handle with its configuration; methods take torch tensors (or numpy arrays for host data)."""

    def __init__(self, *, n_layers, d_model, d_ff, n_experts, top_k, n_shared=0, shared_d_ff=None,
                 fmt=MOE_FMT_Q2_32, act_dtype=MOE_BF16, router_dtype=MOE_BF16, out_dtype=MOE_F32,
                 max_tokens=8, codebook_grid=None, device=0, bias_mode=MOE_BIAS_LOGIT, shared_gate=0):
        self._grid = None
        if codebook_grid is not None:
            import numpy as np

            self._grid = np.ascontiguousarray(codebook_grid, dtype=np.int8).reshape(-1)
        self.cfg = moe_config(C.sizeof(moe_config), n_layers, d_model, d_ff, n_experts, top_k, n_shared,
                              shared_d_ff if shared_d_ff is not None else d_ff, fmt, act_dtype, router_dtype,
                              out_dtype, max_tokens,
                              None if self._grid is None else self._grid.ctypes.data, device, bias_mode,
                              int(shared_gate))
        self.h = moe_create(self.cfg)

    def _check(self, st: int, what: str):
        if st != MOE_OK:
            raise MoeError(st, f"{what}: {moe_last_error(self.h)}")

    def load_layer(self, layer, router_w, router_bias, expert_blocks, shared_blocks=None, shared_gate_w=None):
        w = moe_layer_weights(_ptr(router_w), _ptr(router_bias), _ptr(expert_blocks), _ptr(shared_blocks),
                              _ptr(shared_gate_w))
        self._keep = (router_w, router_bias, expert_blocks, shared_blocks, shared_gate_w)
        self._check(moe_load_layer(self.h, layer, w, _stream()), "moe_load_layer")

    def forward(self, layer, x, y, n_tokens=None, route=None):
        n = x.shape[0] if n_tokens is None else n_tokens
        r = None
        if route is not None:
            r = moe_route_out(*[_ptr(route.get(k)) for k in ("idx", "w", "counts")])
        self._check(moe_forward(self.h, layer, _ptr(x), _ptr(y), n, _stream(), r), "moe_forward")

    def forward_stack(self, first_layer, n_layers, x_in, x_out, n_tokens=None, routes=None, x_trace=None):
        n = x_in.shape[0] if n_tokens is None else n_tokens
        arr = None
        if routes is not None:
            arr = (moe_route_out * n_layers)(
                *[moe_route_out(*[_ptr(r.get(k)) for k in ("idx", "w", "counts")]) for r in routes])
        self._check(moe_forward_stack(self.h, first_layer, n_layers, _ptr(x_in), _ptr(x_out), n, _stream(), arr,
                                      _ptr(x_trace)), "moe_forward_stack")

    def forward_blocks(self, first_layer, blocks, x_in, x_out, adapter_ids=None, routes=None):
        """Layers first_layer .. with their norms, gates, dense blocks and adapters: one ``Block`` per layer
        (``moe_forward_blocks`` in include/moe.h).  The workspace of the dense blocks comes from PyTorch."""
        import torch

        from . import block as B

        dev = torch.device("cuda", self.cfg.device)
        n, nl, d = x_in.shape[0], len(blocks), self.cfg.d_model
        B.matrix(x_in, "x_in", dev, (None, d), dtype=B.TYPES[self.cfg.act_dtype], dense=True)
        B.matrix(x_out, "x_out", dev, (n, d), dtype=B.TYPES[self.cfg.out_dtype], dense=True)
        if adapter_ids is not None:
            B.vector(adapter_ids, "adapter_ids", dev, n, torch.int32)
        arr = (moe_block * nl)(*[b.args(d, dev) for b in blocks])
        nbytes = lib().moe_blocks_workspace(self.h, arr, nl, n)
        r = None
        if routes is not None:
            if len(routes) != nl:
                raise ValueError("routes: one entry per layer")
            r = (moe_route_out * nl)(*[moe_route_out(*[_ptr(q.get(k)) for k in ("idx", "w", "counts")]) for q in routes])
        with torch.cuda.device(dev):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
            self._check(lib().moe_forward_blocks(self.h, first_layer, nl, arr, x_in.data_ptr(), x_out.data_ptr(), n,
                                                 _ptr(adapter_ids), _ptr(ws), nbytes, _stream(), r),
                        "moe_forward_blocks")

    def check(self) -> int:
        return moe_check(self.h)

    def device_bytes(self) -> int:
        return moe_device_bytes(self.h)

    def close(self):
        if getattr(self, "h", None):
            moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# The block operators' wrappers (block.py) need torch, which this module only imports when it is used.
_BLOCK = ("norm_in", "norm_out", "norm_in_backward", "norm_out_backward", "Adapters", "ffn_forward", "ffn_backward",
          "block_check", "Block")


def __getattr__(name):
    if name not in _BLOCK:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import block

    globals().update({k: getattr(block, k) for k in _BLOCK})
    return globals()[name]
