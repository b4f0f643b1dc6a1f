"""Python binding of the B200 DECO MoE FFN library (libdeco_moe.so).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  Importing
this package loads the in-tree shared library and fails loudly if it is
missing; there is no fallback implementation.

The C ABI and the layer's definition are documented in include/deco_moe.h.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdeco_moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python sparse_moe_ffn_relu_b200/build.py` "
        "(the DECO MoE layer has no non-CUDA implementation)")
_lib = ctypes.CDLL(LIB_PATH)

DECO_F32, DECO_BF16 = 0, 1
_DT = {torch.float32: DECO_F32, torch.bfloat16: DECO_BF16}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace", 4: "cuda", 5: "device"}


class DecoError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = f"{what}: {_lib.deco_status_string(code).decode()} (status {code})"
        if code == 4:
            msg += f" -- {_lib.deco_last_cuda_error().decode()}"
        super().__init__(msg)
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d_model", ctypes.c_int), ("E", ctypes.c_int),
                ("d_e", ctypes.c_int), ("d_s", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("residual", ctypes.c_int), ("topk", ctypes.c_int),
                ("gated", ctypes.c_int), ("experts_on_host", ctypes.c_int)]


WEIGHT_NAMES = ("W_r", "b_r", "W_up", "W_bar_up", "W_down", "s", "W_s_up", "W_s_down", "W_val")


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_NAMES]


GRAD_NAMES = ("dx", "dW_r", "db_r", "dW_up", "dW_down", "ds", "dW_s_up", "dW_s_down", "dW_val")


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GRAD_NAMES]


class Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("r", "active", "counts", "offsets", "perm", "n_tok")]


class BlockNorm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d_model", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("branch_scale", ctypes.c_float), ("gate", ctypes.c_int),
                ("ld_x", ctypes.c_longlong), ("ld_y", ctypes.c_longlong), ("ld_gate", ctypes.c_longlong),
                ("ld_out", ctypes.c_longlong), ("ld_h", ctypes.c_longlong),
                ("dh_dtype", ctypes.c_int), ("dout_dtype", ctypes.c_int)]


class BlockNormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "dy", "dg_pre", "dg_post", "dgate")]


class Dispatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("counts", "offsets", "slot_of", "row_of", "n_pairs", "xs")]
    _fields_ += [("ld_xs", ctypes.c_longlong), ("capacity", ctypes.c_longlong)]


_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
_i, _ll = ctypes.c_int, ctypes.c_longlong
_sig = {
    "deco_moe_workspace_size": [ctypes.POINTER(Shape), ctypes.POINTER(_sz)],
    "deco_moe_forward": [ctypes.POINTER(Shape), _vp, ctypes.POINTER(Weights), _vp, _vp, _sz, _vp],
    "deco_moe_routing": [ctypes.POINTER(Shape), _vp, ctypes.POINTER(Weights),
                         ctypes.POINTER(Routing), _vp, _sz, _vp],
    "deco_moe_mean_up": [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp],
    "deco_dense_ffn_workspace_size": [ctypes.c_int] * 4 + [ctypes.POINTER(_sz)],
    "deco_dense_ffn_forward": [ctypes.c_int] * 4 + [_vp] * 4 + [_vp, _sz, _vp],
    "deco_moe_device_error": [_vp, ctypes.POINTER(ctypes.c_int), _vp],
    "deco_moe_set_profiling": [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int],
    "deco_moe_forward_static": [ctypes.POINTER(Shape), _vp, ctypes.POINTER(Weights), _vp, _vp],
    "deco_moe_static_device_error": [ctypes.POINTER(ctypes.c_int), _vp],
    "deco_set_wait_limit": [ctypes.c_longlong],
    "deco_moe_backward_workspace_size": [ctypes.POINTER(Shape), ctypes.POINTER(_sz)],
    "deco_moe_backward": [ctypes.POINTER(Shape), _vp, ctypes.POINTER(Weights), _vp, _vp,
                          ctypes.POINTER(Grads), _vp, _sz, _vp],
    "deco_moe_router_entropy": [ctypes.c_int, ctypes.c_int, _vp, _vp, ctypes.c_float, _vp, _vp, _vp],
    "deco_sparsity_controller": [ctypes.POINTER(ctypes.c_double), ctypes.c_double, ctypes.c_double,
                                 ctypes.c_double],
    "deco_block_norm_forward": [ctypes.POINTER(BlockNorm)] + [_vp] * 8,
    "deco_block_norm_backward_workspace_size": [ctypes.POINTER(BlockNorm), ctypes.POINTER(_sz)],
    "deco_block_norm_backward": [ctypes.POINTER(BlockNorm)] + [_vp] * 7
                                + [ctypes.POINTER(BlockNormGrads), _vp, _sz, _vp],
    "deco_moe_dispatch_workspace_size": [_i] * 5 + [ctypes.POINTER(_sz)],
    "deco_moe_dispatch": [_i] * 5 + [_vp, _vp, _vp, _ll, ctypes.POINTER(Dispatch), _vp, _sz, _vp],
    "deco_moe_combine": [_i] * 5 + [_vp, _vp, _vp, _ll, _ll, _vp, _ll, _vp, _ll, _vp],
    "deco_moe_combine_backward": [_i] * 4 + [_vp, _vp, _vp, _ll, _ll, _vp, _ll, _vp, _ll, _vp, _vp],
    "deco_q4_quantize": [_ll, _i, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "deco_q4_pack": [_ll, _i, _vp, _vp, _vp],
    "deco_q4_dequantize": [_ll, _i, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "deco_q4_matvec": [_i] * 6 + [_vp, _ll, _vp, _vp, _vp, _vp, _ll, _vp],
    "deco_q4_expert_matvec": [_i] * 6 + [_vp, _vp, _i, _vp, _ll, _vp, _vp, _vp, _ll, _vp, _ll, _vp],
}
for _name, _args in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
_lib.deco_status_string.argtypes = [ctypes.c_int]
_lib.deco_status_string.restype = ctypes.c_char_p
_lib.deco_last_cuda_error.argtypes = []
_lib.deco_last_cuda_error.restype = ctypes.c_char_p

# every symbol include/deco_moe.h declares
EXPORTS = tuple(_sig) + ("deco_status_string", "deco_last_cuda_error")


def _check(code: int, what: str):
    if code != 0:
        raise DecoError(code, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_shape(T, D, E, d_e, d_s, dtype, eps=1e-6, residual=False, topk=0, gated=False,
               experts_on_host=False) -> Shape:
    return Shape(T, D, E, d_e, d_s, _DT[dtype] if isinstance(dtype, torch.dtype) else dtype,
                 eps, int(bool(residual)), int(topk), int(bool(gated)), int(bool(experts_on_host)))


def _weights(L: dict) -> Weights:
    return Weights(*[_ptr(L.get(n)) for n in WEIGHT_NAMES])


def layer_shape(x: torch.Tensor, L: dict, eps=1e-6, residual=False, topk=0) -> Shape:
    """The shape of a call; routed experts held in pinned host tensors (W_up,
    W_down, W_val on the CPU, pin_memory) select experts_on_host."""
    E, d_e, D = L["W_up"].shape if "W_up" in L else (L["W_r"].shape[0], 64, x.shape[1])
    d_s = L["W_s_up"].shape[0] if "W_s_up" in L else 64
    on_host = "W_up" in L and L["W_up"].device.type == "cpu"
    return make_shape(x.shape[0], x.shape[1], L["W_r"].shape[0], d_e, d_s, x.dtype, eps, residual,
                      topk, "W_val" in L, on_host)


def workspace_size(shape: Shape) -> int:
    n = _sz(0)
    _check(_lib.deco_moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "workspace_size")
    return n.value


def alloc_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    return torch.empty(max(workspace_size(shape), 256), dtype=torch.uint8, device=device)


def forward(x: torch.Tensor, L: dict, out=None, workspace=None, eps=1e-6, residual=False,
            stream=None, topk=0) -> torch.Tensor:
    """out = DECO MoE layer(x) (+ x if residual).  L: dict of device tensors.
    topk > 0 replaces ReLU routing by the TopK baseline with k = topk."""
    shape = layer_shape(x, L, eps, residual, topk)
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = alloc_workspace(shape, x.device)
    w = _weights(L)
    _check(_lib.deco_moe_forward(ctypes.byref(shape), _ptr(x), ctypes.byref(w), _ptr(out),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "forward")
    return out


STATIC_SCRATCH_BYTES = 64 << 20


def forward_static(x: torch.Tensor, L: dict, out=None, eps=1e-6, residual=False,
                   stream=None) -> torch.Tensor:
    """forward() on the library's built-in 64 MiB device scratch instead of a
    workspace, for callers that cannot allocate device memory while running
    layers.  Calls on one device share that scratch: do not let them overlap
    on the GPU.  The first call on a device should come before any stream
    capture.  Raises DecoError (status 3) if the shape needs more scratch."""
    shape = layer_shape(x, L, eps, residual)
    if out is None:
        out = torch.empty_like(x)
    w = _weights(L)
    _check(_lib.deco_moe_forward_static(ctypes.byref(shape), _ptr(x), ctypes.byref(w), _ptr(out),
                                        _stream(stream)), "forward_static")
    return out


def routing(x: torch.Tensor, L: dict, workspace=None, stream=None, topk=0) -> dict:
    """Router + token->expert tables; returns r, active, counts, offsets, perm, n_tok."""
    T, E = x.shape[0], L["W_r"].shape[0]
    shape = layer_shape(x, L, topk=topk)
    if workspace is None:
        workspace = alloc_workspace(shape, x.device)
    dev = x.device
    res = dict(r=torch.empty(T, E, dtype=torch.float32, device=dev),
               active=torch.empty(T, E, dtype=torch.uint8, device=dev),
               counts=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               perm=torch.empty(max(T * E, 1), dtype=torch.int32, device=dev),
               n_tok=torch.empty(max(T, 1), dtype=torch.int32, device=dev))
    out = Routing(*[_ptr(res[n]) for n in ("r", "active", "counts", "offsets", "perm", "n_tok")])
    w = _weights(L)
    _check(_lib.deco_moe_routing(ctypes.byref(shape), _ptr(x), ctypes.byref(w), ctypes.byref(out),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "routing")
    return res


def mean_up(W_up: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """W_bar_up = mean over experts of W_up [E, d_e, D] (fp64 sum, one rounding)."""
    E, d_e, D = W_up.shape
    if out is None:
        out = torch.empty(d_e, D, dtype=W_up.dtype, device=W_up.device)
    _check(_lib.deco_moe_mean_up(E, d_e, D, _DT[W_up.dtype], _ptr(W_up), _ptr(out),
                                 _stream(stream)), "mean_up")
    return out


def dense_workspace_size(T, D, d_ff, dtype) -> int:
    n = _sz(0)
    _check(_lib.deco_dense_ffn_workspace_size(T, D, d_ff, _DT[dtype], ctypes.byref(n)),
           "dense_ffn_workspace_size")
    return n.value


def dense_ffn(x, W1, W2, out=None, workspace=None, stream=None) -> torch.Tensor:
    """out = W2 SiLU(W1 x), the equal-parameter dense FFN baseline."""
    T, D = x.shape
    d_ff = W1.shape[0]
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = torch.empty(dense_workspace_size(T, D, d_ff, x.dtype), dtype=torch.uint8,
                                device=x.device)
    _check(_lib.deco_dense_ffn_forward(T, D, d_ff, _DT[x.dtype], _ptr(x), _ptr(W1), _ptr(W2),
                                       _ptr(out), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "dense_ffn")
    return out


# timing slots of deco_moe_set_profiling: slot i is bracketed by events 2i and
# 2i+1.  The general path fills route..down, the prefill path (bf16, T > 16)
# route..combine, the decode path (bf16, T <= 16) only "layer" (one kernel).
KERNELS = ("route", "count", "scatter", "up", "down")
PREFILL_KERNELS = KERNELS + ("proj", "shared", "combine")
ALL_SLOTS = PREFILL_KERNELS + ("layer",)


def set_profiling(events):
    """Record events[2i] / events[2i+1] around the i-th kernel of every later
    forward call (a list of torch.cuda.Event, len 2*len(KERNELS)); None stops."""
    global _prof_keep
    if events is None:
        _prof_keep = None
        _check(_lib.deco_moe_set_profiling(None, 0), "set_profiling")
        return
    handles = [e.cuda_event for e in events]
    if not all(handles):
        raise ValueError("set_profiling: every event must exist (record it once first)")
    arr = (ctypes.c_void_p * len(events))(*handles)
    _prof_keep = (arr, events)
    _check(_lib.deco_moe_set_profiling(arr, len(events)), "set_profiling")


_prof_keep = None


def device_error(workspace, stream=None) -> int:
    code = ctypes.c_int(0)
    _check(_lib.deco_moe_device_error(_ptr(workspace), ctypes.byref(code), _stream(stream)),
           "device_error")
    return code.value


def static_device_error(stream=None) -> int:
    """The device error word of the last forward_static call on this device (cleared)."""
    code = ctypes.c_int(0)
    _check(_lib.deco_moe_static_device_error(ctypes.byref(code), _stream(stream)),
           "static_device_error")
    return code.value


def set_wait_limit(cycles: int):
    """Test hook: kernels give up waits for data after `cycles` SM cycles (0: default)."""
    _check(_lib.deco_set_wait_limit(int(cycles)), "set_wait_limit")


# --------------------------------------------------------------------------
# training side

def backward(x: torch.Tensor, L: dict, dy: torch.Tensor, dz_extra=None, workspace=None, eps=1e-6,
             residual=False, stream=None) -> dict:
    """Gradients of the loss through the layer given dy = dLoss/dout: a dict
    of fp32 tensors dx, dW_r, db_r, dW_up (with the mean up-projection's
    share), dW_down, ds, dW_s_up, dW_s_down (and dW_val for gated experts).
    dz_extra [T][E] fp32: an extra gradient on the router logits (see
    router_entropy)."""
    shape = layer_shape(x, L, eps, residual)
    n = _sz(0)
    _check(_lib.deco_moe_backward_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "backward_workspace_size")
    if workspace is None:
        workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = {"dx": torch.empty(x.shape, **f32)}
    for name, src in (("dW_r", "W_r"), ("db_r", "b_r"), ("dW_up", "W_up"), ("dW_down", "W_down"),
                      ("ds", "s"), ("dW_s_up", "W_s_up"), ("dW_s_down", "W_s_down"), ("dW_val", "W_val")):
        if src in L:
            g[name] = torch.empty(L[src].shape, **f32)
    gs = Grads(*[_ptr(g.get(n)) for n in GRAD_NAMES])
    w = _weights(L)
    _check(_lib.deco_moe_backward(ctypes.byref(shape), _ptr(x), ctypes.byref(w), _ptr(dy), _ptr(dz_extra),
                                  ctypes.byref(gs), _ptr(workspace), workspace.numel(), _stream(stream)),
           "backward")
    return g


def router_entropy(r: torch.Tensor, active: torch.Tensor, lam: float, stream=None):
    """(H [T+1] with the per-token router entropies and their mean last,
    dz [T][E] = lam * d(mean entropy)/dz) from deco_moe_routing's r and
    active."""
    T, E = r.shape
    H = torch.empty(T + 1, dtype=torch.float32, device=r.device)
    dz = torch.empty(T, E, dtype=torch.float32, device=r.device)
    _check(_lib.deco_moe_router_entropy(T, E, _ptr(r), _ptr(active), float(lam), _ptr(H), _ptr(dz),
                                        _stream(stream)), "router_entropy")
    return H, dz


def sparsity_controller(lam: float, ratio: float, target: float, factor: float = 1.002) -> float:
    """One step of the adaptive sparsity coefficient (x factor above the
    target activation ratio, / factor below)."""
    v = ctypes.c_double(lam)
    _check(_lib.deco_sparsity_controller(ctypes.byref(v), float(ratio), float(target), float(factor)),
           "sparsity_controller")
    return v.value


# --------------------------------------------------------------------------
# the block around the layer: norms, tokens sorted by expert and back, 4-bit
# weights.  These run on the device of their tensors, on `stream` or that
# device's current stream; what they allocate belongs to that stream.

# Small calls are bound by the time this module takes, so the checks below look
# at each property once, with PyTorch's cheapest accessors; builds of PyTorch
# that lack the private ones have the public calls.
def _public_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)     # of a device, as an integer
_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def _elsewhere(t: torch.Tensor, stream):
    """The context a call on t's device and `stream` needs, None if it is already current."""
    if not t.is_cuda:
        raise ValueError(f"expected tensors on a CUDA device, got {t.device}")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream on {stream.device}, tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() != _current_device():
        return torch.cuda.device(t.device)
    return None


def _mismatch(t, what, shape, dtype, dev):
    where = f"cuda:{dev}" if dev >= 0 else "cpu"
    return ValueError(f"{what}: expected {dtype} {tuple(shape)} on {where}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _whole(t, what: str, shape, dtype, dev: int):
    """The address of an optional contiguous tensor on device number dev."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise _mismatch(t, what, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor, got strides {t.stride()}")
    return t.data_ptr()


def _rows(t, what: str, shape, dtype, dev: int):
    """The address and row stride of an optional tensor [n][width] whose rows may have gaps between them."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise _mismatch(t, what, shape, dtype, dev)
    n, width = shape
    if t.is_contiguous():
        return t.data_ptr(), width
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: expected rows without gaps between their elements, got strides {t.stride()}")
    if n > 1 and t.stride(0) < width:
        raise ValueError(f"{what}: rows overlap, strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if n > 1 else width


def _storage(t: torch.Tensor, what: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: expected float32 or bfloat16, got {t.dtype}")
    return dt


# The C side takes most sizes as 32-bit integers, and ctypes cuts what it is
# given to that without a word.
def _matrix(t: torch.Tensor, what: str, row_bits: int = 31):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what}: expected two dimensions, got {tuple(shape)}")
    if t.numel() >> 31 and (shape[0] >> row_bits or shape[1] >> 31):
        raise ValueError(f"{what}: {tuple(shape)} has a size of 2^31 or more")
    return shape


def _experts(E: int) -> int:
    if E >> 31:
        raise ValueError(f"E: expected a number below 2^31, got {E}")
    return E


_GATES = {"channel": 1, "token": 2, "full": 3}     # deco_gate_t


def _gate_kind(gate, T: int, D: int, kind=None) -> int:
    """deco_gate_t of a gate, by its shape: [D] per channel, [T] or [T][1] per
    token, [T][D] full.  kind ("channel", "token", "full") names it, which a
    gate [n] with n = T = D needs."""
    if gate is None:
        if kind is not None:
            raise ValueError(f"gate_kind {kind!r} without a gate")
        return 0
    shape = gate.shape
    if kind is not None:
        if kind not in _GATES:
            raise ValueError(f"gate_kind: expected one of {tuple(_GATES)}, got {kind!r}")
        if shape != {"channel": (D,), "token": (T,), "full": (T, D)}[kind] and not (kind == "token" and shape == (T, 1)):
            raise ValueError(f"gate: {tuple(shape)} is not a {kind} gate of {T} tokens of {D} channels")
        return _GATES[kind]
    if shape == (D,):
        if T == D and D > 1:
            raise ValueError(f"gate: [{D}] with {T} tokens of {D} channels is per channel or per token: name it with gate_kind")
        return 1
    if shape == (T, D) and not (D == 1 and gate.dtype is _F32):
        return 3
    if shape == (T,) or shape == (T, 1):
        return 2
    raise ValueError(f"gate: expected [{D}], [{T}], [{T}][1] or [{T}][{D}], got {tuple(shape)}")


def block_norm(x: torch.Tensor, g_pre=None, y=None, g_post=None, gate=None, branch_scale: float = 1.0,
               eps=1e-6, out=None, h=None, stream=None, gate_kind=None):
    """(out, h) with out = x + branch_scale * gate * RMSNorm(y) * g_post and
    h = RMSNorm(out) * g_pre: the norm, gate and residual scale behind a block
    and the norm before the next, in one pass.

    x, y [T][D] fp32 or bf16; g_pre, g_post [D] fp32.  gate: [D] fp32 (per
    channel), [T] or [T][1] fp32 (per token) or [T][D] (x's type); gate_kind
    "channel", "token" or "full" says which, and has to where a gate has one
    dimension and T = D > 1.  Without y, h = RMSNorm(x) * g_pre and out is None.  Without g_post y is added as it
    is; without g_pre there is no h.  out may be x."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return block_norm(x, g_pre, y, g_post, gate, branch_scale, eps, out, h, None, gate_kind)
    dt, dtype, dev, shape = _storage(x, "x"), x.dtype, x.get_device(), _matrix(x, "x")
    T, D = shape
    px, ld_x = _rows(x, "x", shape, dtype, dev)
    py, ld_y = _rows(y, "y", shape, dtype, dev)
    kind, ld_gate = _gate_kind(gate, T, D, gate_kind), 0
    if kind == 3:
        p_gate, ld_gate = _rows(gate, "gate", shape, dtype, dev)
    else:
        p_gate = None if kind == 0 else _whole(gate, "gate", gate.shape, _F32, dev)
    if y is not None and out is None:
        out = torch.empty_like(x)       # a row-strided x: without its gaps
    if g_pre is not None and h is None:
        h = torch.empty_like(x)
    p_out, ld_out = _rows(out, "out", shape, dtype, dev)
    ph, ld_h = _rows(h, "h", shape, dtype, dev)
    s = BlockNorm(T, D, dt, eps, branch_scale, kind, ld_x, ld_y, ld_gate, ld_out, ld_h, dt, dt)
    rc = _lib.deco_block_norm_forward(s, px, py, _whole(g_post, "g_post", (D,), _F32, dev), p_gate,
                                      _whole(g_pre, "g_pre", (D,), _F32, dev), p_out, ph, _raw_stream(dev))
    if rc:
        raise DecoError(rc, "block_norm")
    return out, h


@functools.lru_cache(maxsize=256)
def _norm_workspace(T: int, D: int, dt: int, dev: int) -> int:
    """Bytes of the backward pass's workspace: by sizes and device alone."""
    n = _sz(0)
    _check(_lib.deco_block_norm_backward_workspace_size(BlockNorm(T, D, dt), n), "block_norm_backward_workspace_size")
    return n.value


def block_norm_backward(x: torch.Tensor, g_pre=None, y=None, g_post=None, gate=None, branch_scale: float = 1.0,
                        eps=1e-6, dout=None, dh=None, dx=None, workspace=None, stream=None, gate_kind=None) -> dict:
    """Gradients of block_norm: a dict of dx, dy, dg_pre, dg_post, dgate (those
    that exist).  x is the sum the forward pass stored (its out, or its x where
    it had no y).  dout: gradient with respect to out apart from h's share, dh:
    with respect to h; one of them may be missing.  Each is in x's type or fp32
    (the type of backward()'s dx); dx comes in dout's type (x's without dout)
    and may be dout.  dg_pre, dg_post and the gradients of [D] and [T] gates
    are fp32, dy and a [T][D] gate's gradient in x's type.  Without dh, g_pre
    is not used.  gate_kind as in block_norm."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return block_norm_backward(x, g_pre, y, g_post, gate, branch_scale, eps, dout, dh, dx, workspace, None, gate_kind)
    dt, dtype, dev, shape = _storage(x, "x"), x.dtype, x.get_device(), _matrix(x, "x")
    T, D = shape
    if dh is None:
        g_pre = None
    px, ld_x = _rows(x, "x", shape, dtype, dev)
    py, ld_y = _rows(y, "y", shape, dtype, dev)
    kind, ld_gate = _gate_kind(gate, T, D, gate_kind), 0
    if kind == 3:
        p_gate, ld_gate = _rows(gate, "gate", shape, dtype, dev)
    else:
        p_gate = None if kind == 0 else _whole(gate, "gate", gate.shape, _F32, dev)
    dh_t, dx_t, dx_dtype = dt, dt, dtype
    if dh is not None:
        dh_t = _storage(dh, "dh")
    if dout is not None:
        dx_t, dx_dtype = _storage(dout, "dout"), dout.dtype
    p_dout, ld_dout = _rows(dout, "dout", shape, dx_dtype, dev)
    p_dh, ld_dh = _rows(dh, "dh", shape, None if dh is None else dh.dtype, dev)
    if dx is None:
        dx = torch.empty_like(x, dtype=dx_dtype, memory_format=torch.contiguous_format)
    s = BlockNorm(T, D, dt, eps, branch_scale, kind, ld_x, ld_y, ld_gate, ld_dout, ld_dh, dh_t, dx_t)
    if workspace is None:
        workspace = x.new_empty(_norm_workspace(T, D, dt, dev), dtype=_U8)
    g = {"dx": dx}
    gs = BlockNormGrads(_whole(dx, "dx", shape, dx_dtype, dev))
    if y is not None:
        g["dy"] = torch.empty_like(y, memory_format=torch.contiguous_format)
        gs.dy = g["dy"].data_ptr()
    if dh is not None:
        g["dg_pre"] = torch.empty_like(g_pre)
        gs.dg_pre = g["dg_pre"].data_ptr()
    if g_post is not None:
        g["dg_post"] = torch.empty_like(g_post)
        gs.dg_post = g["dg_post"].data_ptr()
    if gate is not None:
        g["dgate"] = torch.empty_like(gate, memory_format=torch.contiguous_format)
        gs.dgate = g["dgate"].data_ptr()
    rc = _lib.deco_block_norm_backward(s, px, py, _whole(g_post, "g_post", (D,), _F32, dev), p_gate,
                                       _whole(g_pre, "g_pre", (D,), _F32, dev), p_dout, p_dh, gs,
                                       _whole(workspace, "workspace", workspace.shape, _U8, dev), workspace.numel(), _raw_stream(dev))
    if rc:
        raise DecoError(rc, "block_norm_backward")
    return g


@functools.lru_cache(maxsize=256)
def _dispatch_workspace(T: int, S: int, E: int, D: int, dt: int) -> int:
    n = _sz(0)
    _check(_lib.deco_moe_dispatch_workspace_size(T, S, E, D, dt, n), "dispatch_workspace_size")
    return n.value


_NO_WORKSPACE = 1024     # slots that a batch is sorted without one, whatever its rows


def dispatch(x, E=None, experts=None, active=None, capacity=None, out=None, workspace=None, stream=None) -> dict:
    """(token, expert) pairs sorted by expert, and the tokens' rows in that
    order: a dict of xs [capacity][D], counts [E], offsets [E+1], slot_of
    [capacity], row_of [T][slots] and n_pairs [1] (int32), as described with
    deco_dispatch_t in the C header.

    The pairs: `experts` [T][slots] int32 with E (numbers outside 0..E-1 are
    empty slots), or `active` [T][E] uint8 or bool (routing()'s mask).
    capacity: rows of xs, T * slots unless given; pairs beyond it get no row,
    n_pairs tells.  Rows of xs and slot_of behind the last pair are left as
    they were (uninitialised when allocated here).  out: a dict of the same
    tensors to write into.  x None: the tables alone."""
    pairs = active if experts is None else experts
    if pairs is None or (experts is not None and active is not None):
        raise ValueError("dispatch: give either experts or active")
    ctx = _elsewhere(pairs, stream)
    if ctx is not None:
        with ctx:
            return dispatch(x, E, experts, active, capacity, out, workspace)
    shape, dev = _matrix(pairs, "pairs"), pairs.get_device()
    T, S = shape
    p_experts = p_active = None
    if experts is None:
        if active.dtype is torch.bool:
            active = active.view(_U8)
        p_active = _whole(active, "active", shape, _U8, dev)
        if E is not None and E != S:
            raise ValueError(f"active has {S} experts, E is {E}")
        E = S
    else:
        if E is None:
            raise ValueError("dispatch: E is needed with experts")
        E = _experts(E)
        p_experts = _whole(experts, "experts", shape, _I32, dev)
    D, dt, px, ld_x = 1, DECO_F32, None, 0
    if x is not None:
        dt, dtype = _storage(x, "x"), x.dtype
        D = _matrix(x, "x")[1]
        px, ld_x = _rows(x, "x", (T, D), dtype, dev)
    if out is None:
        cap = T * S if capacity is None else int(capacity)
        i32 = dict(dtype=_I32, device=pairs.device)
        out = dict(counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32), slot_of=torch.empty(cap, **i32),
                   row_of=torch.empty(shape, **i32), n_pairs=torch.empty(1, **i32))
        if x is not None:
            out["xs"] = torch.empty((cap, D), dtype=dtype, device=pairs.device)
    else:
        cap = out["slot_of"].shape[0]
        if capacity is not None and capacity != cap:
            raise ValueError(f"capacity is {capacity}, out has {cap} rows")
        if ("xs" in out) != (x is not None):
            raise ValueError("dispatch: out has xs if and only if there is x")
    o = Dispatch(_whole(out["counts"], "counts", (E,), _I32, dev), _whole(out["offsets"], "offsets", (E + 1,), _I32, dev),
                 _whole(out["slot_of"], "slot_of", (cap,), _I32, dev), _whole(out["row_of"], "row_of", shape, _I32, dev),
                 _whole(out["n_pairs"], "n_pairs", (1,), _I32, dev))
    if x is not None:
        o.xs, o.ld_xs = _rows(out["xs"], "xs", (cap, D), dtype, dev)
    o.capacity = cap
    p_ws = n_ws = 0
    if T * S > _NO_WORKSPACE or D > 8192:
        if workspace is None and (n := _dispatch_workspace(T, S, E, D, dt)):
            workspace = pairs.new_empty(n, dtype=_U8)
    if workspace is not None:
        p_ws, n_ws = _whole(workspace, "workspace", workspace.shape, _U8, dev), workspace.numel()
    rc = _lib.deco_moe_dispatch(T, S, E, D, dt, p_experts, p_active, px, ld_x, o, p_ws, n_ws, _raw_stream(dev))
    if rc:
        raise DecoError(rc, "dispatch")
    return out


def combine(ys: torch.Tensor, row_of: torch.Tensor, w=None, base=None, out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """Rows back to token order: y[t] = base[t] + sum_k w[t][k] ys[row_of[t][k]]
    over the slots that have a row; w [T][slots] fp32 (None: 1), base [T][D] in
    ys's type (None: 0).  out_dtype: ys's type (default) or float32.  out may
    be base."""
    ctx = _elsewhere(ys, stream)
    if ctx is not None:
        with ctx:
            return combine(ys, row_of, w, base, out, out_dtype)
    dt, dtype, dev, table = _storage(ys, "ys"), ys.dtype, ys.get_device(), _matrix(row_of, "row_of")
    T, S = table
    n, D = _matrix(ys, "ys", 63)
    p_ys, ld_ys = _rows(ys, "ys", (n, D), dtype, dev)
    p_base, ld_base = _rows(base, "base", (T, D), dtype, dev)
    if out is None:
        out = torch.empty((T, D), dtype=out_dtype or dtype, device=ys.device)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    p_out, ld_out = _rows(out, "out", (T, D), out.dtype, dev)
    rc = _lib.deco_moe_combine(T, S, D, dt, _storage(out, "out"), _whole(row_of, "row_of", table, _I32, dev), _whole(w, "w", table, _F32, dev),
                               p_ys, n, ld_ys, p_base, ld_base, p_out, ld_out, _raw_stream(dev))
    if rc:
        raise DecoError(rc, "combine")
    return out


def combine_backward(ys: torch.Tensor, row_of: torch.Tensor, w, dy: torch.Tensor, dys=None, stream=None):
    """(dys, dw): gradients of combine with respect to ys (its type; rows that
    no slot names are left as they were, uninitialised when allocated here) and
    w (fp32, 0 where a slot has no row; None without w).  The gradient of base
    is dy; that of ys without weights (w None) is dispatch's copy of dy."""
    ctx = _elsewhere(ys, stream)
    if ctx is not None:
        with ctx:
            return combine_backward(ys, row_of, w, dy, dys)
    dt, dtype, dev, table = _storage(ys, "ys"), ys.dtype, ys.get_device(), _matrix(row_of, "row_of")
    T, S = table
    n, D = _matrix(ys, "ys", 63)
    p_ys, ld_ys = _rows(ys, "ys", (n, D), dtype, dev)
    p_dy, ld_dy = _rows(dy, "dy", (T, D), dtype, dev)
    if dys is None:
        dys = torch.empty_like(ys, memory_format=torch.contiguous_format)
    p_dys, ld_dys = _rows(dys, "dys", (n, D), dtype, dev)
    p_w = _whole(w, "w", table, _F32, dev)
    dw = None if w is None else torch.empty_like(w)
    rc = _lib.deco_moe_combine_backward(T, S, D, dt, _whole(row_of, "row_of", table, _I32, dev), p_w, p_ys, n, ld_ys, p_dy, ld_dy, p_dys,
                                        ld_dys, None if dw is None else dw.data_ptr(), _raw_stream(dev))
    if rc:
        raise DecoError(rc, "combine_backward")
    return dys, dw


def dispatch_backward(dxs: torch.Tensor, row_of: torch.Tensor, out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """dx[t] = the sum of dxs over the rows that dispatch gave token t."""
    return combine(dxs, row_of, out=out, out_dtype=out_dtype, stream=stream)


Q4_GROUPS = (32, 64, 128)


def _q4_sizes(K: int, group: int):
    """Bytes of codes and number of groups of a row, its padding included."""
    if group not in Q4_GROUPS:
        raise ValueError(f"group: expected one of {Q4_GROUPS}, got {group}")
    if K >> 31:
        raise ValueError(f"K: expected a number below 2^31, got {K}")
    Kp = -(-K // 128) * 128
    return Kp // 2, Kp // group


def q4_quantize(W: torch.Tensor, group: int = 64, zero: bool = False, stream=None) -> dict:
    """4-bit weights of W [..][N][K] (fp32 or bf16): a dict of q, scale, zero
    (None if symmetric), K and group, as the C header describes them."""
    ctx = _elsewhere(W, stream)
    if ctx is not None:
        with ctx:
            return q4_quantize(W, group, zero)
    dt, dev = _storage(W, "W"), W.get_device()
    pW = _whole(W, "W", W.shape, W.dtype, dev)
    *lead, K = W.shape
    nq, ns = _q4_sizes(K, group)
    r = dict(q=torch.empty((*lead, nq), dtype=_U8, device=W.device), scale=torch.empty((*lead, ns), dtype=_BF16, device=W.device),
             zero=torch.empty((*lead, ns), dtype=_U8, device=W.device) if zero else None, K=K, group=group)
    _check(_lib.deco_q4_quantize(W.numel() // max(K, 1), K, group, dt, pW, _ptr(r["q"]), _ptr(r["scale"]), _ptr(r["zero"]),
                                 _raw_stream(dev)), "q4_quantize")
    return r


def q4_pack(codes: torch.Tensor, scale: torch.Tensor, zero=None, group: int = 64, stream=None) -> dict:
    """4-bit weights from given codes [..][N][K] (uint8, 0..15), scale
    [..][N][Kp / group] bf16 and zero (the same, uint8, or None: 8), Kp = K
    rounded up to a multiple of 128."""
    ctx = _elsewhere(codes, stream)
    if ctx is not None:
        with ctx:
            return q4_pack(codes, scale, zero, group)
    *lead, K = codes.shape
    dev = codes.get_device()
    nq, ns = _q4_sizes(K, group)
    p = _whole(codes, "codes", codes.shape, _U8, dev)
    _whole(scale, "scale", (*lead, ns), _BF16, dev)
    _whole(zero, "zero", (*lead, ns), _U8, dev)
    q = torch.empty((*lead, nq), dtype=_U8, device=codes.device)
    _check(_lib.deco_q4_pack(codes.numel() // max(K, 1), K, p, _ptr(q), _raw_stream(dev)), "q4_pack")
    return dict(q=q, scale=scale, zero=zero, K=K, group=group)


def _q4_weights(W: dict, dims: int, dev: int):
    """Checks 4-bit weights: their leading sizes, K, group and addresses."""
    q, K, group = W["q"], W["K"], W["group"]
    nq, ns = _q4_sizes(K, group)
    lead = tuple(q.shape[:-1])
    if dims and len(lead) != dims:
        raise ValueError(f"q: expected {dims + 1} dimensions, got {tuple(q.shape)}")
    groups = (*lead, ns)
    return (lead, K, group, _whole(q, "q", (*lead, nq), _U8, dev), _whole(W["scale"], "scale", groups, _BF16, dev),
            _whole(W["zero"], "zero", groups, _U8, dev))


def q4_dequantize(W: dict, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The weights [..][N][K] in dtype."""
    q = W["q"]
    ctx = _elsewhere(q, stream)
    if ctx is not None:
        with ctx:
            return q4_dequantize(W, dtype)
    lead, K, group, pq, ps, pz = _q4_weights(W, 0, q.get_device())
    out = torch.empty((*lead, K), dtype=dtype, device=q.device)
    _check(_lib.deco_q4_dequantize(out.numel() // max(K, 1), K, group, _storage(out, "dtype"), pq, ps, pz, _ptr(out),
                                   _raw_stream(q.get_device())), "q4_dequantize")
    return out


def q4_matvec(x: torch.Tensor, W: dict, out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """y = x W^T for x [T][K] and 4-bit weights W [N][K] (q4_quantize, q4_pack);
    y [T][N] in x's type or float32.  Made for the few rows of a decode batch."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return q4_matvec(x, W, out, out_dtype)
    dt, dev, T = _storage(x, "x"), x.get_device(), _matrix(x, "x")[0]
    (N,), K, group, pq, ps, pz = _q4_weights(W, 1, dev)
    px, ld_x = _rows(x, "x", (T, K), x.dtype, dev)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype or x.dtype, device=x.device)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    py, ld_y = _rows(out, "out", (T, N), out.dtype, dev)
    rc = _lib.deco_q4_matvec(T, N, K, group, dt, _storage(out, "out"), px, ld_x, pq, ps, pz, py, ld_y, _raw_stream(dev))
    if rc:
        raise DecoError(rc, "q4_matvec")
    return out


def q4_expert_matvec(x: torch.Tensor, W: dict, offsets: torch.Tensor, perm=None, out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """Row i of y, in offsets[e] .. offsets[e+1]-1, = W[e] x[perm[i]] (x[i]
    without perm), for 4-bit weights W [E][N][K] and the offsets [E+1] (and
    perm) of routing() or dispatch().  y has perm's (x's) number of rows, in
    x's type or float32; rows behind offsets[E] are left as they were
    (uninitialised when allocated here)."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return q4_expert_matvec(x, W, offsets, perm, out, out_dtype)
    dt, dev, T = _storage(x, "x"), x.get_device(), _matrix(x, "x")[0]
    (E, N), K, group, pq, ps, pz = _q4_weights(W, 2, dev)
    px, ld_x = _rows(x, "x", (T, K), x.dtype, dev)
    rows = T if perm is None else perm.shape[0]
    p_perm = _whole(perm, "perm", (rows,), _I32, dev)
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype or x.dtype, device=x.device)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    py, ld_y = _rows(out, "out", (rows, N), out.dtype, dev)
    rc = _lib.deco_q4_expert_matvec(E, N, K, group, dt, _storage(out, "out"), _whole(offsets, "offsets", (E + 1,), _I32, dev), p_perm, T,
                                    px, ld_x, pq, ps, pz, rows, py, ld_y, _raw_stream(dev))
    if rc:
        raise DecoError(rc, "q4_expert_matvec")
    return out
