"""libq4: Q4_0 block-quantised linear layers on AMD MI355X (gfx950).

This module is the thin Python binding over the C ABI declared in
``include/q4.h``: it marshals torch device tensors into pointers, dtype codes
and a HIP stream handle and calls ``libq4.so``.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.  If the
library has not been built, every call raises ``Q4LibraryMissing`` (build it
with ``python -m bit_block_quantized_q4_amd.build``).

Functions mirror the C entry points: ``q4_packed_size``,
``q4_gemm_workspace_size``, ``q4_gemm_workspace_size_dt``, ``q4_quantize``, ``q4_gemv``, ``q4_gemm``,
``q4_gemm_noalloc``, ``q4_status_string``, ``q4_abi_version``; the fused linear
layer ``q4_linear``; the experts' ``q4_route``, ``q4_route_plan``, ``q4_experts``
and ``q4_moe``, with their size helpers.
"""

from __future__ import annotations

import ctypes
from pathlib import Path
from typing import Optional, Tuple

PKG_DIR = Path(__file__).resolve().parent
LIB_PATH = PKG_DIR / "libq4.so"
HEADER_PATH = PKG_DIR.parent / "include" / "q4.h"

ABI_VERSION = 1
QK = 32
BLOCK_BYTES = 18
GEMV_MAX_M = 32

Q4_OK = 0
Q4_ERR_INVALID_ARG = 1
Q4_ERR_SHAPE = 2
Q4_ERR_DTYPE = 3
Q4_ERR_ALIGNMENT = 4
Q4_ERR_HIP = 5
Q4_ERR_WORKSPACE = 6
Q4_ERR_UNSUPPORTED = 7
Q4_ERR_SCRATCH = 8
NOALLOC_SCRATCH_BYTES = 64 << 20

Q4_F32 = 0
Q4_F16 = 1
Q4_BF16 = 2

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_erf": 3, "silu": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
MAX_EXPERTS = 1024
MAX_TOPK = 32


class Epilogue(ctypes.Structure):
    """q4_epilogue."""
    _fields_ = [("bias", ctypes.c_void_p), ("bias_dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("gated", ctypes.c_int),
                ("residual", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    """q4_routing."""
    _fields_ = [("score", ctypes.c_int), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int),
                ("group_topk", ctypes.c_int), ("group_score", ctypes.c_int),
                ("renormalise", ctypes.c_int), ("scale", ctypes.c_float)]


_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t

# Every function the header declares, with (restype, argtypes).
_SIGS = {
    "q4_abi_version": (ctypes.c_int, []),
    "q4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "q4_packed_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "q4_gemm_workspace_size": (ctypes.c_size_t, [ctypes.c_int64] * 3),
    "q4_gemm_workspace_size_dt": (ctypes.c_size_t, [ctypes.c_int64] * 3 + [ctypes.c_int]),
    "q4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "q4_gemv": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                               ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "q4_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                               ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                               ctypes.c_size_t, ctypes.c_void_p]),
    "q4_gemm_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "q4_linear_workspace_size": (_Z, [_L, _L, _L, _I, _I]),
    "q4_linear": (_I, [_P, _I, _P, _P, _P, _I, _L, _L, _L, _P, _Z, _P]),
    "q4_route_plan_size": (_Z, [_L, _L, _L]),
    "q4_route": (_I, [_P, _I, _L, _L, _L, _P, _P, _P, _P, _P]),
    "q4_route_plan": (_I, [_P, _L, _L, _L, _P, _P]),
    "q4_experts_workspace_size": (_Z, [_L] * 6 + [_I] * 3),
    "q4_experts": (_I, [_P, _I, _L, _P, _P, _P, _P, _P, _I] + [_L] * 5 + [_P, _Z, _P]),
    "q4_moe_workspace_size": (_Z, [_L] * 5 + [_I] * 2),
    "q4_moe": (_I, [_P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _I] + [_L] * 5 + [_P, _P, _P, _Z, _P]),
}


class Q4LibraryMissing(RuntimeError):
    """libq4.so is not built or cannot be loaded."""


class Q4Error(RuntimeError):
    """A libq4 call returned a non-OK status."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({q4_status_string(status)})")


_LIB: Optional[ctypes.CDLL] = None


def hip_runtimes_loaded():
    """Distinct libamdhip64 files mapped into this process (Linux)."""
    try:
        maps = Path("/proc/self/maps").read_text()
    except OSError:  # pragma: no cover
        return []
    return sorted({ln.split()[-1] for ln in maps.splitlines()
                   if "libamdhip64" in ln and ln.split()[-1].startswith("/")})


def lib() -> ctypes.CDLL:
    """The loaded libq4.so (raises Q4LibraryMissing when absent)."""
    global _LIB
    if _LIB is None:
        if not LIB_PATH.exists():
            raise Q4LibraryMissing(
                f"{LIB_PATH} is not built; run `python -m bit_block_quantized_q4_amd.build`")
        # torch ships its own HIP runtime under the same soname as ROCm's.  Load
        # torch first so libq4 binds to that runtime: device pointers and streams
        # handed over by torch are only valid inside the runtime that made them.
        try:
            import torch  # noqa: F401
        except ImportError:  # pragma: no cover - a C caller without torch
            pass
        try:
            L = ctypes.CDLL(str(LIB_PATH))
        except OSError as e:  # pragma: no cover - depends on the host
            raise Q4LibraryMissing(f"cannot load {LIB_PATH}: {e}") from e
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name, None)
            if fn is None:  # functions are added within one ABI version
                raise Q4LibraryMissing(f"{LIB_PATH} has no {name}: it is older than this package; rebuild it")
            fn.restype = res
            fn.argtypes = args
        if L.q4_abi_version() != ABI_VERSION:
            raise Q4LibraryMissing("libq4.so ABI version mismatch; rebuild it")
        runtimes = hip_runtimes_loaded()
        if len(runtimes) > 1:
            raise Q4LibraryMissing(
                "two HIP runtimes are loaded in this process (" + ", ".join(runtimes) +
                "); import torch before loading libq4")
        _LIB = L
    return _LIB


# ------------------------------------------------------------ plain wrappers

def q4_abi_version() -> int:
    return lib().q4_abi_version()


def q4_status_string(status: int) -> str:
    return lib().q4_status_string(int(status)).decode()


def q4_packed_size(n: int, k: int) -> int:
    return lib().q4_packed_size(int(n), int(k))


def q4_gemm_workspace_size(m: int, n: int, k: int) -> int:
    return lib().q4_gemm_workspace_size(int(m), int(n), int(k))


def q4_gemm_workspace_size_dt(m: int, n: int, k: int, x_dtype: int) -> int:
    return lib().q4_gemm_workspace_size_dt(int(m), int(n), int(k), int(x_dtype))


# ------------------------------------------------------------ torch marshalling

def _torch():
    import torch  # imported lazily: the symbol checks above need no torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    dtype = t.dtype
    if dtype == torch.float32:
        return Q4_F32
    if dtype == torch.float16:
        return Q4_F16
    if dtype == torch.bfloat16:
        return Q4_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; libq4 takes float32, float16 or bfloat16")


def _torch_dtype(code_or_dtype):
    torch = _torch()
    if code_or_dtype in (Q4_F32, torch.float32, "f32", "float32"):
        return torch.float32
    if code_or_dtype in (Q4_F16, torch.float16, "f16", "float16"):
        return torch.float16
    raise TypeError(f"unsupported output dtype {code_or_dtype!r}")


def _stream_handle(stream, device) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def packed_shape(packed, n: Optional[int] = None, k: Optional[int] = None) -> Tuple[int, int]:
    """(n, k) of a packed weight: [n, k/32*18] uint8 unless given explicitly."""
    if n is not None and k is not None:
        return int(n), int(k)
    if packed.dim() != 2 or packed.shape[1] % BLOCK_BYTES:
        raise ValueError("packed must be [n, k/32*18] uint8, or pass n and k")
    return int(packed.shape[0]), int(packed.shape[1] // BLOCK_BYTES * QK)


def _check(status: int, what: str):
    if status != Q4_OK:
        raise Q4Error(status, what)


def q4_quantize(w, packed=None, stream=None):
    """Quantise a [n, k] fp32/fp16/bf16 device weight into a [n, k/32*18] uint8 tensor."""
    torch = _torch()
    _need_device(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be 2-D [n, k]")
    n, k = int(w.shape[0]), int(w.shape[1])
    if packed is None:
        packed = torch.empty((n, (k // QK) * BLOCK_BYTES), dtype=torch.uint8, device=w.device)
    _need_device(packed, "packed")
    _check(lib().q4_quantize(w.data_ptr(), _dtype_code(w), n, k, packed.data_ptr(),
                             _stream_handle(stream, w.device)), "q4_quantize")
    return packed


def _out(x, m, n, y, y_dtype):
    torch = _torch()
    if y is None:
        # outputs are fp32 or fp16: bf16 activations default to an fp32 output
        dflt = torch.float32 if x.dtype == torch.bfloat16 else x.dtype
        y = torch.empty((m, n), dtype=_torch_dtype(y_dtype if y_dtype is not None else dflt),
                        device=x.device)
    _need_device(y, "y")
    return y


def q4_gemv(x, packed, y=None, y_dtype=None, stream=None, n=None, k=None):
    """Batched-decode GEMV y[m, n] = x[m, k] . dequant(W)^T, 1 <= m <= 32."""
    _need_device(x, "x")
    _need_device(packed, "packed")
    n, k = packed_shape(packed, n, k)
    m = int(x.numel() // k) if x.dim() != 2 else int(x.shape[0])
    y = _out(x, m, n, y, y_dtype)
    _check(lib().q4_gemv(x.data_ptr(), _dtype_code(x), packed.data_ptr(), y.data_ptr(),
                         _dtype_code(y), m, n, k, _stream_handle(stream, x.device)), "q4_gemv")
    return y


def q4_gemm(x, packed, y=None, y_dtype=None, workspace=None, stream=None, n=None, k=None):
    """Prefill GEMM y[m, n] = x[m, k] . dequant(W)^T on fp16 MFMA (x fp16, or bf16
    staged as fp16 in the workspace)."""
    torch = _torch()
    _need_device(x, "x")
    _need_device(packed, "packed")
    n, k = packed_shape(packed, n, k)
    m = int(x.numel() // k) if x.dim() != 2 else int(x.shape[0])
    y = _out(x, m, n, y, y_dtype)
    need = q4_gemm_workspace_size_dt(m, n, k, _dtype_code(x))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().q4_gemm(x.data_ptr(), _dtype_code(x), packed.data_ptr(), y.data_ptr(),
                         _dtype_code(y), m, n, k, wptr, wbytes,
                         _stream_handle(stream, x.device)), "q4_gemm")
    return y


def q4_gemm_noalloc(x, packed, y, stream=None, n=None, k=None):
    """q4_gemm with its workspace taken from the library's fixed per-device
    scratch array (no allocation by the library; y must be given).  Calls that
    may overlap on one device race on that array."""
    _need_device(x, "x")
    _need_device(packed, "packed")
    _need_device(y, "y")
    n, k = packed_shape(packed, n, k)
    m = int(x.numel() // k) if x.dim() != 2 else int(x.shape[0])
    _check(lib().q4_gemm_noalloc(x.data_ptr(), _dtype_code(x), packed.data_ptr(), y.data_ptr(),
                                 _dtype_code(y), m, n, k, _stream_handle(stream, x.device)),
           "q4_gemm_noalloc")
    return y


# ------------------------------------------------------------ fused layers

_FAST = None  # the native short way (_q4_torch), or False where it is not built


def _fast():
    """The native module that takes ordinary calls (no y, workspace or stream of
    the caller's) the short way; None where it is not built.  It returns None
    for a call that it does not take, which then goes the full way here."""
    global _FAST
    if _FAST is None:
        L = lib()
        try:
            from . import _q4_torch
        except ImportError:
            _FAST = False
        else:
            _q4_torch.bind(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
                "q4_linear", "q4_linear_workspace_size", "q4_route", "q4_route_plan",
                "q4_route_plan_size", "q4_experts", "q4_experts_workspace_size", "q4_moe",
                "q4_moe_workspace_size")))
            _FAST = _q4_torch
    return _FAST or None


def _code(table, value, what):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {value!r}") from None


def _need_no_gradient(tensors):
    """The fused calls have no gradient: refuse tensors whose results autograd would
    take for constants."""
    torch = _torch()
    for name, t in tensors.items():
        if t is not None and (t.requires_grad and torch.is_grad_enabled()
                              or torch.autograd.forward_ad.unpack_dual(t).tangent is not None):
            raise RuntimeError(f"{name} takes part in a gradient, and this call has none; detach it or call "
                               "under torch.no_grad()")


def _same_device(x, **others):
    """Refuse host and non-contiguous tensors, tensors of several devices and ones
    that take part in a gradient; the device's index."""
    dual = getattr(_torch().autograd.forward_ad, "_current_level", 0) >= 0
    if dual or x.requires_grad or any([t is not None and t.requires_grad for t in others.values()]):
        _need_no_gradient({"x": x, **others})  # (1 us if always asked)
    _need_device(x, "x")
    index = x.get_device()
    for name, t in others.items():
        if t is not None:
            if not t.is_cuda or not t.is_contiguous():
                _need_device(t, name)
            if t.get_device() != index:
                raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    return index


def _on(stream, x):
    """A context in which `stream` (a torch stream or a handle) is the current one
    of x's device: what a call allocates then belongs to that stream, and is used
    again only by work behind the call's."""
    torch = _torch()
    _need_device(x, "x")
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=x.device) if stream
                  else torch.cuda.default_stream(x.device))
    if stream.device != x.device:
        raise ValueError(f"stream is on {stream.device}, x on {x.device}")
    return torch.cuda.stream(stream)


def _launch(index, what, fn, *args):
    """fn(*args, stream) on device `index`'s current stream, with that device current."""
    torch = _torch()
    handle = torch.cuda.current_stream(index).cuda_stream
    if torch.cuda.current_device() == index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != Q4_OK:
        raise Q4Error(status, what)


def _need_packed(packed, name="packed"):
    if packed.dtype != _torch().uint8:
        raise TypeError(f"{name} must be uint8; got {packed.dtype}")


def _full_out(y, shape, dtype, device):
    torch = _torch()
    if y is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(y.shape) != tuple(shape):
        raise ValueError(f"y must have shape {tuple(shape)}; got {tuple(y.shape)}")
    return y


def _out_dtype(y, y_dtype, x):
    torch = _torch()
    if y is not None:
        return y.dtype
    if y_dtype is None:
        return x.dtype
    if y_dtype in (Q4_BF16, torch.bfloat16, "bf16", "bfloat16"):
        return torch.bfloat16
    return _torch_dtype(y_dtype)


def _epilogue(bias, activation, gated, residual, bias_shape, y):
    if bias is not None and tuple(bias.shape) != tuple(bias_shape):
        raise ValueError(f"bias must have shape {tuple(bias_shape)}; got {tuple(bias.shape)}")
    if residual is not None and (residual.dtype != y.dtype or residual.shape != y.shape):
        raise ValueError("residual must have y's shape and dtype "
                         f"({tuple(y.shape)}, {y.dtype}); got {tuple(residual.shape)}, {residual.dtype}")
    return Epilogue(None if bias is None else bias.data_ptr(),
                    0 if bias is None else _dtype_code(bias), _code(ACTIVATIONS, activation, "activation"),
                    1 if gated else 0, None if residual is None else residual.data_ptr())


def _workspace(workspace, need, device):
    """(tensor, pointer, bytes) of a workspace: the caller's, or one allocated here."""
    torch = _torch()
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def q4_linear_workspace_size(m: int, n: int, k: int, x_dtype: int, gated: bool = False) -> int:
    return lib().q4_linear_workspace_size(int(m), int(n), int(k), int(x_dtype), int(bool(gated)))


def q4_linear(x, packed, bias=None, activation="none", gated=False, residual=None, y=None,
              y_dtype=None, workspace=None, stream=None):
    """Fused linear layer for any number of rows: z = x . dequant(packed)^T + bias,
    then act(z), or with a gate act(z[:, :n/2]) * z[:, n/2:], plus the residual.

    x [m, k] fp32, fp16 or bf16; packed [n, k/32*18] uint8; bias [n]; residual of
    y's shape and dtype (it may be y itself).  activation: none, relu, gelu (tanh
    form), gelu_erf or silu.  y defaults to x's dtype.  None of the fused calls has a
    gradient: tensors that need one are refused (RuntimeError) unless under no_grad."""
    if stream is not None:
        with _on(stream, x):
            return q4_linear(x, packed, bias, activation, gated, residual, y, y_dtype, workspace)
    if y is None and y_dtype is None and workspace is None:
        fast = _FAST or _fast()
        if fast is not None:
            out = fast.linear(x, packed, bias, ACTIVATIONS.get(activation), gated, residual)
            if out is not None:
                return out
    index = _same_device(x, packed=packed, bias=bias, residual=residual, y=y, workspace=workspace)
    _need_packed(packed)
    n, k = packed_shape(packed)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [m, {k}]; got {tuple(x.shape)}")
    m = int(x.shape[0])
    y = _full_out(y, (m, n // 2 if gated else n), _out_dtype(y, y_dtype, x), x.device)
    ep = _epilogue(bias, activation, gated, residual, (n,), y)
    xd = _dtype_code(x)
    L = lib()
    workspace, wptr, wbytes = _workspace(
        workspace, L.q4_linear_workspace_size(m, n, k, xd, ep.gated), x.device)
    _launch(index, "q4_linear", L.q4_linear, x.data_ptr(), xd, packed.data_ptr(),
            ctypes.byref(ep), y.data_ptr(), _dtype_code(y), m, n, k, wptr, wbytes)
    return y


class Plan:
    """The pairs (token, chosen expert) ordered by expert: what q4_route and
    q4_route_plan return and q4_experts takes.

    words: int32 device tensor; offsets [experts + 1] and order [m * topk] are
    views of it (expert e's pairs i * topk + j are order[offsets[e]:offsets[e + 1]];
    -1 behind the last pair that has an expert)."""

    __slots__ = ("words", "m", "topk", "experts")

    def __init__(self, words, m, topk, experts):
        self.words, self.m, self.topk, self.experts = words, m, topk, experts

    @property
    def offsets(self):
        return self.words[:self.experts + 1]

    @property
    def order(self):
        at = (self.experts + 4) // 4 * 4
        return self.words[at:at + self.m * self.topk]


def q4_route_plan_size(m: int, topk: int, experts: int) -> int:
    return lib().q4_route_plan_size(int(m), int(topk), int(experts))


def _new_plan(m, topk, experts, device):
    torch = _torch()
    size = q4_route_plan_size(m, topk, experts)
    if not size:
        raise Q4Error(Q4_ERR_SHAPE, f"plan of {m} tokens, {topk} of {experts} experts")
    return Plan(torch.empty(size // 4, dtype=torch.int32, device=device), m, topk, experts)


def _need_plan(plan):
    """Refuse words that are no plan of the Plan's sizes: the kernels go by them."""
    size = q4_route_plan_size(plan.m, plan.topk, plan.experts)
    if plan.words.dtype != _torch().int32 or not size or plan.words.numel() * 4 != size:
        raise ValueError(f"a plan of {plan.m} tokens, {plan.topk} of {plan.experts} experts is {size // 4} int32 "
                         f"words; got {plan.words.dtype} {tuple(plan.words.shape)}")


def _routing(score, bias, groups, group_topk, group_score, renormalise, scale, experts):
    torch = _torch()
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (experts,)):
        raise ValueError(f"routing bias must be float32 [{experts}]; got {bias.dtype} {tuple(bias.shape)}")
    return Routing(_code(SCORES, score, "score"), None if bias is None else bias.data_ptr(), int(groups),
                   int(group_topk), _code(GROUP_SCORES, group_score, "group_score"),
                   1 if renormalise else 0, float(scale))


def _ids_out(t, shape, dtype, device, name):
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {dtype} {shape}; got {t.dtype} {tuple(t.shape)}")
    return t


def q4_route(logits, topk, score="softmax", bias=None, groups=1, group_topk=1, group_score="max",
             renormalise=True, scale=1.0, ids=None, weights=None, stream=None):
    """Choose topk experts per token from logits [m, experts] (fp32, fp16 or bf16).

    score: softmax or sigmoid; bias [experts] fp32 is added for the choice only;
    groups > 1 keeps the experts of the group_topk best groups (group_score: max,
    or top2 for the sum of a group's two best).  Returns (ids [m, topk] int32,
    weights [m, topk] fp32, plan); ties go to the lowest index, an expert with a
    logit of -inf or NaN is not chosen, and a place without an expert is id -1,
    weight 0."""
    if stream is not None:
        with _on(stream, logits):
            return q4_route(logits, topk, score, bias, groups, group_topk, group_score, renormalise, scale, ids,
                            weights)
    if ids is None and weights is None:
        fast = _FAST or _fast()
        if fast is not None:
            out = fast.route(logits, topk, bias, SCORES.get(score), groups, group_topk,
                             GROUP_SCORES.get(group_score), renormalise, scale)
            if out is not None:
                return out[0], out[1], Plan(out[2], logits.shape[0], topk, logits.shape[1])
    torch = _torch()
    index = _same_device(logits, bias=bias, ids=ids, weights=weights)
    if logits.dim() != 2:
        raise ValueError(f"logits must be [m, experts]; got {tuple(logits.shape)}")
    m, experts, topk = int(logits.shape[0]), int(logits.shape[1]), int(topk)
    r = _routing(score, bias, groups, group_topk, group_score, renormalise, scale, experts)
    plan = _new_plan(m, topk, experts, logits.device)
    ids = _ids_out(ids, (m, topk), torch.int32, logits.device, "ids")
    weights = _ids_out(weights, (m, topk), torch.float32, logits.device, "weights")
    _launch(index, "q4_route", lib().q4_route, logits.data_ptr(), _dtype_code(logits), m, experts,
            topk, ctypes.byref(r), ids.data_ptr(), weights.data_ptr(), plan.words.data_ptr())
    return ids, weights, plan


def q4_route_plan(ids, experts, stream=None):
    """The plan of given ids [m, topk] int32; ids outside 0 .. experts - 1 name no expert."""
    if stream is not None:
        with _on(stream, ids):
            return q4_route_plan(ids, experts)
    fast = _FAST or _fast()
    if fast is not None:
        words = fast.route_plan(ids, experts)
        if words is not None:
            return Plan(words, ids.shape[0], ids.shape[1], experts)
    torch = _torch()
    index = _same_device(ids)
    if ids.dtype != torch.int32 or ids.dim() != 2:
        raise ValueError(f"ids must be int32 [m, topk]; got {ids.dtype} {tuple(ids.shape)}")
    m, topk = int(ids.shape[0]), int(ids.shape[1])
    plan = _new_plan(m, topk, int(experts), ids.device)
    _launch(index, "q4_route_plan", lib().q4_route_plan, ids.data_ptr(), m, topk, int(experts),
            plan.words.data_ptr())
    return plan


def q4_experts_workspace_size(m: int, topk: int, experts: int, n: int, k: int, x_rows: int,
                              x_dtype: int, gated: bool = False, combine: bool = False) -> int:
    return lib().q4_experts_workspace_size(int(m), int(topk), int(experts), int(n), int(k), int(x_rows),
                                           int(x_dtype), int(bool(gated)), int(bool(combine)))


def _expert_shape(packed, what="packed"):
    _need_packed(packed, what)
    if packed.dim() != 3 or packed.shape[2] % BLOCK_BYTES:
        raise ValueError(f"{what} must be [experts, n, k/32*18] uint8; got {tuple(packed.shape)}")
    return int(packed.shape[0]), int(packed.shape[1]), int(packed.shape[2]) // BLOCK_BYTES * QK


def q4_experts(x, packed, plan, bias=None, activation="none", gated=False, weights=None,
               residual=None, y=None, y_dtype=None, workspace=None, stream=None):
    """The chosen experts' products: row p = i * topk + j is
    act(x_p . dequant(packed[e])^T + bias[e]) (gated as in q4_linear) for token i's
    j-th expert e.

    x: [m, k] (a token's row goes to all its experts) or [m * topk, k] (row p);
    packed: [experts, n, k/32*18] uint8; bias: [experts, n].  Without `weights` y
    is [m * topk, nout], and rows of pairs without an expert are not written, the
    residual included: a y of the caller's keeps them, one allocated here holds
    anything in them (a second q4_experts over the plan does not read them); with weights [m, topk] fp32 y is [m, nout], the weighted
    sum over a token's experts.  The residual has y's shape and dtype."""
    if stream is not None:
        with _on(stream, x):
            return q4_experts(x, packed, plan, bias, activation, gated, weights, residual, y, y_dtype, workspace)
    if y is None and y_dtype is None and workspace is None:
        fast = _FAST or _fast()
        if fast is not None:
            out = fast.experts(x, packed, plan.words, plan.m, plan.topk, plan.experts, bias,
                               ACTIVATIONS.get(activation), gated, weights, residual)
            if out is not None:
                return out
    torch = _torch()
    _need_plan(plan)
    index = _same_device(x, packed=packed, bias=bias, plan=plan.words, weights=weights, residual=residual, y=y,
                 workspace=workspace)
    experts, n, k = _expert_shape(packed)
    m, topk = plan.m, plan.topk
    if experts != plan.experts:
        raise ValueError(f"packed has {experts} experts, the plan {plan.experts}")
    if x.dim() != 2 or x.shape[1] != k or x.shape[0] not in (m, m * topk):
        raise ValueError(f"x must be [{m} or {m * topk}, {k}]; got {tuple(x.shape)}")
    if weights is not None and (weights.dtype != torch.float32 or tuple(weights.shape) != (m, topk)):
        raise ValueError(f"weights must be float32 [{m}, {topk}]; got {weights.dtype} {tuple(weights.shape)}")
    x_rows = int(x.shape[0])
    y = _full_out(y, (m if weights is not None else m * topk, n // 2 if gated else n),
                  _out_dtype(y, y_dtype, x), x.device)
    ep = _epilogue(bias, activation, gated, residual, (experts, n), y)
    xd = _dtype_code(x)
    L = lib()
    workspace, wptr, wbytes = _workspace(
        workspace, L.q4_experts_workspace_size(m, topk, experts, n, k, x_rows, xd, ep.gated,
                                               0 if weights is None else 1), x.device)
    _launch(index, "q4_experts", L.q4_experts, x.data_ptr(), xd, x_rows, packed.data_ptr(),
            ctypes.byref(ep), plan.words.data_ptr(), None if weights is None else weights.data_ptr(),
            y.data_ptr(), _dtype_code(y), m, topk, experts, n, k, wptr, wbytes)
    return y


def q4_moe_workspace_size(m: int, topk: int, experts: int, hidden: int, inter: int, x_dtype: int,
                          gated: bool = True) -> int:
    return lib().q4_moe_workspace_size(int(m), int(topk), int(experts), int(hidden), int(inter),
                                       int(x_dtype), int(bool(gated)))


def q4_moe(x, logits, up, down, topk, activation="silu", gated=True, up_bias=None, down_bias=None,
           residual=None, score="softmax", route_bias=None, groups=1, group_topk=1, group_score="max",
           renormalise=True, scale=1.0, ids=None, weights=None, y=None, y_dtype=None, workspace=None,
           stream=None):
    """A whole expert layer in one call: route the tokens by logits [m, experts], run
    x [m, hidden] through the chosen experts' `up` ([experts, 2 * inter, ..] gated,
    else [experts, inter, ..]; gate rows first) and `down` ([experts, hidden, ..]),
    and add the rows up by the routing weights, plus the residual.  The rows between
    the products have x's dtype.  Routing options as in q4_route; ids and weights
    receive the routing if given."""
    if stream is not None:
        with _on(stream, x):
            return q4_moe(x, logits, up, down, topk, activation, gated, up_bias, down_bias, residual, score,
                          route_bias, groups, group_topk, group_score, renormalise, scale, ids, weights, y,
                          y_dtype, workspace)
    if y is None and y_dtype is None and workspace is None and ids is None and weights is None:
        fast = _FAST or _fast()
        if fast is not None:
            out = fast.moe(x, logits, up, down, topk, ACTIVATIONS.get(activation), gated, up_bias,
                           down_bias, residual, route_bias, SCORES.get(score), groups, group_topk,
                           GROUP_SCORES.get(group_score), renormalise, scale)
            if out is not None:
                return out
    torch = _torch()
    index = _same_device(x, logits=logits, up=up, down=down, up_bias=up_bias, down_bias=down_bias,
                 residual=residual, route_bias=route_bias, ids=ids, weights=weights, y=y,
                 workspace=workspace)
    experts, nup, hidden = _expert_shape(up, "up")
    e2, n2, inter = _expert_shape(down, "down")
    if e2 != experts or n2 != hidden or nup != (2 * inter if gated else inter):
        raise ValueError(f"up [{experts}, {nup}, k = {hidden}] and down [{e2}, {n2}, k = {inter}] do not match")
    if x.dim() != 2 or x.shape[1] != hidden:
        raise ValueError(f"x must be [m, {hidden}]; got {tuple(x.shape)}")
    m, topk = int(x.shape[0]), int(topk)
    if tuple(logits.shape) != (m, experts):
        raise ValueError(f"logits must be [{m}, {experts}]; got {tuple(logits.shape)}")
    r = _routing(score, route_bias, groups, group_topk, group_score, renormalise, scale, experts)
    for t, dt, name in ((ids, torch.int32, "ids"), (weights, torch.float32, "weights")):
        if t is not None:
            _ids_out(t, (m, topk), dt, x.device, name)
    y = _full_out(y, (m, hidden), _out_dtype(y, y_dtype, x), x.device)
    if up_bias is not None and tuple(up_bias.shape) != (experts, nup):
        raise ValueError(f"up_bias must have shape {(experts, nup)}; got {tuple(up_bias.shape)}")
    up_ep = Epilogue(None if up_bias is None else up_bias.data_ptr(),
                     0 if up_bias is None else _dtype_code(up_bias),
                     _code(ACTIVATIONS, activation, "activation"), 1 if gated else 0, None)
    down_ep = _epilogue(down_bias, "none", False, residual, (experts, hidden), y)
    xd = _dtype_code(x)
    L = lib()
    workspace, wptr, wbytes = _workspace(
        workspace, L.q4_moe_workspace_size(m, topk, experts, hidden, inter, xd, up_ep.gated), x.device)
    _launch(index, "q4_moe", L.q4_moe, x.data_ptr(), xd, logits.data_ptr(), _dtype_code(logits),
            ctypes.byref(r), up.data_ptr(), ctypes.byref(up_ep), down.data_ptr(), ctypes.byref(down_ep),
            y.data_ptr(), _dtype_code(y), m, topk, experts, hidden, inter,
            None if ids is None else ids.data_ptr(), None if weights is None else weights.data_ptr(), wptr,
            wbytes)
    return y
