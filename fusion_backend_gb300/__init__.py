"""Python binding of libmoe_ffn.so, the fused MoE FFN layer for GB300.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current CUDA stream.  The
functions carry the names of the C ABI in ``include/moe_ffn.h``.

There is no CPU fallback: if the library has not been built, or the device is
not a GB300 (sm_103), the calls raise.
"""

from __future__ import annotations

import ctypes
import numbers
import os
from dataclasses import dataclass

from . import _build

LIB_PATH = _build.LIB

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_MISALIGNED = -4
ERR_CUDA = -5
ERR_TIMEOUT = -6
ERR_DEVICE = -7

ACT_F32 = 0
ACT_BF16 = 1
ACT_F16 = 2
W_BF16 = 0
W_Q4B32 = 1
W_I8 = 2

QUERY_PATH = 0
QUERY_LAUNCHES_PER_EXECUTE = 1
QUERY_TWO_STREAM_WORKSPACE = 2

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
GROUP_MAX = 0
GROUP_TOP2 = 1
GATE_LINEAR = 0
GATE_SIGMOID = 1

EXPORTS = (
    "moe_ffn_prepare",
    "moe_ffn_execute",
    "moe_ffn_execute_ex",
    "moe_ffn_execute_block",
    "moe_ffn_read_status",
    "moe_ffn_read_routing",
    "moe_ffn_probe_timeout",
    "moe_ffn_query",
    "moe_ffn_destroy",
    "moe_ffn_strerror",
    "moe_ffn_execute_static_scratch",
    "moe_ffn_last_cuda_error",
    "moe_ffn_execute_two_stream",
    "moe_ffn_execute_routed",
    "moe_ffn_route",
    "moe_ffn_norm_residual",
    "moe_ffn_adapters_workspace",
    "moe_ffn_add_adapters",
    "moe_ffn_project",
    "moe_ffn_append_kv",
    "moe_ffn_attend_workspace",
    "moe_ffn_attend",
)

STATIC_SCRATCH_BYTES = 1 << 24


class MoeFFNError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} ({status})")
        self.status = status


class Shapes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "top_k", "I", "Is")]


class DType(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("wfmt", ctypes.c_int32)]


def _fields(i32="", f32="", i64=""):
    return [(n, t) for names, t in ((i32, ctypes.c_int32), (f32, ctypes.c_float), (i64, ctypes.c_int64))
            for n in names.split()]


def _block(cls, *values):
    """An argument block; ctypes would take a number past a field's 32 bits modulo 2^32."""
    for (name, kind), v in zip(cls._fields_, values):
        if kind is ctypes.c_int32 and not -(2**31) <= v < 2**31:
            raise ValueError(f"{name}: {v} does not fit in 32 bits")
    return cls(*values)


class RouteArgs(ctypes.Structure):
    _fields_ = _fields("T E top_k score groups top_groups group_score renorm dtype", "scale", "row_stride")


class NormArgs(ctypes.Structure):
    _fields_ = _fields("T H y_dtype res_dtype normed_dtype gate_dtype w_post_dtype w_pre_dtype post_norm gate_layout "
                       "gate_sigmoid", "alpha beta w_offset eps",
                       "y_stride res_stride res_out_stride normed_stride gate_stride")


class AdaptersArgs(ctypes.Structure):
    _fields_ = _fields("T K N R n_adapters x_dtype y_dtype", "", "x_stride y_stride out_stride")


class ProjectArgs(ctypes.Structure):
    _fields_ = _fields("T K N group x_dtype y_dtype", "", "x_stride y_stride w_stride")


_CACHES = "kc_page_stride kc_slot_stride kc_head_stride vc_page_stride vc_slot_stride vc_head_stride"


class AppendArgs(ctypes.Structure):
    _fields_ = _fields("T q_heads kv_heads D rot interleaved x_dtype q_out_dtype cache_dtype page_size pages", "scale",
                       "q_stride q_head_stride k_stride k_head_stride v_stride v_head_stride q_out_stride "
                       f"q_out_head_stride {_CACHES}")


class AttendArgs(ctypes.Structure):
    _fields_ = _fields("T B q_heads kv_heads D dtype out_dtype page_size pages max_pages mask_words", "scale softcap",
                       f"q_stride q_head_stride out_stride out_head_stride {_CACHES} table_stride mask_stride")


_lib = None


def build(force: bool = False) -> str:
    """Compile the library for sm_103a (nvcc) if it is missing or stale."""
    return _build.build(force=force)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run fusion_backend_gb300.build() first")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.moe_ffn_prepare.restype = ctypes.c_int
        L.moe_ffn_prepare.argtypes = [ctypes.POINTER(Shapes), DType, ctypes.POINTER(vp), ctypes.POINTER(sz)]
        L.moe_ffn_execute.restype = ctypes.c_int
        L.moe_ffn_execute.argtypes = [vp, vp, vp, sz, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_execute_ex.restype = ctypes.c_int
        L.moe_ffn_execute_ex.argtypes = [vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_execute_block.restype = ctypes.c_int
        L.moe_ffn_execute_block.argtypes = [vp, vp, vp, sz, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
        L.moe_ffn_read_status.restype = ctypes.c_int
        L.moe_ffn_read_status.argtypes = [vp, vp, vp, ctypes.POINTER(i32)]
        L.moe_ffn_read_routing.restype = ctypes.c_int
        L.moe_ffn_read_routing.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(i32)]
        L.moe_ffn_query.restype = ctypes.c_int
        L.moe_ffn_query.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int64)]
        L.moe_ffn_destroy.restype = None
        L.moe_ffn_destroy.argtypes = [vp]
        L.moe_ffn_execute_static_scratch.restype = ctypes.c_int
        L.moe_ffn_execute_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_strerror.restype = ctypes.c_char_p
        L.moe_ffn_strerror.argtypes = [ctypes.c_int]
        L.moe_ffn_probe_timeout.restype = ctypes.c_int
        L.moe_ffn_probe_timeout.argtypes = [vp, vp, vp, sz, i32]
        L.moe_ffn_last_cuda_error.restype = ctypes.c_char_p
        L.moe_ffn_last_cuda_error.argtypes = []
        L.moe_ffn_execute_two_stream.restype = ctypes.c_int
        L.moe_ffn_execute_two_stream.argtypes = [vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_execute_routed.restype = ctypes.c_int
        L.moe_ffn_execute_routed.argtypes = [vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_route.restype = ctypes.c_int
        L.moe_ffn_route.argtypes = [ctypes.POINTER(RouteArgs), vp, vp, vp, vp, vp]
        L.moe_ffn_norm_residual.restype = ctypes.c_int
        L.moe_ffn_norm_residual.argtypes = [ctypes.POINTER(NormArgs), vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_adapters_workspace.restype = ctypes.c_int
        L.moe_ffn_adapters_workspace.argtypes = [ctypes.POINTER(AdaptersArgs), ctypes.POINTER(sz)]
        L.moe_ffn_add_adapters.restype = ctypes.c_int
        L.moe_ffn_add_adapters.argtypes = [ctypes.POINTER(AdaptersArgs), vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_ffn_project.restype = ctypes.c_int
        L.moe_ffn_project.argtypes = [ctypes.POINTER(ProjectArgs), vp, vp, vp, vp, vp]
        L.moe_ffn_append_kv.restype = ctypes.c_int
        L.moe_ffn_append_kv.argtypes = [ctypes.POINTER(AppendArgs)] + 10 * [vp]
        L.moe_ffn_attend_workspace.restype = ctypes.c_int
        L.moe_ffn_attend_workspace.argtypes = [ctypes.POINTER(AttendArgs), ctypes.POINTER(sz)]
        L.moe_ffn_attend.restype = ctypes.c_int
        L.moe_ffn_attend.argtypes = [ctypes.POINTER(AttendArgs), vp, vp, sz] + 9 * [vp]
        _lib = L
    return _lib


def strerror(status: int) -> str:
    try:
        return lib().moe_ffn_strerror(status).decode()
    except RuntimeError:
        return f"status {status}"


def _check(status: int, what: str) -> None:
    if status != OK:
        if status == ERR_CUDA:
            what = f"{what} [{lib().moe_ffn_last_cuda_error().decode()}]"
        raise MoeFFNError(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------------------------
# Functions with the C ABI names (raise MoeFFNError on a non-zero status)


def moe_ffn_prepare(shapes, act: int, wfmt: int):
    """Return (plan handle, workspace bytes).  Host only."""
    s = Shapes(shapes.T, shapes.H, shapes.E, shapes.top_k, shapes.I, shapes.Is)
    plan = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib().moe_ffn_prepare(ctypes.byref(s), DType(act, wfmt), ctypes.byref(plan), ctypes.byref(ws)),
           "moe_ffn_prepare")
    return plan.value, ws.value


def moe_ffn_execute(plan, workspace, x, router_w, expert_w, shexp_w, shexp_gate_w, out, stream=None,
                    workspace_bytes=None):
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _check(lib().moe_ffn_execute(plan, _stream(stream), _ptr(workspace), nbytes, _ptr(x), _ptr(router_w),
                                 _ptr(expert_w), _ptr(shexp_w), _ptr(shexp_gate_w), _ptr(out)), "moe_ffn_execute")


def moe_ffn_execute_ex(plan, workspace, x, router_w, expert_w, shexp_w, shexp_gate_w, out, topk_ids=None,
                       topk_w=None, stream=None, workspace_bytes=None):
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _check(lib().moe_ffn_execute_ex(plan, _stream(stream), _ptr(workspace), nbytes, _ptr(x), _ptr(router_w),
                                    _ptr(expert_w), _ptr(shexp_w), _ptr(shexp_gate_w), _ptr(out), _ptr(topk_ids),
                                    _ptr(topk_w)), "moe_ffn_execute_ex")


def moe_ffn_execute_block(plan, workspace, x_res, router_w, expert_w, shexp_w, shexp_gate_w, eps=1e-6,
                          topk_ids=None, topk_w=None, stream=None, workspace_bytes=None):
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _check(lib().moe_ffn_execute_block(plan, _stream(stream), _ptr(workspace), nbytes, _ptr(x_res), _ptr(router_w),
                                       _ptr(expert_w), _ptr(shexp_w), _ptr(shexp_gate_w), eps, _ptr(topk_ids),
                                       _ptr(topk_w)), "moe_ffn_execute_block")


def moe_ffn_read_status(plan, workspace, stream=None) -> int:
    st = ctypes.c_int32()
    _check(lib().moe_ffn_read_status(plan, _ptr(workspace), _stream(stream), ctypes.byref(st)), "moe_ffn_read_status")
    return st.value


def moe_ffn_read_routing(plan, workspace, E: int, T: int, top_k: int, stream=None):
    import numpy as np

    counts = np.zeros(E, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    perm = np.zeros(T * top_k, np.int32)
    active = np.zeros(E, np.int32)
    n = ctypes.c_int32()
    _check(lib().moe_ffn_read_routing(plan, _ptr(workspace), _stream(stream), counts.ctypes.data, offsets.ctypes.data,
                                      perm.ctypes.data, active.ctypes.data, ctypes.byref(n)), "moe_ffn_read_routing")
    return counts, offsets, perm, active[: n.value].copy()


def moe_ffn_probe_timeout(plan, workspace, which: int, stream=None, workspace_bytes=None) -> None:
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _check(lib().moe_ffn_probe_timeout(plan, _stream(stream), _ptr(workspace), nbytes, which), "moe_ffn_probe_timeout")


def moe_ffn_query(plan, what: int) -> int:
    v = ctypes.c_int64()
    _check(lib().moe_ffn_query(plan, what, ctypes.byref(v)), "moe_ffn_query")
    return v.value


def moe_ffn_destroy(plan) -> None:
    if plan:
        lib().moe_ffn_destroy(plan)


def moe_ffn_execute_static_scratch(plan, x, router_w, expert_w, shexp_w, shexp_gate_w, out, stream=None):
    """moe_ffn_execute without a workspace: the scratch is the library's own
    device array (STATIC_SCRATCH_BYTES).  Allocates nothing.  Calls that overlap
    on the GPU share that array and race; serialise them."""
    _check(lib().moe_ffn_execute_static_scratch(plan, _stream(stream), _ptr(x), _ptr(router_w), _ptr(expert_w),
                                                _ptr(shexp_w), _ptr(shexp_gate_w), _ptr(out)),
           "moe_ffn_execute_static_scratch")


def moe_ffn_execute_two_stream(plan, workspace, x, router_w, expert_w, shexp_w, shexp_gate_w, out, aux_stream=None,
                               fork_event=None, join_event=None, stream=None, workspace_bytes=None):
    """The layer as two branches on two streams joined by an add (routed on ``stream``, the gated shared expert
    on ``aux_stream``, torch.cuda.Event objects or raw handles as the fork and join events); with no aux stream the
    same kernels run one after the other on ``stream``."""
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    ev = lambda e: None if e is None else (e if isinstance(e, int) else e.cuda_event)
    _check(lib().moe_ffn_execute_two_stream(plan, _stream(stream), None if aux_stream is None else _stream(aux_stream),
                                            ev(fork_event), ev(join_event), _ptr(workspace), nbytes, _ptr(x),
                                            _ptr(router_w), _ptr(expert_w), _ptr(shexp_w), _ptr(shexp_gate_w),
                                            _ptr(out)), "moe_ffn_execute_two_stream")


def moe_ffn_execute_routed(plan, workspace, x, ids, weights, expert_w, shexp_w, shexp_gate_w, out, stream=None,
                           workspace_bytes=None):
    """The layer for a routing that the caller brings: ``ids`` int32 and ``weights`` fp32 [T, top_k], an id outside
    0..E-1 dropping the choice.  shexp_gate_w None: the shared expert is not gated; shexp_w None: no shared expert."""
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _check(lib().moe_ffn_execute_routed(plan, _stream(stream), _ptr(workspace), nbytes, _ptr(x), _ptr(ids),
                                        _ptr(weights), _ptr(expert_w), _ptr(shexp_w), _ptr(shexp_gate_w), _ptr(out)),
           "moe_ffn_execute_routed")


# ----------------------------------------------------------------------------
# Operators around the layer.  Types, layouts and strides come from the
# tensors: matrices [rows, columns] with adjacent columns, in rows of any
# stride; a tensor of another type, shape or device raises ValueError.  Outputs
# that are not given are allocated on the call's stream.
#
# The checks and the argument block depend on the tensors' shapes, strides,
# types and device alone, so a block is built once per such signature (never
# per tensor) and found again in _blocks: a call of a few microseconds on the
# GPU would otherwise wait for 10 microseconds of Python.


_CODES: dict = {}
_blocks: dict = {}
_torch_c = None


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _by_value(v) -> bool:
    return v is None or isinstance(v, (numbers.Number, tuple)) or type(v).__name__ == "dtype"


def _flat(t):
    """The signature of a tensor whose shape does not matter (an address has none)."""
    return None if t is None else 0 if isinstance(t, int) else (t.is_contiguous(), t.nbytes, t.dtype, t.get_device())


def _remember(key, block):
    # a number held in a tensor is found by the tensor's identity and may change: its block serves one call
    if all(_by_value(v) for v in key):
        if len(_blocks) >= 4096:
            _blocks.clear()
        _blocks[key] = block
    return block


def _raw_stream(stream, t) -> int | None:
    """The call's stream; the library launches on the current device, so t has to be there."""
    global _torch_c
    if _torch_c is None:
        import torch

        _torch_c = torch._C
    device, current = t.get_device(), _torch_c._cuda_getDevice()
    if device != current:
        raise ValueError(f"the call's tensors are on cuda:{device}, the current device is cuda:{current}")
    return _torch_c._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _code(t, name: str, allowed=(ACT_F32, ACT_BF16, ACT_F16)) -> int:
    if not _CODES:
        import torch

        _CODES.update({torch.float32: ACT_F32, torch.bfloat16: ACT_BF16, torch.float16: ACT_F16})
    c = _CODES.get(t.dtype)
    if c not in allowed:
        raise ValueError(f"{name}: dtype {t.dtype} is not supported")
    return c


def _require(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _matrix(t, rows: int, cols: int, name: str) -> int:
    """Row stride of t, a [rows, cols] tensor with adjacent columns."""
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({rows}, {cols})")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns of a row must be adjacent")
    # a single row has no stride of its own (the tensor's may be anything)
    return t.stride(0) if rows > 1 else cols


def _whole(t, shape, dtype, name: str) -> None:
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _on_device(first, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != first.device):
            raise ValueError(f"{name}: must be on the call's CUDA device")


def _new(stream, shape, dtype, device, zero=False):
    """A tensor allocated (and filled with zeros) on the stream that the call runs on."""
    import torch

    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return make(shape, dtype=dtype, device=device)


def _route_block(logits, top_k, bias, score, groups, top_groups, group_score, renorm, scale, ids, weights):
    import torch

    _require(logits.dim() == 2, "logits: expected [T, E]")
    T, E = logits.shape
    a = _block(RouteArgs, T, E, top_k, score, groups, top_groups, group_score, bool(renorm), _code(logits, "logits"),
               scale, _matrix(logits, T, E, "logits"))
    if bias is not None:
        _whole(bias, (E,), torch.float32, "bias")
    if ids is not None:
        _whole(ids, (T, top_k), torch.int32, "ids")
    if weights is not None:
        _whole(weights, (T, top_k), torch.float32, "weights")
    _on_device(logits, logits=logits, bias=bias, ids=ids, weights=weights)
    return a


def moe_ffn_route(logits, top_k: int, bias=None, score: int = SCORE_SOFTMAX, groups: int = 1, top_groups: int = 1,
                  group_score: int = GROUP_MAX, renorm: bool = True, scale: float = 1.0, ids=None, weights=None,
                  stream=None):
    """Experts (int32 [T, top_k], best first, -1 where none is left) and weights (fp32 [T, top_k]) of every row of
    ``logits`` [T, E]; the scores, the balance ``bias`` [E], the groups and the weights as in ``moe_ffn_route`` of
    ``include/moe_ffn.h``.  Returns (ids, weights)."""
    key = (0, _sig(logits), top_k, _sig(bias), score, groups, top_groups, group_score, renorm, scale, _sig(ids),
           _sig(weights))
    a = _blocks.get(key) or _remember(key, _route_block(logits, top_k, bias, score, groups, top_groups, group_score,
                                                        renorm, scale, ids, weights))
    if ids is None or weights is None:
        import torch

        shape = (a.T, max(top_k, 0))
        ids = _new(stream, shape, torch.int32, logits.device) if ids is None else ids
        weights = _new(stream, shape, torch.float32, logits.device) if weights is None else weights
    rc = (_lib or lib()).moe_ffn_route(a, _raw_stream(stream, logits), logits.data_ptr(),
                                       None if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr())
    if rc:
        _check(rc, "moe_ffn_route")
    return ids, weights


def _norm_block(res, y, post_norm, w_post, gate, gate_act, alpha, beta, w_pre, w_offset, eps, res_out, normed,
                norm_dtype):
    _require(res.dim() == 2, "res: expected [T, H]")
    T, H = res.shape
    _require(res_out.dtype == res.dtype, "res_out: must have res's dtype")
    rd, rs, os_ = _code(res, "res"), _matrix(res, T, H, "res"), _matrix(res_out, T, H, "res_out")
    yd, ys = (_code(y, "y"), _matrix(y, T, H, "y")) if y is not None else (ACT_F32, H)
    layout, gd, gs = 0, ACT_F32, H
    if gate is not None:
        gd = _code(gate, "gate")
        if gate.dim() == 1:
            _whole(gate, (H,), gate.dtype, "gate")
        elif tuple(gate.shape) == (T, 1):
            layout, gs = 1, gate.stride(0) if T > 1 else 1
        else:
            layout, gs = 2, _matrix(gate, T, H, "gate")
    codes = []
    for w, name in ((w_post, "w_post"), (w_pre, "w_pre")):
        codes.append(ACT_F32 if w is None else _code(w, name, (ACT_F32, ACT_BF16)))
        if w is not None:
            _whole(w, (H,), w.dtype, name)
    nd, ns = ACT_BF16, H
    if normed is not None:
        _require(norm_dtype is None or norm_dtype == normed.dtype, "normed: not of norm_dtype")
        nd, ns = _code(normed, "normed"), _matrix(normed, T, H, "normed")
    elif norm_dtype is not None:
        _code(res, "res")
        _require(norm_dtype in _CODES, f"norm_dtype: {norm_dtype} is not supported")
        nd = _CODES[norm_dtype]
    _on_device(res, res=res, y=y, w_post=w_post, gate=gate, w_pre=w_pre, res_out=res_out, normed=normed)
    return _block(NormArgs, T, H, yd, rd, nd, gd, codes[0], codes[1], bool(post_norm), layout,
                  gate_act == GATE_SIGMOID, alpha, beta, w_offset, eps, ys, rs, os_, ns, gs)


def moe_ffn_norm_residual(res, y=None, post_norm: bool = False, w_post=None, gate=None, gate_act: int = GATE_LINEAR,
                          alpha: float = 1.0, beta: float = 1.0, w_pre=None, w_offset: float = 0.0,
                          eps: float = 1e-6, res_out=None, normed=None, norm_dtype=None, stream=None):
    """``res_out = alpha res + beta a(gate) z``, z being the block's output ``y`` or (``post_norm``) its RMSNorm, and
    ``normed``, the RMSNorm of res_out for the next block (see ``include/moe_ffn.h``).  ``gate``: [H] per channel,
    [T, 1] per token or [T, H].  res_out defaults to ``res`` (in place; not written where ``y`` is None and alpha is
    1), normed to a new tensor of ``norm_dtype`` (bf16).  Returns (res_out, normed)."""
    if res_out is None:
        res_out = res
    key = (1, _sig(res), _sig(y), post_norm, _sig(w_post), _sig(gate), gate_act, alpha, beta, _sig(w_pre), w_offset,
           eps, _sig(res_out), _sig(normed), norm_dtype)
    a = _blocks.get(key) or _remember(key, _norm_block(res, y, post_norm, w_post, gate, gate_act, alpha, beta, w_pre,
                                                       w_offset, eps, res_out, normed, norm_dtype))
    if normed is None:
        import torch

        normed = _new(stream, (a.T, a.H), norm_dtype or torch.bfloat16, res.device)
    unchanged = y is None and alpha == 1.0 and res_out is res
    rc = (_lib or lib()).moe_ffn_norm_residual(
        a, _raw_stream(stream, res), res.data_ptr(), None if y is None else y.data_ptr(),
        None if w_post is None else w_post.data_ptr(), None if gate is None else gate.data_ptr(),
        None if w_pre is None else w_pre.data_ptr(), None if unchanged else res_out.data_ptr(), normed.data_ptr())
    if rc:
        _check(rc, "moe_ffn_norm_residual")
    return res_out, normed


def moe_ffn_adapters_workspace(T: int, K: int, N: int, R: int) -> int:
    """Workspace bytes of moe_ffn_add_adapters for T tokens, widths K and N and a pool of rank R."""
    n = ctypes.c_size_t()
    a = _block(AdaptersArgs, T, K, N, R, 0, ACT_BF16, ACT_F32, (K + 7) // 8 * 8, N, N)
    _check(lib().moe_ffn_adapters_workspace(a, ctypes.byref(n)), "moe_ffn_adapters_workspace")
    return max(n.value, 256)


def _adapters_block(y, x, adapter_ids, a, b, ranks, scales, out, workspace):
    import torch

    _require(x.dim() == 2 and y.dim() == 2 and a.dim() == 3 and b.dim() == 3,
             "expected x [T, K], y [T, N], a [n, R, K], b [n, N, R]")
    T, K = x.shape
    n, R = a.shape[:2]
    N = b.shape[1]
    xd = _code(x, "x", (ACT_BF16, ACT_F16))
    _whole(a, (n, R, K), x.dtype, "a")
    _whole(b, (n, N, R), x.dtype, "b")
    _whole(adapter_ids, (T,), torch.int32, "adapter_ids")
    _require(out.dtype == y.dtype, "out: must have y's dtype")
    if ranks is not None:
        _whole(ranks, (n,), torch.int32, "ranks")
    if scales is not None:
        _whole(scales, (n,), torch.float32, "scales")
    xs = _matrix(x, T, K, "x")
    args = _block(AdaptersArgs, T, K, N, R, n, xd, _code(y, "y"), xs if T > 1 else (K + 7) // 8 * 8,
                  _matrix(y, T, N, "y"), _matrix(out, T, N, "out"))
    _on_device(x, x=x, y=y, adapter_ids=adapter_ids, a=a, b=b, ranks=ranks, scales=scales, out=out,
               workspace=workspace)
    if workspace is not None:
        _require(workspace.is_contiguous(), "workspace: must be contiguous")
    return args


def moe_ffn_add_adapters(y, x, adapter_ids, a, b, ranks=None, scales=None, out=None, workspace=None, stream=None):
    """``out_t = y_t + scales_i b_i (a_i x_t)`` with i = ``adapter_ids[t]`` (int32 [T]; -1: no adapter).  x [T, K],
    y [T, N], a [n, R, K], b [n, N, R], ranks int32 [n], scales fp32 [n] (see ``include/moe_ffn.h``).  out defaults to
    y (in place), the workspace (a tensor of moe_ffn_adapters_workspace bytes) to a new one.  Returns out."""
    if out is None:
        out = y
    key = (2, _sig(y), _sig(x), _sig(adapter_ids), _sig(a), _sig(b), _sig(ranks), _sig(scales), _sig(out),
           _sig(workspace))
    args = _blocks.get(key) or _remember(key, _adapters_block(y, x, adapter_ids, a, b, ranks, scales, out, workspace))
    if workspace is None:
        import torch

        workspace = _new(stream, (moe_ffn_adapters_workspace(args.T, args.K, args.N, args.R),), torch.uint8, x.device)
    rc = (_lib or lib()).moe_ffn_add_adapters(
        args, _raw_stream(stream, x), workspace.data_ptr(), workspace.numel() * workspace.element_size(), x.data_ptr(),
        adapter_ids.data_ptr(), a.data_ptr(), b.data_ptr(), None if ranks is None else ranks.data_ptr(),
        None if scales is None else scales.data_ptr(), y.data_ptr(), out.data_ptr())
    if rc:
        _check(rc, "moe_ffn_add_adapters")
    return out


# ----------------------------------------------------------------------------
# The attention half of a block: products with 4-bit weights, the paged cache
# and attention over it.  Heads are [tokens, heads, D] tensors with adjacent
# elements of a head, caches [pages, page_size, kv_heads, D]; other strides are
# free (a transposed cache whose pages hold their heads one behind the other
# included).


def _project_block(x, w, group, bias, out):
    import torch

    _require(x.dim() == 2 and w.dim() == 2, "expected x [T, K], w [N, row bytes]")
    _require(group in (32, 64, 128), f"group: {group}, expected 32, 64 or 128")
    T, K = x.shape
    N = w.shape[0]
    _require(w.dtype == torch.uint8, f"w: dtype {w.dtype}, expected uint8 rows of codes and scales")
    _require(K % group == 0, f"x: {K} columns are no multiple of the group")
    need = K // 2 + 2 * (K // group)
    _require(w.shape[1] >= need, f"w: rows of {w.shape[1]} bytes, expected {need}")
    _require(w.stride(1) == 1, "w: the bytes of a row must be adjacent")
    if bias is not None:
        _whole(bias, (N,), torch.float32, "bias")
    xs = _matrix(x, T, K, "x")
    a = _block(ProjectArgs, T, K, N, group, _code(x, "x", (ACT_BF16, ACT_F16)), _code(out, "out"),
               xs if T > 1 else (K + 7) // 8 * 8, _matrix(out, T, N, "out"),
               w.stride(0) if N > 1 else (need + 15) // 16 * 16)
    _on_device(x, x=x, w=w, bias=bias, out=out)
    return a


def moe_ffn_project(x, w, group: int = 32, bias=None, out=None, out_dtype=None, stream=None):
    """``out = x W^T + bias`` for few tokens: x [T, K] bf16 or fp16, w uint8 [N, row bytes] in rows of K/2 bytes of
    4-bit codes and K/group fp16 scales (the layer's 4-bit rows with group 32; see ``include/moe_ffn.h``), bias fp32
    [N].  out [T, N] defaults to a new tensor of ``out_dtype`` (x's type).  Returns out."""
    if out is None:
        _require(x.dim() == 2 and w.dim() == 2, "expected x [T, K], w [N, row bytes]")
        out = _new(stream, (x.shape[0], w.shape[0]), out_dtype or x.dtype, x.device)
    else:
        _require(out_dtype is None or out_dtype == out.dtype, "out: not of out_dtype")
    key = (3, x.shape, x.stride(), x.dtype, x.get_device(), w.shape, w.stride(), w.dtype, w.get_device(), group,
           _sig(bias), out.shape, out.stride(), out.dtype, out.get_device())
    a = _blocks.get(key) or _remember(key, _project_block(x, w, group, bias, out))
    rc = (_lib or lib()).moe_ffn_project(a, _raw_stream(stream, x), x.data_ptr(), w.data_ptr(),
                                         None if bias is None else bias.data_ptr(), out.data_ptr())
    if rc:
        _check(rc, "moe_ffn_project")
    return out


def _heads(t, T: int, H: int, D: int, name: str):
    """Token and head strides of t, a [T, H, D] tensor with adjacent elements of a head."""
    if tuple(t.shape) != (T, H, D):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({T}, {H}, {D})")
    if D > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    # a single token or head has no stride of its own
    return t.stride(0) if T > 1 else H * D, t.stride(1) if H > 1 else D


def _cache_strides(t, shape, name: str):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    own = (shape[3] + 7) // 8 * 8
    return tuple(t.stride(i) if shape[i] > 1 else own for i in range(3))


def _append_block(k, v, positions, slots, inv_freq, k_cache, v_cache, q, q_out, interleaved, scale):
    import torch

    _require(k.dim() == 3 and k_cache.dim() == 4, "expected k [T, kv_heads, D], k_cache [pages, page_size, kv_heads, D]")
    T, Hkv, D = k.shape
    pages, page_size = k_cache.shape[:2]
    shape = (pages, page_size, Hkv, D)
    _require(v.dtype == k.dtype and (q is None or q.dtype == k.dtype), "q, k, v: must have one dtype")
    _require(v_cache.dtype == k_cache.dtype, "k_cache, v_cache: must have one dtype")
    _require((q is None) == (q_out is None), "q_out: given without q")
    _whole(positions, (T,), torch.int32, "positions")
    _whole(slots, (T,), torch.int32, "slots")
    rot = 0
    if inv_freq is not None:
        _require(inv_freq.dim() == 1, "inv_freq: expected [rot / 2]")
        rot = 2 * inv_freq.shape[0]
        _whole(inv_freq, (rot // 2,), torch.float32, "inv_freq")
        _require(rot <= D, f"inv_freq: {rot} rotated elements of heads of {D}")
    Hq, qs, qos, qod = 0, (D, D), (D, D), ACT_F32
    if q is not None:
        _require(q.dim() == 3, "q: expected [T, q_heads, D]")
        Hq = q.shape[1]
        qs, qos, qod = _heads(q, T, Hq, D, "q"), _heads(q_out, T, Hq, D, "q_out"), _code(q_out, "q_out")
    a = _block(AppendArgs, T, Hq, Hkv, D, rot, bool(interleaved), _code(k, "k"), qod, _code(k_cache, "k_cache"),
               page_size, pages, scale, *qs, *_heads(k, T, Hkv, D, "k"), *_heads(v, T, Hkv, D, "v"), *qos,
               *_cache_strides(k_cache, shape, "k_cache"), *_cache_strides(v_cache, shape, "v_cache"))
    _on_device(k, k=k, v=v, positions=positions, slots=slots, inv_freq=inv_freq, k_cache=k_cache, v_cache=v_cache, q=q,
               q_out=q_out)
    return a


def moe_ffn_append_kv(k, v, positions, slots, inv_freq, k_cache, v_cache, q=None, q_out=None,
                      interleaved: bool = False, scale: float = 1.0, stream=None):
    """k and v [T, kv_heads, D] into the caches [pages, page_size, kv_heads, D] at ``slots`` (int32 [T], page *
    page_size + slot, -1: padding), k and q [T, q_heads, D] rotated by ``positions`` (int32 [T]) times ``inv_freq``
    (fp32 [rot / 2]; None: no rotation) on the way (see ``include/moe_ffn.h``).  q_out defaults to q (in place).
    Returns q_out."""
    if q_out is None:
        q_out = q
    key = (4, k.shape, k.stride(), k.dtype, k.get_device(), v.shape, v.stride(), v.dtype, v.get_device(),
           positions.shape, positions.stride(), positions.dtype, positions.get_device(), slots.shape, slots.stride(),
           slots.dtype, slots.get_device(), _sig(inv_freq), k_cache.shape, k_cache.stride(), k_cache.dtype,
           k_cache.get_device(), v_cache.shape, v_cache.stride(), v_cache.dtype, v_cache.get_device(), _sig(q),
           _sig(q_out), interleaved, scale)
    a = _blocks.get(key) or _remember(key, _append_block(k, v, positions, slots, inv_freq, k_cache, v_cache, q, q_out,
                                                         interleaved, scale))
    rc = (_lib or lib()).moe_ffn_append_kv(
        a, _raw_stream(stream, k), None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), None if inv_freq is None else inv_freq.data_ptr(),
        None if q_out is None else q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr())
    if rc:
        _check(rc, "moe_ffn_append_kv")
    return q_out


def moe_ffn_attend_workspace(T: int, B: int, q_heads: int, kv_heads: int, D: int) -> int:
    """Workspace bytes of moe_ffn_attend for up to T rows of up to B sequences and heads of D elements."""
    n = ctypes.c_size_t()
    a = _block(AttendArgs, T, B, q_heads, kv_heads, D, ACT_BF16, ACT_F32, 1, 0, 0, 0, 1.0, 0.0, *(10 * [256]), 0, 0)
    _check(lib().moe_ffn_attend_workspace(a, ctypes.byref(n)), "moe_ffn_attend_workspace")
    return max(n.value, 256)


def _attend_block(q, k_cache, v_cache, page_table, lens, q_start, mask, scale, softcap, out, lse, workspace):
    import torch

    _require(q.dim() == 3 and k_cache.dim() == 4 and page_table.dim() == 2,
             "expected q [T, q_heads, D], k_cache [pages, page_size, kv_heads, D], page_table [B, max_pages]")
    T, Hq, D = q.shape
    pages, page_size, Hkv = k_cache.shape[:3]
    B, max_pages = page_table.shape
    shape = (pages, page_size, Hkv, D)
    _require(k_cache.dtype == q.dtype and v_cache.dtype == q.dtype, "k_cache, v_cache: must have q's dtype")
    for t, name in ((page_table, "page_table"), (mask, "mask")):
        _require(t is None or t.dtype == torch.int32, f"{name}: expected int32")
    _whole(lens, (B,), torch.int32, "lens")
    _whole(q_start, (B + 1,), torch.int32, "q_start")
    words, ms = 0, 0
    if mask is not None:
        _require(mask.dim() == 2, "mask: expected [T, words]")
        words = mask.shape[1]
        ms = _matrix(mask, T, words, "mask")
    if lse is not None:
        _whole(lse, (T, Hq), torch.float32, "lse")
    qs, os_ = _heads(q, T, Hq, D, "q"), _heads(out, T, Hq, D, "out")
    a = _block(AttendArgs, T, B, Hq, Hkv, D, _code(q, "q", (ACT_BF16, ACT_F16)), _code(out, "out"), page_size, pages,
               max_pages, words, D**-0.5 if scale is None else scale, softcap, *qs, *os_,
               *_cache_strides(k_cache, shape, "k_cache"), *_cache_strides(v_cache, shape, "v_cache"),
               _matrix(page_table, B, max_pages, "page_table"), ms)
    _on_device(q, q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, lens=lens, q_start=q_start, mask=mask,
               out=out, lse=lse, workspace=workspace)
    if workspace is not None:
        _require(workspace.is_contiguous(), "workspace: must be contiguous")
    return a


def moe_ffn_attend(q, k_cache, v_cache, page_table, lens, q_start, mask=None, scale=None, softcap: float = 0.0,
                   out=None, lse=None, workspace=None, stream=None):
    """Attention of B sequences' newest tokens over the paged cache that holds them.  q [T, q_heads, D]; sequence b's
    rows are ``q_start[b] .. q_start[b + 1]`` (int32 [B + 1]), the last of its ``lens[b]`` cached tokens (int32 [B]),
    which lie in the pages ``page_table[b]`` (int32 [B, max_pages]).  mask int32 [T, words]: which of its sequence's
    rows a row sees (bit j: the j-th), None: those up to itself.  scale defaults to D ** -0.5; softcap 0: no cap (see
    ``include/moe_ffn.h``).  out defaults to a new tensor of q's shape and type (rows of no sequence are then 0), lse
    (fp32 [T, q_heads]) is written where given; neither overlaps another tensor.  workspace (a tensor of
    moe_ffn_attend_workspace bytes) defaults to a new one.  Returns out."""
    if out is None:
        out = _new(stream, q.shape, q.dtype, q.device, zero=True)
    key = (5, q.shape, q.stride(), q.dtype, q.get_device(), k_cache.shape, k_cache.stride(), k_cache.dtype,
           k_cache.get_device(), v_cache.shape, v_cache.stride(), v_cache.dtype, v_cache.get_device(), page_table.shape,
           page_table.stride(), page_table.dtype, page_table.get_device(), lens.shape, lens.stride(), lens.dtype,
           lens.get_device(), q_start.shape, q_start.stride(), q_start.dtype, q_start.get_device(), _sig(mask), scale,
           softcap, out.shape, out.stride(), out.dtype, out.get_device(), _sig(lse), _flat(workspace))
    a = _blocks.get(key) or _remember(key, _attend_block(q, k_cache, v_cache, page_table, lens, q_start, mask, scale,
                                                         softcap, out, lse, workspace))
    if workspace is None:
        import torch

        workspace = _new(stream, (moe_ffn_attend_workspace(a.T, a.B, a.q_heads, a.kv_heads, a.D),), torch.uint8,
                         q.device)
    rc = (_lib or lib()).moe_ffn_attend(
        a, _raw_stream(stream, q), workspace.data_ptr(), workspace.numel() * workspace.element_size(), q.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lens.data_ptr(), q_start.data_ptr(),
        None if mask is None else mask.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr())
    if rc:
        _check(rc, "moe_ffn_attend")
    return out


def moe_ffn_strerror(status: int) -> str:
    return strerror(status)


# ----------------------------------------------------------------------------
# Convenience wrapper


@dataclass
class MoeFFN:
    """A prepared layer: owns the plan and a workspace tensor on the current device."""

    shapes: object
    act: int
    wfmt: int

    def __post_init__(self):
        import torch

        self.plan, self.workspace_bytes = moe_ffn_prepare(self.shapes, self.act, self.wfmt)
        self.workspace = torch.empty(max(self.workspace_bytes, 256), dtype=torch.uint8, device="cuda")

    def __call__(self, x, router_w, expert_w, shexp_w, shexp_gate_w, out=None, topk_ids=None, topk_w=None,
                 stream=None):
        import torch

        if out is None:
            out = torch.empty((self.shapes.T, self.shapes.H), dtype=torch.float32, device=x.device)
        moe_ffn_execute_ex(self.plan, self.workspace, x, router_w, expert_w, shexp_w, shexp_gate_w, out, topk_ids,
                           topk_w, stream)
        return out

    def block(self, x_res, router_w, expert_w, shexp_w, shexp_gate_w, eps=1e-6, topk_ids=None, stream=None):
        moe_ffn_execute_block(self.plan, self.workspace, x_res, router_w, expert_w, shexp_w, shexp_gate_w, eps,
                              topk_ids, None, stream)
        return x_res

    def _check_routed(self, x, ids, weights, expert_w, shexp_w, shexp_gate_w, out):
        import torch

        s = self.shapes
        _whole(ids, (s.T, s.top_k), torch.int32, "ids")
        _whole(weights, (s.T, s.top_k), torch.float32, "weights")
        _on_device(x, x=x, ids=ids, weights=weights)
        x_types = (torch.float32,) if self.act == ACT_F32 else (torch.bfloat16, torch.int16, torch.uint16)
        for t, types, name in ((x, x_types, "x"), (out, (torch.float32,), "out")):
            if t is None or isinstance(t, int):
                continue
            if t.dtype not in types or t.numel() != s.T * s.H or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous tensor of shape {(s.T, s.H)} and {types[0]}, got "
                                 f"{tuple(t.shape)}, {t.dtype}")
        row = {W_BF16: 2 * s.H, W_Q4B32: s.H // 2 + s.H // 16, W_I8: s.H + 16}[self.wfmt]
        gate = shexp_gate_w if shexp_w is not None else None  # ignored without a shared expert
        need = {"expert_w": (expert_w, 3 * s.E * s.I * row, self.wfmt), "shexp_w": (shexp_w, 3 * s.Is * row, self.wfmt),
                "shexp_gate_w": (gate, 2 * s.H, W_BF16)}
        for name, (t, nbytes, wfmt) in need.items():
            if t is None or isinstance(t, int):
                continue
            if t.dtype.is_floating_point and (wfmt != W_BF16 or t.dtype != torch.bfloat16):
                raise ValueError(f"{name}: dtype {t.dtype} is not that of the plan's weights")
            if not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
                raise ValueError(f"{name}: expected a contiguous tensor of {nbytes} bytes, got "
                                 f"{t.numel() * t.element_size()}")
        rest = dict(expert_w=expert_w, shexp_w=shexp_w, shexp_gate_w=gate, out=out)
        _on_device(x, **{n: t for n, t in rest.items() if not isinstance(t, int)})

    def routed(self, x, ids, weights, expert_w, shexp_w=None, shexp_gate_w=None, out=None, stream=None):
        """The layer for a given routing (moe_ffn_execute_routed); returns out.  x [T, H] of the plan's type and out
        fp32 [T, H], both contiguous; the weights contiguous, of bf16 or as bytes, at least as many as the plan's."""
        s = self.shapes
        key = (_sig(ids), _sig(weights), _flat(x), _flat(expert_w), _flat(shexp_w), _flat(shexp_gate_w), _flat(out))
        # signatures that this layer has checked
        passed = getattr(self, "_routed", None)
        if passed is None:
            passed = self._routed = set()
        if key not in passed:
            self._check_routed(x, ids, weights, expert_w, shexp_w, shexp_gate_w, out)
            if len(passed) >= 4096:
                passed.clear()
            passed.add(key)
        if out is None:
            import torch

            out = _new(stream, (s.T, s.H), torch.float32, x.device)
        moe_ffn_execute_routed(self.plan, self.workspace, x, ids, weights, expert_w, shexp_w, shexp_gate_w, out,
                               _raw_stream(stream, x), self.workspace_bytes)
        return out

    def status(self, stream=None) -> int:
        return moe_ffn_read_status(self.plan, self.workspace, stream)

    def routing(self, stream=None):
        s = self.shapes
        return moe_ffn_read_routing(self.plan, self.workspace, s.E, s.T, s.top_k, stream)

    def close(self):
        if getattr(self, "plan", None):
            moe_ffn_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
