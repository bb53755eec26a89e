"""GB300 (sm_103a) fused MoE-FFN: Python binding of libhmm.so.

The functions ``hmm_*`` mirror the C entry points of ``include/hmm.h`` one to
one and only marshal arguments (torch tensors -> device pointers and sizes,
the current CUDA stream).  Every step of the computation runs in the CUDA
kernels of the library; there is no Python or CPU fallback: if ``libhmm.so``
is missing, every call raises.

``moe_ffn(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight)`` is
the autograd entry point (forward saves what the backward needs, backward
returns one gradient per public argument and None for topk_ids), following
the HyperMegaMoE API (§3.1) and its DFunction semantics (§3.2).

``moe_gate`` is the router in front of it (differentiable in the logits);
``mx4_quantize_experts`` and ``moe_ffn_mx4`` serve the same layer with
microscaled 4-bit expert weights.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

__all__ = [
    "HmmError", "HmmShape", "hmm_create", "hmm_destroy", "hmm_set_option",
    "hmm_workspace_size", "hmm_route", "hmm_route_static", "hmm_forward", "hmm_backward",
    "hmm_backward_dx", "hmm_backward_dw", "hmm_forward_shared", "hmm_backward_shared",
    "hmm_gate_forward", "hmm_gate_backward", "HmmGate", "make_gate", "moe_gate",
    "hmm_mx4_size", "hmm_mx4_quantize", "hmm_mx4_dequantize", "hmm_mx4_workspace_size",
    "hmm_forward_mx4", "HmmMx4", "make_mx4", "Mx4Tensor", "mx4_quantize", "mx4_quantize_experts",
    "moe_ffn_mx4",
    "hmm_status",
    "hmm_error_string", "Context", "moe_ffn", "library_path", "load_library",
    "hmm_profile_read", "hmm_phase_name", "hmm_set_trace",
    "HMM_OPT_VALIDATE", "HMM_OPT_WAIT_BUDGET_NS", "HMM_OPT_INJECT_SKIP_READY", "HMM_OPT_PROFILE",
    "HMM_OPT_PAIR_ROWS", "HMM_OPT_OVERLAP_LAUNCHES", "HMM_OPT_FUSED_COMBINE",
    "HMM_DTYPE_BF16", "HMM_DTYPE_F32", "HMM_SCORE_SOFTMAX", "HMM_SCORE_SIGMOID",
    "HMM_MX4_ROWS", "HMM_MX4_COLUMNS", "HMM_MX4_GATE_UP", "HMM_STATUS_EXPERT_ID", "HMM_STATUS_TIMEOUT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_LIB_PATH = os.path.join(_HERE, "libhmm.so")
_HEADER = os.path.join(_ROOT, "include", "hmm.h")


def _header_constants():
    consts = {}
    with open(_HEADER) as f:
        for m in re.finditer(r"#define\s+(HMM_\w+)\s+\(?(-?\w+?)u?\)?\s", f.read()):
            try:
                consts[m.group(1)] = int(m.group(2), 0)
            except ValueError:
                pass
    return consts


_C = _header_constants()
HMM_OK = _C["HMM_OK"]
HMM_ERR_TIMEOUT = _C["HMM_ERR_TIMEOUT"]
HMM_ERR_EXPERT_ID = _C["HMM_ERR_EXPERT_ID"]
HMM_OPT_VALIDATE = _C["HMM_OPT_VALIDATE"]
HMM_OPT_WAIT_BUDGET_NS = _C["HMM_OPT_WAIT_BUDGET_NS"]
HMM_OPT_INJECT_SKIP_READY = _C["HMM_OPT_INJECT_SKIP_READY"]
HMM_OPT_PROFILE = _C["HMM_OPT_PROFILE"]
HMM_OPT_PAIR_ROWS = _C["HMM_OPT_PAIR_ROWS"]
HMM_OPT_OVERLAP_LAUNCHES = _C["HMM_OPT_OVERLAP_LAUNCHES"]
HMM_OPT_FUSED_COMBINE = _C["HMM_OPT_FUSED_COMBINE"]
HMM_DTYPE_BF16 = _C["HMM_DTYPE_BF16"]
HMM_DTYPE_F32 = _C["HMM_DTYPE_F32"]
HMM_SCORE_SOFTMAX = _C["HMM_SCORE_SOFTMAX"]
HMM_SCORE_SIGMOID = _C["HMM_SCORE_SIGMOID"]
HMM_MX4_ROWS = _C["HMM_MX4_ROWS"]
HMM_MX4_COLUMNS = _C["HMM_MX4_COLUMNS"]
HMM_MX4_GATE_UP = _C["HMM_MX4_GATE_UP"]
HMM_STATUS_EXPERT_ID = _C["HMM_STATUS_EXPERT_ID"]
HMM_STATUS_TIMEOUT = _C["HMM_STATUS_TIMEOUT"]


class HmmShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("K", ctypes.c_int64),
                ("weights_dtype", ctypes.c_int32), ("shared", ctypes.c_int32)]


class HmmGate(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ld_logits", ctypes.c_int64), ("logits_dtype", ctypes.c_int32),
                ("weights_dtype", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class HmmMx4(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32)]


class HmmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {hmm_error_string(code)} (code {code})")


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice

_lib = None
_lib_lock = threading.Lock()


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libhmm.so (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing; build it with "
                "`python -m dispatch_grouped_gemm_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        sp, gp = ctypes.POINTER(HmmShape), ctypes.POINTER(HmmGate)
        mp, szp = ctypes.POINTER(HmmMx4), ctypes.POINTER(sz)
        sig = {
            "hmm_create": [ctypes.POINTER(vp), i32],
            "hmm_destroy": [vp],
            "hmm_set_option": [vp, i32, i64],
            "hmm_workspace_size": [sp, i32, ctypes.POINTER(sz), ctypes.POINTER(sz),
                                   ctypes.POINTER(sz)],
            "hmm_route": [vp, sp, vp, vp, vp, vp, vp, vp, sz, vp],
            "hmm_route_static": [sp, vp, vp, vp, vp, vp, vp],
            "hmm_forward": [vp, sp, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp],
            "hmm_backward": [vp, sp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp, sz, vp],
            "hmm_backward_dx": [vp, sp, vp, vp, vp, vp, vp, sz, vp, vp, vp, sz, vp],
            "hmm_forward_shared": [vp, sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, vp],
            "hmm_backward_shared": [vp, sp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp,
                                    vp, vp, sz, vp],
            "hmm_backward_dw": [vp, sp, vp, sz, vp, vp, vp, sz, vp],
            "hmm_gate_forward": [vp, gp, vp, vp, vp, vp, vp, vp],
            "hmm_gate_backward": [vp, gp, vp, vp, vp, vp, vp, vp],
            "hmm_mx4_size": [mp, szp, szp],
            "hmm_mx4_quantize": [vp, mp, vp, vp, vp, vp],
            "hmm_mx4_dequantize": [vp, mp, vp, vp, vp, vp],
            "hmm_mx4_workspace_size": [sp, szp],
            "hmm_forward_mx4": [vp, sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "hmm_status": [vp, vp, ctypes.POINTER(i32)],
            "hmm_profile_read": [vp, i32, ctypes.POINTER(ctypes.c_double),
                                 ctypes.POINTER(ctypes.c_int64)],
            "hmm_set_trace": [vp, vp, sz, i32],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = i32
        lib.hmm_error_string.argtypes = [i32]
        lib.hmm_error_string.restype = ctypes.c_char_p
        lib.hmm_phase_name.argtypes = [i32]
        lib.hmm_phase_name.restype = ctypes.c_char_p
        _lib = lib
        return lib


# ------------------------------------------------------------ marshalling
def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without building the objects (3 us)
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != HMM_OK:
        raise HmmError(rc, where)


def make_shape(T, H, I, E, K, weights_dtype=HMM_DTYPE_BF16, shared=0) -> HmmShape:
    return HmmShape(int(T), int(H), int(I), int(E), int(K), int(weights_dtype), int(shared))


def hmm_error_string(code: int) -> str:
    return load_library().hmm_error_string(int(code)).decode()


def hmm_create(device: int = 0):
    h = ctypes.c_void_p()
    _check(load_library().hmm_create(ctypes.byref(h), int(device)), "hmm_create")
    return h


def hmm_destroy(ctx):
    _check(load_library().hmm_destroy(ctx), "hmm_destroy")


def hmm_set_option(ctx, option: int, value: int):
    _check(load_library().hmm_set_option(ctx, int(option), int(value)), "hmm_set_option")


def hmm_workspace_size(shape: HmmShape, training: bool):
    f, s, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().hmm_workspace_size(ctypes.byref(shape), int(bool(training)),
                                             ctypes.byref(f), ctypes.byref(s), ctypes.byref(b)),
           "hmm_workspace_size")
    return f.value, s.value, b.value


def hmm_route(ctx, shape, topk_ids, counts, offsets, slot2row, row2slot, workspace, stream=None):
    rc = load_library().hmm_route(ctx, ctypes.byref(shape), _ptr(topk_ids), _ptr(counts),
                                  _ptr(offsets), _ptr(slot2row), _ptr(row2slot), _ptr(workspace),
                                  _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_route")


def hmm_route_static(shape, topk_ids, counts, offsets, slot2row, row2slot, stream=None):
    """Routing on the current device with the library's static scratch (no
    allocation, no context); see include/hmm.h."""
    rc = load_library().hmm_route_static(ctypes.byref(shape), _ptr(topk_ids), _ptr(counts),
                                         _ptr(offsets), _ptr(slot2row), _ptr(row2slot),
                                         _stream(stream))
    _check(rc, "hmm_route_static")


def hmm_forward(ctx, shape, x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, y,
                saved, workspace, stream=None):
    rc = load_library().hmm_forward(ctx, ctypes.byref(shape), _ptr(x), _ptr(topk_ids),
                                    _ptr(topk_weights), _ptr(up_proj_weight),
                                    _ptr(down_proj_weight), _ptr(y), _ptr(saved), _nbytes(saved),
                                    _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_forward")


def hmm_backward(ctx, shape, dy, topk_weights, up_proj_weight, down_proj_weight, saved, dx,
                 d_up_proj_weight, d_down_proj_weight, d_topk_weights, workspace, stream=None):
    rc = load_library().hmm_backward(ctx, ctypes.byref(shape), _ptr(dy), _ptr(topk_weights),
                                     _ptr(up_proj_weight), _ptr(down_proj_weight), _ptr(saved),
                                     _nbytes(saved), _ptr(dx), _ptr(d_up_proj_weight),
                                     _ptr(d_down_proj_weight), _ptr(d_topk_weights),
                                     _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_backward")


def hmm_forward_shared(ctx, shape, x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                       shared_up_proj_weight, shared_down_proj_weight, y, saved, workspace,
                       stream=None):
    rc = load_library().hmm_forward_shared(
        ctx, ctypes.byref(shape), _ptr(x), _ptr(topk_ids), _ptr(topk_weights),
        _ptr(up_proj_weight), _ptr(down_proj_weight), _ptr(shared_up_proj_weight),
        _ptr(shared_down_proj_weight), _ptr(y), _ptr(saved), _nbytes(saved), _ptr(workspace),
        _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_forward_shared")


def hmm_backward_shared(ctx, shape, dy, topk_weights, up_proj_weight, down_proj_weight,
                        shared_up_proj_weight, shared_down_proj_weight, saved, dx,
                        d_up_proj_weight, d_down_proj_weight, d_shared_up_proj_weight,
                        d_shared_down_proj_weight, d_topk_weights, workspace, stream=None):
    rc = load_library().hmm_backward_shared(
        ctx, ctypes.byref(shape), _ptr(dy), _ptr(topk_weights), _ptr(up_proj_weight),
        _ptr(down_proj_weight), _ptr(shared_up_proj_weight), _ptr(shared_down_proj_weight),
        _ptr(saved), _nbytes(saved), _ptr(dx), _ptr(d_up_proj_weight), _ptr(d_down_proj_weight),
        _ptr(d_shared_up_proj_weight), _ptr(d_shared_down_proj_weight), _ptr(d_topk_weights),
        _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_backward_shared")


def hmm_backward_dx(ctx, shape, dy, topk_weights, up_proj_weight, down_proj_weight, saved, dx,
                    d_topk_weights, workspace, stream=None):
    rc = load_library().hmm_backward_dx(ctx, ctypes.byref(shape), _ptr(dy), _ptr(topk_weights),
                                        _ptr(up_proj_weight), _ptr(down_proj_weight),
                                        _ptr(saved), _nbytes(saved), _ptr(dx),
                                        _ptr(d_topk_weights), _ptr(workspace), _nbytes(workspace),
                                        _stream(stream))
    _check(rc, "hmm_backward_dx")


def hmm_backward_dw(ctx, shape, saved, d_up_proj_weight, d_down_proj_weight, workspace,
                    stream=None):
    rc = load_library().hmm_backward_dw(ctx, ctypes.byref(shape), _ptr(saved), _nbytes(saved),
                                        _ptr(d_up_proj_weight), _ptr(d_down_proj_weight),
                                        _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_backward_dw")


def make_gate(T, E, K, *, score=HMM_SCORE_SOFTMAX, ld_logits=None, logits_dtype=HMM_DTYPE_F32,
              weights_dtype=HMM_DTYPE_F32, renormalize=0, groups=1, topk_groups=1, group_top=1,
              scale=1.0) -> HmmGate:
    return HmmGate(int(T), int(E), int(K), int(E if ld_logits is None else ld_logits),
                   int(logits_dtype), int(weights_dtype), int(score), int(renormalize),
                   int(groups), int(topk_groups), int(group_top), float(scale))


def hmm_gate_forward(ctx, gate, logits, bias, topk_ids, topk_weights, scores=None, stream=None):
    rc = load_library().hmm_gate_forward(ctx, ctypes.byref(gate), _ptr(logits), _ptr(bias),
                                         _ptr(topk_ids), _ptr(topk_weights), _ptr(scores),
                                         _stream(stream))
    _check(rc, "hmm_gate_forward")


def hmm_gate_backward(ctx, gate, logits, topk_ids, d_topk_weights, d_scores, d_logits,
                      stream=None):
    rc = load_library().hmm_gate_backward(ctx, ctypes.byref(gate), _ptr(logits), _ptr(topk_ids),
                                          _ptr(d_topk_weights), _ptr(d_scores), _ptr(d_logits),
                                          _stream(stream))
    _check(rc, "hmm_gate_backward")


def make_mx4(rows, cols, *, batch=1, ld=None, dtype=HMM_DTYPE_BF16, layout=HMM_MX4_ROWS) -> HmmMx4:
    return HmmMx4(int(batch), int(rows), int(cols), int(cols if ld is None else ld), int(dtype),
                  int(layout))


def hmm_mx4_size(desc):
    """(bytes of the codes, bytes of the scales)."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().hmm_mx4_size(ctypes.byref(desc), ctypes.byref(c), ctypes.byref(s)),
           "hmm_mx4_size")
    return c.value, s.value


def hmm_mx4_quantize(ctx, desc, values, codes, scales, stream=None):
    rc = load_library().hmm_mx4_quantize(ctx, ctypes.byref(desc), _ptr(values), _ptr(codes),
                                         _ptr(scales), _stream(stream))
    _check(rc, "hmm_mx4_quantize")


def hmm_mx4_dequantize(ctx, desc, codes, scales, values, stream=None):
    rc = load_library().hmm_mx4_dequantize(ctx, ctypes.byref(desc), _ptr(codes), _ptr(scales),
                                           _ptr(values), _stream(stream))
    _check(rc, "hmm_mx4_dequantize")


def hmm_mx4_workspace_size(shape: HmmShape) -> int:
    n = ctypes.c_size_t()
    _check(load_library().hmm_mx4_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "hmm_mx4_workspace_size")
    return n.value


def hmm_forward_mx4(ctx, shape, x, topk_ids, topk_weights, up_codes, up_scales, down_codes,
                    down_scales, y, workspace, stream=None):
    rc = load_library().hmm_forward_mx4(ctx, ctypes.byref(shape), _ptr(x), _ptr(topk_ids),
                                        _ptr(topk_weights), _ptr(up_codes), _ptr(up_scales),
                                        _ptr(down_codes), _ptr(down_scales), _ptr(y),
                                        _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "hmm_forward_mx4")


def hmm_status(ctx, stream=None):
    """Synchronise the stream, read and clear the device status word.
    Returns (return code, HMM_STATUS_* bits) without raising."""
    bits = ctypes.c_int(0)
    rc = load_library().hmm_status(ctx, _stream(stream), ctypes.byref(bits))
    return rc, bits.value


def hmm_phase_name(phase: int):
    r = load_library().hmm_phase_name(int(phase))
    return None if r is None else r.decode()


def hmm_profile_read(ctx):
    """{phase name: (GPU ms, kernel launches)} since the previous read."""
    n = _C["HMM_NUM_PHASES"]
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(load_library().hmm_profile_read(ctx, n, ms, cnt), "hmm_profile_read")
    return {hmm_phase_name(i): (ms[i], cnt[i]) for i in range(n)}


def hmm_set_trace(ctx, buffer, which: int):
    """Record the per-tile timeline of the next GEMM launch of kind `which`
    (0 forward, 1 backward data, 2 backward weight) into `buffer` (a device
    tensor; None disables)."""
    _check(load_library().hmm_set_trace(ctx, _ptr(buffer), _nbytes(buffer), int(which)),
           "hmm_set_trace")


# ------------------------------------------------------------ torch layer
_WDTYPES = {torch.bfloat16: HMM_DTYPE_BF16, torch.float32: HMM_DTYPE_F32}
_TORCH_WDTYPES = {code: dtype for dtype, code in _WDTYPES.items()}


def _u8(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


class Context:
    """A library context on one device plus shape checks of torch arguments."""

    _cache: dict = {}
    _cache_lock = threading.Lock()

    def __init__(self, device=None):
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                           torch.device(device).index or 0)
        self.device = dev
        self.handle = hmm_create(dev.index)

    def close(self):
        if self.handle is not None:
            hmm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @classmethod
    def for_device(cls, device) -> "Context":
        idx = device.index if device.index is not None else torch.cuda.current_device()
        c = cls._cache.get(idx)
        if c is not None:
            return c
        with cls._cache_lock:
            c = cls._cache.get(idx)
            if c is None:
                c = cls._cache[idx] = cls(torch.device("cuda", idx))
            return c

    def set_option(self, option: int, value: int):
        hmm_set_option(self.handle, option, value)

    @staticmethod
    def shape_of(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                 shared_up_proj_weight=None, shared_down_proj_weight=None) -> HmmShape:
        if x.dim() != 2 or topk_ids.dim() != 2 or up_proj_weight.dim() != 3:
            raise ValueError("x [T,H], topk_ids [T,K], up_proj_weight [E,H,2I] expected")
        T, H = x.shape
        E, H1, I2 = up_proj_weight.shape
        if H1 != H or I2 % 2:
            raise ValueError(f"up_proj_weight {tuple(up_proj_weight.shape)} does not match x {tuple(x.shape)}")
        I = I2 // 2
        if tuple(down_proj_weight.shape) != (E, I, H):
            raise ValueError(f"down_proj_weight must be {(E, I, H)}, got {tuple(down_proj_weight.shape)}")
        if topk_ids.shape[0] != T or tuple(topk_weights.shape) != tuple(topk_ids.shape):
            raise ValueError("topk_ids / topk_weights must both be [T, K]")
        if x.dtype != torch.bfloat16 or up_proj_weight.dtype != torch.bfloat16 or \
                down_proj_weight.dtype != torch.bfloat16:
            raise TypeError("x, up_proj_weight and down_proj_weight must be bfloat16")
        if topk_ids.dtype != torch.int32:
            raise TypeError("topk_ids must be int32")
        if topk_weights.dtype not in _WDTYPES:
            raise TypeError("topk_weights must be bfloat16 or float32")
        shared = shared_up_proj_weight is not None or shared_down_proj_weight is not None
        if shared:
            if shared_up_proj_weight is None or shared_down_proj_weight is None:
                raise ValueError("the shared expert needs both shared weights")
            if tuple(shared_up_proj_weight.shape) != (H, 2 * I) or \
                    tuple(shared_down_proj_weight.shape) != (I, H):
                raise ValueError(f"shared weights must be {(H, 2 * I)} and {(I, H)}")
            if shared_up_proj_weight.dtype != torch.bfloat16 or \
                    shared_down_proj_weight.dtype != torch.bfloat16:
                raise TypeError("shared weights must be bfloat16")
        for t in (x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                  shared_up_proj_weight, shared_down_proj_weight):
            if t is not None and (not t.is_cuda or not t.is_contiguous()):
                raise ValueError("all arguments must be contiguous CUDA tensors")
        return make_shape(T, H, I, E, topk_ids.shape[1], _WDTYPES[topk_weights.dtype],
                          1 if shared else 0)

    def forward(self, x, topk_ids, topk_weights, W1, W2, training: bool, stream=None,
                Ws1=None, Ws2=None):
        shape = self.shape_of(x, topk_ids, topk_weights, W1, W2, Ws1, Ws2)
        fwd, sv, _ = hmm_workspace_size(shape, training)
        y = torch.empty_like(x)
        ws = _u8(fwd, x.device)
        saved = _u8(sv, x.device) if training else None
        if shape.shared:
            hmm_forward_shared(self.handle, shape, x, topk_ids, topk_weights, W1, W2, Ws1, Ws2, y,
                               saved, ws, stream)
        else:
            hmm_forward(self.handle, shape, x, topk_ids, topk_weights, W1, W2, y, saved, ws,
                        stream)
        return y, saved

    def backward(self, dy, x, topk_ids, topk_weights, W1, W2, saved, need=(True, True, True, True),
                 stream=None, Ws1=None, Ws2=None, need_shared=(True, True)):
        """(dx, dW1, dW2, d_topk_weights) and, with the shared expert, (dWs1, dWs2)
        appended; `need` / `need_shared` skip outputs."""
        shape = self.shape_of(x, topk_ids, topk_weights, W1, W2, Ws1, Ws2)
        _, _, bwd = hmm_workspace_size(shape, True)
        dy = dy.contiguous()
        if dy.dtype != torch.bfloat16 or tuple(dy.shape) != tuple(x.shape):
            raise ValueError("dy must be bfloat16 with the shape of x")
        dx = torch.empty_like(x) if need[0] else None
        dW1 = torch.empty_like(W1) if need[1] else None
        dW2 = torch.empty_like(W2) if need[2] else None
        dw = torch.empty_like(topk_weights) if need[3] else None
        ws = _u8(bwd, x.device)
        if not shape.shared:
            hmm_backward(self.handle, shape, dy, topk_weights, W1, W2, saved, dx, dW1, dW2, dw,
                         ws, stream)
            return dx, dW1, dW2, dw
        dWs1 = torch.empty_like(Ws1) if need_shared[0] else None
        dWs2 = torch.empty_like(Ws2) if need_shared[1] else None
        hmm_backward_shared(self.handle, shape, dy, topk_weights, W1, W2, Ws1, Ws2, saved, dx,
                            dW1, dW2, dWs1, dWs2, dw, ws, stream)
        return dx, dW1, dW2, dw, dWs1, dWs2


class _FirstOrder(torch.autograd.Function):
    """A gradient under create_graph: the kernels that computed it have no
    backward of their own, so that differentiating it is an error rather than a
    constant.  (`inputs` make it require a gradient.)"""

    @staticmethod
    def forward(ctx, name, grad, *inputs):
        ctx.name = name
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError(f"{ctx.name} has no second derivative")


def _first_order(name, grads, inputs):
    """The gradients, marked as above where create_graph asks for it."""
    if not torch.is_grad_enabled():
        return grads
    return tuple(g if g is None else _FirstOrder.apply(name, g, *inputs) for g in grads)


class _MoEFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_ids, topk_weights, W1, W2):
        c = Context.for_device(x.device)
        y, saved = c.forward(x, topk_ids, topk_weights, W1, W2, training=True)
        ctx.save_for_backward(x, topk_ids, topk_weights, W1, W2, saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, topk_ids, topk_weights, W1, W2, saved = ctx.saved_tensors
        need = (ctx.needs_input_grad[0], ctx.needs_input_grad[3], ctx.needs_input_grad[4],
                ctx.needs_input_grad[2])
        c = Context.for_device(x.device)
        dx, dW1, dW2, dw = _first_order(
            "moe_ffn", c.backward(dy, x, topk_ids, topk_weights, W1, W2, saved, need),
            (x, topk_weights, W1, W2))
        return dx, None, dw, dW1, dW2


class _MoEFFNShared(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_ids, topk_weights, W1, W2, Ws1, Ws2):
        c = Context.for_device(x.device)
        y, saved = c.forward(x, topk_ids, topk_weights, W1, W2, training=True, Ws1=Ws1, Ws2=Ws2)
        ctx.save_for_backward(x, topk_ids, topk_weights, W1, W2, Ws1, Ws2, saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, topk_ids, topk_weights, W1, W2, Ws1, Ws2, saved = ctx.saved_tensors
        n = ctx.needs_input_grad
        c = Context.for_device(x.device)
        grads = c.backward(dy, x, topk_ids, topk_weights, W1, W2, saved, (n[0], n[3], n[4], n[2]),
                           Ws1=Ws1, Ws2=Ws2, need_shared=(n[5], n[6]))
        dx, dW1, dW2, dw, dWs1, dWs2 = _first_order(
            "moe_ffn", grads, (x, topk_weights, W1, W2, Ws1, Ws2))
        return dx, None, dw, dW1, dW2, dWs1, dWs2


def moe_ffn(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, *,
            shared_up_proj_weight=None, shared_down_proj_weight=None):
    """y[T,H] = sum_k topk_weights[t,k] * FFN_{topk_ids[t,k]}(x[t]) with SwiGLU
    experts (gate = first I columns of up_proj's 2I outputs), plus FFN_s(x[t])
    of the optional shared expert (keyword-only weights [H, 2I] and [I, H]).
    Differentiable (once) in x, topk_weights and every weight tensor; topk_ids
    is not."""
    shared = (shared_up_proj_weight, shared_down_proj_weight)
    has_shared = shared[0] is not None or shared[1] is not None
    tensors = (x, topk_weights, up_proj_weight, down_proj_weight) + (shared if has_shared else ())
    if not (torch.is_grad_enabled() and any(t.requires_grad for t in tensors)):
        c = Context.for_device(x.device)
        y, _ = c.forward(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                         training=False, Ws1=shared[0], Ws2=shared[1])
        return y
    if has_shared:
        return _MoEFFNShared.apply(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                                   *shared)
    return _MoEFFN.apply(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight)


_SCORES = {"softmax": HMM_SCORE_SOFTMAX, "sigmoid": HMM_SCORE_SIGMOID}


def _gate_forward(logits, gate, bias, return_scores):
    dev = logits.device
    shape = (gate.T, gate.K)
    ids = torch.empty(shape, dtype=torch.int32, device=dev)
    w = torch.empty(shape, dtype=_TORCH_WDTYPES[gate.weights_dtype], device=dev)
    scores = (torch.empty((gate.T, gate.E), dtype=torch.float32, device=dev)
              if return_scores else None)
    # (the library's function itself: a decode step's router is host time)
    rc = load_library().hmm_gate_forward(
        Context.for_device(dev).handle, ctypes.byref(gate), logits.data_ptr(),
        None if bias is None else bias.data_ptr(), ids.data_ptr(), w.data_ptr(),
        None if scores is None else scores.data_ptr(), _raw_stream(dev.index))
    if rc != HMM_OK:
        raise HmmError(rc, "hmm_gate_forward")
    return ids, w, scores


class _MoEGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, gate, bias, return_scores):
        ids, w, scores = _gate_forward(logits, gate, bias, return_scores)
        ctx.gate = gate
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return ids, w, scores

    @staticmethod
    def backward(ctx, _, dw, ds):
        if dw is None and ds is None:
            return None, None, None, None
        logits, ids = ctx.saved_tensors
        if dw is not None and not dw.is_contiguous():
            dw = dw.contiguous()
        if ds is not None and not ds.is_contiguous():
            ds = ds.contiguous()
        dev = logits.device
        dl = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        rc = load_library().hmm_gate_backward(
            Context.for_device(dev).handle, ctypes.byref(ctx.gate), logits.data_ptr(),
            ids.data_ptr(), None if dw is None else dw.data_ptr(),
            None if ds is None else ds.data_ptr(), dl.data_ptr(), _raw_stream(dev.index))
        if rc != HMM_OK:
            raise HmmError(rc, "hmm_gate_backward")
        return *_first_order("moe_gate", (dl,), (logits,)), None, None, None


def moe_gate(logits, k, *, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1,
             renormalize=False, scale=1.0, weights_dtype=torch.float32, return_scores=False):
    """Router: logits [T, E] (bfloat16 or float32, unit stride along E) to
    (topk_ids int32 [T, k], topk_weights [T, k]), the inputs of moe_ffn, and
    with return_scores the scores p, float32 [T, E].

    p = softmax or sigmoid of the logits; the k best p + bias are selected
    (bias: float32 [E], selection only; equal keys by ascending expert), with
    groups > 1 only inside the topk_groups best of `groups` groups of
    consecutive experts, a group counting by the sum of its group_top best
    keys; the weights are scale * p of the selected experts, divided by their
    sum with renormalize.  A logit of -inf has p = 0: without a bias its expert
    comes last; with one its key is the bias alone.  Differentiable (once) in
    the logits through the weights and the scores."""
    if logits.dim() != 2:
        raise ValueError("logits [T, E] expected")
    ldt, wdt = _WDTYPES.get(logits.dtype), _WDTYPES.get(weights_dtype)
    if ldt is None or wdt is None:
        raise TypeError("logits and weights_dtype must be bfloat16 or float32")
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    T, E = logits.shape
    if not logits.is_cuda or (E > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor with unit stride along the experts")
    ld = logits.stride(0)
    if ld < E:
        if T > 1:
            logits = logits.contiguous()  # broadcast or overlapping rows
        ld = E
    if bias is not None:
        if bias.shape != (E,) or not bias.is_contiguous() or bias.device != logits.device:
            raise ValueError(f"bias must be a contiguous [{E}] tensor on the logits' device")
        if bias.dtype != torch.float32:
            raise TypeError("bias must be float32")
    gate = HmmGate(T, E, k, ld, ldt, wdt, kind, 1 if renormalize else 0, groups,
                   groups if topk_groups is None else topk_groups, group_top, scale)
    if logits.requires_grad and torch.is_grad_enabled():
        ids, w, scores = _MoEGate.apply(logits, gate, bias, return_scores)
    else:
        ids, w, scores = _gate_forward(logits, gate, bias, return_scores)
    return (ids, w, scores) if return_scores else (ids, w)


class Mx4Tensor:
    """A microscaled 4-bit operand, or a stack of them for the experts: uint8
    `codes` [N, K/2] and `scales` [N tiles, K tiles, 512] (with a leading batch
    dimension for experts) in the storage that include/hmm.h describes.

    layout HMM_MX4_ROWS stands for values [rows, cols]; HMM_MX4_COLUMNS and
    HMM_MX4_GATE_UP for expert weights [batch, cols, rows] (cols: the
    contraction)."""

    __slots__ = ("codes", "scales", "batch", "rows", "cols", "layout")

    def __init__(self, codes, scales, batch, rows, cols, layout):
        self.codes, self.scales = codes, scales
        self.batch, self.rows, self.cols, self.layout = batch, rows, cols, layout

    @staticmethod
    def _shapes(batch, rows, cols, layout):
        stored = (rows // 2 + 31) // 32 * 64 if layout == HMM_MX4_GATE_UP else rows
        codes = (stored, (cols + 31) // 32 * 16)
        scales = ((stored + 127) // 128, (cols + 127) // 128, 512)
        return (codes, scales) if layout == HMM_MX4_ROWS else ((batch,) + codes, (batch,) + scales)

    @classmethod
    def _wrap(cls, codes, scales, batch, rows, cols, layout):
        want = cls._shapes(batch, rows, cols, layout)
        if (tuple(codes.shape), tuple(scales.shape)) != want:
            raise ValueError(f"codes and scales must be {want}, got "
                             f"{(tuple(codes.shape), tuple(scales.shape))}")
        for t in (codes, scales):
            if t.dtype != torch.uint8:
                raise TypeError("codes and scales must be uint8")
            if not t.is_cuda or not t.is_contiguous() or t.device != codes.device:
                raise ValueError("codes and scales must be contiguous tensors of one CUDA device")
        return cls(codes, scales, batch, rows, cols, layout)

    @classmethod
    def from_rows(cls, codes, scales, cols):
        """Stored rows (e.g. loaded from a file)."""
        return cls._wrap(codes, scales, 1, codes.shape[0], cols, HMM_MX4_ROWS)

    @classmethod
    def experts(cls, codes, scales, *, K, N, gate_up=False):
        """Stored expert weights [E, K, N], contraction K; gate_up: an
        up-projection (N = 2I) with gate and up rows in turn."""
        return cls._wrap(codes, scales, codes.shape[0], N, K,
                         HMM_MX4_GATE_UP if gate_up else HMM_MX4_COLUMNS)

    @property
    def shape(self):
        """Shape of the values."""
        if self.layout == HMM_MX4_ROWS:
            return (self.rows, self.cols)
        return (self.batch, self.cols, self.rows)

    def dequantize(self, dtype=torch.bfloat16):
        """The values that the codes and scales stand for (exact)."""
        code = _WDTYPES.get(dtype)
        if code is None:
            raise TypeError("dtype must be bfloat16 or float32")
        dev = self.codes.device
        out = torch.empty(self.shape, dtype=dtype, device=dev)
        d = _mx4_args(self.batch, self.rows, self.cols, self.cols, code, self.layout)[0]
        rc = load_library().hmm_mx4_dequantize(
            Context.for_device(dev).handle, ctypes.byref(d), self.codes.data_ptr(),
            self.scales.data_ptr(), out.data_ptr(), _raw_stream(dev.index))
        if rc != HMM_OK:
            raise HmmError(rc, "hmm_mx4_dequantize")
        return out


@functools.lru_cache(maxsize=64)
def _mx4_args(batch, rows, cols, ld, dtype, layout):
    """(hmm_mx4, shape of the codes, of the scales) of an operand."""
    return (HmmMx4(batch, rows, cols, ld, dtype, layout),
            *Mx4Tensor._shapes(batch, rows, cols, layout))


def _mx4_of(values, batch, rows, cols, ld, layout):
    d, cs, ss = _mx4_args(batch, rows, cols, ld, _WDTYPES[values.dtype], layout)
    dev = values.device
    codes = torch.empty(cs, dtype=torch.uint8, device=dev)
    scales = torch.empty(ss, dtype=torch.uint8, device=dev)
    rc = load_library().hmm_mx4_quantize(
        Context.for_device(dev).handle, ctypes.byref(d), values.data_ptr(), codes.data_ptr(),
        scales.data_ptr(), _raw_stream(dev.index))
    if rc != HMM_OK:
        raise HmmError(rc, "hmm_mx4_quantize")
    return Mx4Tensor(codes, scales, batch, rows, cols, layout)


def mx4_quantize(x):
    """Rows [R, C] (bfloat16 or float32, C a multiple of 8, unit stride along
    C) to microscaled 4-bit form, blocks of 32 along C."""
    if x.dim() != 2:
        raise ValueError("x [R, C] expected")
    if x.dtype not in _WDTYPES:
        raise TypeError("x must be bfloat16 or float32")
    R, C = x.shape
    if not x.is_cuda or (C > 1 and x.stride(1) != 1):
        raise ValueError("x must be a CUDA tensor with unit stride along its columns")
    ld = x.stride(0) if R > 1 else C
    if ld < C:
        x, ld = x.contiguous(), C  # broadcast or overlapping rows
    return _mx4_of(x, 1, R, C, ld, HMM_MX4_ROWS)


def mx4_quantize_experts(w, *, gate_up=False):
    """Expert weights [E, K, N] as moe_ffn takes them (bfloat16 or float32) to
    microscaled 4-bit form, blocks of 32 along the contraction K.  gate_up:
    up_proj_weight (N = 2I, gate columns first)."""
    if w.dim() != 3:
        raise ValueError("w [E, K, N] expected")
    if w.dtype not in _WDTYPES:
        raise TypeError("w must be bfloat16 or float32")
    if not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous CUDA tensor")
    E, K, N = w.shape
    return _mx4_of(w, E, N, K, K, HMM_MX4_GATE_UP if gate_up else HMM_MX4_COLUMNS)


@functools.lru_cache(maxsize=64)
def _mx4_call(T, H, I, E, K, weights_dtype):
    """(hmm_shape, workspace bytes) of a shape."""
    shape = HmmShape(T, H, I, E, K, weights_dtype, 0)
    return shape, hmm_mx4_workspace_size(shape)


def moe_ffn_mx4(x, topk_ids, topk_weights, up_proj, down_proj):
    """moe_ffn for inference with microscaled 4-bit expert weights: up_proj and
    down_proj are Mx4Tensors of mx4_quantize_experts (up_proj with gate_up).
    x is rounded to 4-bit blocks along H, the fp32 SwiGLU outputs along I; the
    products accumulate in fp32.  Not differentiable."""
    if up_proj.layout != HMM_MX4_GATE_UP or down_proj.layout != HMM_MX4_COLUMNS:
        raise ValueError("up_proj must be experts with gate_up, down_proj experts without")
    if x.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("x [T, H] and topk_ids [T, K] expected")
    T, H = x.shape
    Tk, K = topk_ids.shape
    E, I = up_proj.batch, up_proj.rows // 2
    if up_proj.cols != H or (down_proj.batch, down_proj.cols, down_proj.rows) != (E, I, H):
        raise ValueError(f"up_proj {up_proj.shape} and down_proj {down_proj.shape} do not match "
                         f"each other and x {tuple(x.shape)}")
    if Tk != T or topk_weights.shape != (T, K):
        raise ValueError("topk_ids / topk_weights must both be [T, K]")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if topk_ids.dtype != torch.int32:
        raise TypeError("topk_ids must be int32")
    wdt = _WDTYPES.get(topk_weights.dtype)
    if wdt is None:
        raise TypeError("topk_weights must be bfloat16 or float32")
    if not (x.is_cuda and topk_ids.is_cuda and topk_weights.is_cuda and x.is_contiguous()
            and topk_ids.is_contiguous() and topk_weights.is_contiguous()):
        raise ValueError("all arguments must be contiguous CUDA tensors")
    dev, at = x.device, x.get_device()
    for t in (topk_ids, topk_weights, up_proj.codes, up_proj.scales, down_proj.codes,
              down_proj.scales):
        if t.get_device() != at:
            raise ValueError(f"all arguments must be on x's device, {dev}, got one on {t.device}")
    if (x.requires_grad or topk_weights.requires_grad) and torch.is_grad_enabled():
        raise RuntimeError("moe_ffn_mx4 has no backward: call it under torch.no_grad(), or train "
                           "with moe_ffn")
    shape, size = _mx4_call(T, H, I, E, K, wdt)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    rc = load_library().hmm_forward_mx4(
        Context.for_device(dev).handle, ctypes.byref(shape), x.data_ptr(), topk_ids.data_ptr(),
        topk_weights.data_ptr(), up_proj.codes.data_ptr(), up_proj.scales.data_ptr(),
        down_proj.codes.data_ptr(), down_proj.scales.data_ptr(), y.data_ptr(), ws.data_ptr(), size,
        _raw_stream(dev.index))
    if rc != HMM_OK:
        raise HmmError(rc, "hmm_forward_mx4")
    return y
