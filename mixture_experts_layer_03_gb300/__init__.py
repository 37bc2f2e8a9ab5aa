"""Python binding of the GB300 MoE layer forward library (libmoe_gb300.so).

Argument marshalling only: every step runs in the library's CUDA kernels. PyTorch
provides device memory and streams. The names mirror the C ABI in include/moe.h.
Importing this module fails loudly when the compiled library is missing; there is
no fallback implementation.

`stream` (a torch stream, or a handle) is the stream of the launch, the current one by
default. What a call allocates, results and workspace, is allocated on that stream; the
order between it and other streams' work on the arguments and results is the caller's.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_ROUTE_DEFAULT = 0
MOE_ROUTE_RENORMALIZE = 1
MOE_ROUTE_DEEPSEEKV3 = 2
MOE_ROUTE_LLAMA4 = 3
MOE_ROUTE_RENORMALIZE_NAIVE = 4
MOE_ROUTE_MINIMAX2 = 5
MOE_ROUTE_SIGMOID_RENORM = 6
MOE_ROUTE_GROUPED_TOPK = 16
MOE_ROUTE_GROUPED_TOPK_SOFTMAX = 17

MOE_REASON_DEGENERATE = 10

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_BAD_ID = 5
MOE_ERR_DEVICE_TIMEOUT = 6
MOE_ERR_NOT_IMPLEMENTED = 7

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2

MOE_FP4_MX = 0
MOE_FP4_NV = 1
MOE_WEIGHTS_16BIT = -1
MOE_FEW_TOKENS = 16

MOE_DEVICE_FLAG_BAD_ID = 1
MOE_DEVICE_FLAG_TIMEOUT = 2


class MoeProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("shared_I", ctypes.c_int32)]


class MoeRouteParams(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("method", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("g", ctypes.c_void_p)]


class MoeWsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("status", "counts", "starts", "offsets", "tile_off1", "tile_off2", "sched", "block_hist",
                 "perm_src", "perm_inv", "x_perm", "h", "out_perm", "total")] + \
               [("rows", ctypes.c_int64), ("groups", ctypes.c_int32), ("n_chunks", ctypes.c_int32),
                ("h_ld", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# Every exported symbol of include/moe.h, with its ctypes signature.
_P = ctypes.c_void_p
_SIGS = {
    "moe_abi_version": (ctypes.c_int32, []),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_route": (ctypes.c_int, [_P, ctypes.c_int64, _P, ctypes.POINTER(MoeRouteParams), _P, _P, _P]),
    "moe_can_implement": (ctypes.c_int, [ctypes.POINTER(MoeProblem), ctypes.POINTER(ctypes.c_int32)]),
    "moe_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MoeProblem)]),
    "moe_workspace_layout": (ctypes.c_int, [ctypes.POINTER(MoeProblem), ctypes.POINTER(MoeWsLayout)]),
    "moe_forward": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P]),
    "moe_forward_static": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, _P, _P, _P, _P,
                                          _P, _P]),
    "moe_forward_partial": (ctypes.c_int, [ctypes.POINTER(MoeProblem), ctypes.c_int32,
                                           ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                           _P, ctypes.c_size_t, _P]),
    "moe_gate": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                ctypes.c_int32, _P, _P, _P]),
    "moe_gate_route": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P,
                                      ctypes.POINTER(MoeRouteParams), _P, _P, _P, _P, _P]),
    "moe_permute": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_fc1": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_fc2": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_fc1_fc2": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, _P, _P, ctypes.c_size_t,
                                   _P]),
    "moe_finalize": (ctypes.c_int, [ctypes.POINTER(MoeProblem), _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_read_device_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_static_read_device_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_selftest_wait": (ctypes.c_int, [_P, _P]),
    "moe_cast_f32_to_bf16": (ctypes.c_int, [_P, _P, ctypes.c_int64, _P]),
    "moe_dispatch_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32,
                                                       ctypes.c_int32]),
    "moe_dispatch": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int32, ctypes.c_int, _P, _P, _P, _P, ctypes.c_size_t,
                                    _P]),
    "moe_dispatch_rows": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int, _P, _P]),
    "moe_dispatch_backward": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, ctypes.c_int, _P, _P]),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                   ctypes.c_int, _P, _P]),
    "moe_combine_backward": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                            ctypes.c_int32, ctypes.c_int, _P, _P, _P]),
    "moe_swiglu_ckpt": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, _P, _P, _P,
                                       _P]),
    "moe_swiglu_ckpt_backward": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                                ctypes.c_int, _P, _P, _P]),
    "moe_experts_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32]),
    "moe_experts_split_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                                  ctypes.c_int32, ctypes.c_int32]),
    "moe_experts_matmul": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                          ctypes.c_int32, ctypes.c_int32, ctypes.c_int, _P, _P,
                                          ctypes.c_size_t, _P]),
    "moe_experts_matmul_dx": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int, _P, _P,
                                             ctypes.c_size_t, _P]),
    "moe_experts_matmul_dw": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int32, _P, _P, ctypes.c_size_t,
                                             _P]),
    "moe_read_timeouts": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_selftest_experts_wait": (ctypes.c_int, [_P]),
    "moe_selftest_fp4_wait": (ctypes.c_int, [_P]),
    "moe_selftest_few_wait": (ctypes.c_int, [_P]),
    "moe_route_backward": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64,
                                          ctypes.POINTER(MoeRouteParams), _P, _P]),
    "moe_quantize_fp4": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                        ctypes.c_int, ctypes.c_int, _P, _P, _P, _P]),
    "moe_swiglu_fp4": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_int,
                                      _P, _P, _P, _P]),
    "moe_dequantize_fp4": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                          ctypes.c_int, ctypes.c_int, _P, _P]),
    "moe_experts_matmul_fp4": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int64,
                                              ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                              ctypes.c_int, ctypes.c_int, _P, _P]),
    "moe_layer_few_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MoeProblem)]),
    "moe_layer_few": (ctypes.c_int, [ctypes.POINTER(MoeProblem), ctypes.POINTER(MoeRouteParams), _P, _P,
                                     ctypes.c_int32, _P] + [ctypes.POINTER(MoeWeights)] * 4 +
                      [ctypes.c_int32, ctypes.c_int, _P, _P, _P, _P, ctypes.c_size_t, _P]),
}
EXPORTED = tuple(_SIGS)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the compiled library and attach the C signatures."""
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.moe_status_string(status).decode()
        detail = _lib.moe_last_error().decode()
        super().__init__(f"{where}: {msg} ({status}) {detail}")
        self.status = status


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without the Stream object around it (2.8 us of a call's 10 on the
# host when it was built for each call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, device, stream, result: bool = True) -> torch.Tensor:
    """Memory that a call launched on `stream` writes. The caching allocator hands a block out again
    in the order of the stream that it was allocated on, so that must be the launch's: one of the
    caller's current stream could still be in use there by work that the launch does not wait for,
    and, dropped on return (a workspace), would be given out again while the kernels run. A result
    is used on the caller's current stream too, and is held until that is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    handle, here = _stream(stream), _stream(None)
    if handle == here:
        return torch.empty(shape, dtype=dtype, device=device)
    # (0, which ExternalStream takes for no handle, and 1 are names of the default stream.)
    where = (torch.cuda.ExternalStream(handle, device) if handle > 1
             else torch.cuda.default_stream(device))
    with torch.cuda.stream(where):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _cuda(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def make_problem(T, H, I, E, k, shared_I=0) -> MoeProblem:
    return MoeProblem(int(T), int(H), int(I), int(E), int(k), int(shared_I))


def moe_can_implement(problem: MoeProblem):
    reason = ctypes.c_int32(0)
    st = _lib.moe_can_implement(ctypes.byref(problem), ctypes.byref(reason))
    return st, reason.value


def moe_workspace_bytes(problem: MoeProblem) -> int:
    return int(_lib.moe_workspace_bytes(ctypes.byref(problem)))


def moe_workspace_layout(problem: MoeProblem) -> dict:
    L = MoeWsLayout()
    _check(_lib.moe_workspace_layout(ctypes.byref(problem), ctypes.byref(L)), "moe_workspace_layout")
    return {n: getattr(L, n) for n, _ in MoeWsLayout._fields_}


@dataclass
class Workspace:
    """Caller-owned device workspace (a torch byte buffer, 1024-byte aligned view)."""
    problem: MoeProblem
    buf: torch.Tensor
    base: int           # byte offset of the aligned start inside buf
    nbytes: int
    layout: dict

    @property
    def ptr(self) -> ctypes.c_void_p:
        return ctypes.c_void_p(self.buf.data_ptr() + self.base)

    def region(self, name: str, count: int, dtype: torch.dtype) -> torch.Tensor:
        off = self.base + self.layout[name]
        nbytes = count * torch.empty((), dtype=dtype).element_size()
        return self.buf[off:off + nbytes].view(dtype)


def alloc_workspace(problem: MoeProblem, device="cuda", stream=None) -> Workspace:
    """The forward's workspace, for calls on `stream` (None: the current one)."""
    n = moe_workspace_bytes(problem)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_workspace_bytes")
    buf = _new(n + 1024, torch.uint8, device, stream, result=False)
    base = (-buf.data_ptr()) % 1024
    return Workspace(problem, buf, base, n, moe_workspace_layout(problem))


def moe_route(logits: torch.Tensor, method: int, top_k: int, bias: Optional[torch.Tensor] = None,
              n_group: int = 1, topk_group: int = 1, routed_scaling_factor: float = 1.0,
              ids: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
              stream=None):
    """Routing: logits fp32 [T, E] -> (ids int32 [T, k], scales fp32 [T, k])."""
    _cuda(logits, "logits", torch.float32)
    T, E = logits.shape
    if bias is not None:
        _cuda(bias, "bias", torch.float32)
    if ids is None:
        ids = _new((T, top_k), torch.int32, logits.device, stream)
    if scales is None:
        scales = _new((T, top_k), torch.float32, logits.device, stream)
    p = MoeRouteParams(E, top_k, method, n_group, topk_group, routed_scaling_factor)
    _check(_lib.moe_route(_ptr(logits), T, _ptr(bias), ctypes.byref(p), _ptr(ids), _ptr(scales),
                          _stream(stream)), "moe_route")
    return ids, scales


def _problem_for(x, ids, w13, w2, w13_s):
    T, H = x.shape
    k = ids.shape[1]
    E, twoI, _ = w13.shape
    return make_problem(T, H, twoI // 2, E, k, 0 if w13_s is None else w13_s.shape[0] // 2)


def moe_forward(x, ids, scales, w13, w2, w13_s=None, w2_s=None, y=None,
                workspace: Optional[Workspace] = None, stream=None):
    """Steps 2-5: permute, FC1+SwiGLU, FC2, finalize. Returns y bf16 [T, H]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(ids, "ids", torch.int32)
    _cuda(scales, "scales", torch.float32)
    _cuda(w13, "w13", torch.bfloat16)
    _cuda(w2, "w2", torch.bfloat16)
    p = _problem_for(x, ids, w13, w2, w13_s)
    if workspace is None:
        workspace = alloc_workspace(p, x.device, stream)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    _check(_lib.moe_forward(ctypes.byref(p), _ptr(x), _ptr(ids), _ptr(scales), _ptr(w13), _ptr(w2),
                            _ptr(w13_s), _ptr(w2_s), _ptr(y), workspace.ptr, workspace.nbytes,
                            _stream(stream)), "moe_forward")
    return y


def moe_forward_partial(x, ids, scales, w13_local, w2_local, e_lo: int, e_hi: int, num_experts: int,
                        w13_s=None, w2_s=None, shared_gate=None, y=None,
                        workspace: Optional[Workspace] = None, stream=None):
    """moe_forward over the experts [e_lo, e_hi) of num_experts only (the expert-parallel
    seam): slots routed elsewhere contribute 0. w13_local / w2_local hold those experts'
    weights, [e_hi - e_lo, 2I, H] / [e_hi - e_lo, H, I]. shared_gate: fp32 [T] logits that
    weight the shared expert by their sigmoid (None: weight 1). Returns y bf16 [T, H]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(ids, "ids", torch.int32)
    _cuda(scales, "scales", torch.float32)
    _cuda(w13_local, "w13_local", torch.bfloat16)
    _cuda(w2_local, "w2_local", torch.bfloat16)
    T, H = x.shape
    k = ids.shape[1]
    I = w2_local.shape[2]
    shared_I = 0 if w13_s is None else w13_s.shape[0] // 2
    p = make_problem(T, H, I, num_experts, k, shared_I)
    if workspace is None:
        workspace = alloc_workspace(p, x.device, stream)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    if shared_gate is not None:
        _cuda(shared_gate, "shared_gate", torch.float32)
    _check(_lib.moe_forward_partial(ctypes.byref(p), int(e_lo), int(e_hi), _ptr(x), _ptr(ids),
                                    _ptr(scales), _ptr(w13_local), _ptr(w2_local), _ptr(w13_s),
                                    _ptr(w2_s), _ptr(shared_gate), _ptr(y), workspace.ptr,
                                    workspace.nbytes, _stream(stream)), "moe_forward_partial")
    return y


def moe_gate(x, wg, num_experts: int, routed_logits=None, shared_logits=None, stream=None):
    """Router gate: x bf16 [T, H] . wg bf16 [E (+1), H]^T -> (routed logits fp32 [T, E],
    shared-expert gate logits fp32 [T] or None). A wg with E + 1 rows carries the fused
    shared-expert gate in its last row."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(wg, "wg", torch.bfloat16)
    T, H = x.shape
    E = int(num_experts)
    n_shared = wg.shape[0] - E
    if n_shared not in (0, 1) or wg.shape[1] != H:
        raise ValueError(f"wg must be [{E} or {E + 1}, {H}], got {tuple(wg.shape)}")
    if routed_logits is None:
        routed_logits = _new((T, E), torch.float32, x.device, stream)
    if n_shared and shared_logits is None:
        shared_logits = _new((T,), torch.float32, x.device, stream)
    _check(_lib.moe_gate(_ptr(x), _ptr(wg), T, H, E, n_shared, _ptr(routed_logits),
                         _ptr(shared_logits) if n_shared else None, _stream(stream)), "moe_gate")
    return routed_logits, (shared_logits if n_shared else None)


def moe_gate_route(x, wg, method: int, top_k: int, num_experts: int,
                   bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                   routed_scaling_factor: float = 1.0, ids=None, scales=None,
                   routed_logits=None, shared_logits=None, want_logits: bool = False,
                   stream=None):
    """Router gate and routing in one launch: x bf16 [T, H], wg bf16 [E (+1), H] ->
    (ids int32 [T, k], scales fp32 [T, k], routed logits fp32 [T, E] or None, shared-expert
    gate logits fp32 [T] or None). The routed logits are written only when want_logits is
    set or routed_logits is passed."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(wg, "wg", torch.bfloat16)
    T, H = x.shape
    E = int(num_experts)
    n_shared = wg.shape[0] - E
    if n_shared not in (0, 1) or wg.shape[1] != H:
        raise ValueError(f"wg must be [{E} or {E + 1}, {H}], got {tuple(wg.shape)}")
    if bias is not None:
        _cuda(bias, "bias", torch.float32)
    if ids is None:
        ids = _new((T, top_k), torch.int32, x.device, stream)
    if scales is None:
        scales = _new((T, top_k), torch.float32, x.device, stream)
    if want_logits and routed_logits is None:
        routed_logits = _new((T, E), torch.float32, x.device, stream)
    if n_shared and shared_logits is None:
        shared_logits = _new((T,), torch.float32, x.device, stream)
    p = MoeRouteParams(E, top_k, method, n_group, topk_group, routed_scaling_factor)
    _check(_lib.moe_gate_route(_ptr(x), _ptr(wg), T, H, n_shared, _ptr(bias), ctypes.byref(p),
                               _ptr(ids), _ptr(scales), _ptr(routed_logits),
                               _ptr(shared_logits) if n_shared else None, _stream(stream)),
           "moe_gate_route")
    return ids, scales, routed_logits, (shared_logits if n_shared else None)


MOE_STATIC_SCRATCH_BYTES = 32 << 20


def moe_forward_static(x, ids, scales, w13, w2, w13_s=None, w2_s=None, y=None, stream=None):
    """moe_forward with the library's built-in scratch instead of a caller workspace.

    For callers that cannot allocate device memory (a plugin whose host engine owns all
    device allocations, or a loop that must not call cudaMalloc). Problems whose workspace
    exceeds MOE_STATIC_SCRATCH_BYTES are rejected. All calls on a GPU share one scratch
    array, so calls that overlap on the GPU race; the first call on a device sets the
    array up and should come before any stream capture. ``y`` is allocated here (by
    torch) only when the caller does not pass it.
    """
    _cuda(x, "x", torch.bfloat16)
    _cuda(ids, "ids", torch.int32)
    _cuda(scales, "scales", torch.float32)
    _cuda(w13, "w13", torch.bfloat16)
    _cuda(w2, "w2", torch.bfloat16)
    p = _problem_for(x, ids, w13, w2, w13_s)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    _check(_lib.moe_forward_static(ctypes.byref(p), _ptr(x), _ptr(ids), _ptr(scales), _ptr(w13),
                                   _ptr(w2), _ptr(w13_s), _ptr(w2_s), _ptr(y), _stream(stream)),
           "moe_forward_static")
    return y


def moe_permute(problem, x, ids, workspace: Workspace, stream=None):
    _check(_lib.moe_permute(ctypes.byref(problem), _ptr(x), _ptr(ids), workspace.ptr,
                            workspace.nbytes, _stream(stream)), "moe_permute")


def moe_fc1(problem, w13, w13_s, workspace: Workspace, stream=None):
    _check(_lib.moe_fc1(ctypes.byref(problem), _ptr(w13), _ptr(w13_s), workspace.ptr,
                        workspace.nbytes, _stream(stream)), "moe_fc1")


def moe_fc2(problem, w2, w2_s, workspace: Workspace, stream=None):
    _check(_lib.moe_fc2(ctypes.byref(problem), _ptr(w2), _ptr(w2_s), workspace.ptr,
                        workspace.nbytes, _stream(stream)), "moe_fc2")


def moe_fc1_fc2(problem, w13, w13_s, w2, w2_s, workspace: Workspace, stream=None):
    _check(_lib.moe_fc1_fc2(ctypes.byref(problem), _ptr(w13), _ptr(w13_s), _ptr(w2), _ptr(w2_s),
                            workspace.ptr, workspace.nbytes, _stream(stream)), "moe_fc1_fc2")


def moe_finalize(problem, scales, y, workspace: Workspace, stream=None):
    _check(_lib.moe_finalize(ctypes.byref(problem), _ptr(scales), _ptr(y), workspace.ptr,
                             workspace.nbytes, _stream(stream)), "moe_finalize")


def moe_read_device_status(workspace: Workspace, stream=None):
    """Synchronise, read and clear the device status word. Returns (status, flags)."""
    flags = ctypes.c_int32(0)
    st = _lib.moe_read_device_status(workspace.ptr, _stream(stream), ctypes.byref(flags))
    return st, flags.value


def moe_static_read_device_status(stream=None):
    """Synchronise, read and clear moe_forward_static's status word on the current device.
    Returns (status, flags)."""
    flags = ctypes.c_int32(0)
    st = _lib.moe_static_read_device_status(_stream(stream), ctypes.byref(flags))
    return st, flags.value


def moe_selftest_wait(workspace: Workspace, stream=None):
    """Enqueue the device failure-path self-test on ``workspace``'s status words: a
    bounded wait that runs out after about 2 s and reports MOE_DEVICE_FLAG_TIMEOUT."""
    _check(_lib.moe_selftest_wait(workspace.ptr, _stream(stream)), "moe_selftest_wait")


def moe_cast_f32_to_bf16(t: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    _cuda(t, "input", torch.float32)
    if out is None:
        out = _new(t.shape, torch.bfloat16, t.device, stream)
    _check(_lib.moe_cast_f32_to_bf16(_ptr(t), _ptr(out), t.numel(), _stream(stream)),
           "moe_cast_f32_to_bf16")
    return out


# ------------------------------------------------------------------ training operators

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16,
           torch.float32: MOE_DTYPE_F32}


@dataclass
class Scratch:
    """Caller-owned device workspace of a training operator; moe_read_device_status takes it."""
    buf: torch.Tensor

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def alloc_dispatch_scratch(T: int, num_experts: int, top_k: int, device="cuda",
                           stream=None) -> Scratch:
    """Workspace of moe_dispatch for T tokens, for calls on `stream` (None: the current one)."""
    n = _lib.moe_dispatch_workspace_bytes(T, num_experts, top_k)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_dispatch_workspace_bytes")
    return Scratch(_new(n, torch.uint8, device, stream, result=False))


def alloc_experts_scratch(num_experts: int, rows: int = 0, N: int = 8, K: int = 8,
                          device="cuda") -> Scratch:
    """Workspace of the experts' products (all three), its status word cleared. With the sizes
    given, large enough for each of them to split its contraction."""
    n = _lib.moe_experts_workspace_bytes(num_experts)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_experts_workspace_bytes")
    n = max(n, *(_lib.moe_experts_split_bytes(p, rows, num_experts, N, K) for p in range(3)))
    scratch = Scratch(torch.empty(n, dtype=torch.uint8, device=device))
    scratch.buf[:16].zero_()
    return scratch


def _split_scratch(product: int, R: int, E: int, N: int, K: int, device,
                   stream) -> Optional[Scratch]:
    """A workspace for one call whose contraction is split, else None. (Nobody reads its status word;
    moe_read_timeouts has what it would say.)"""
    n = _lib.moe_experts_split_bytes(product, R, E, N, K)
    return Scratch(_new(n, torch.uint8, device, stream, result=False)) if n else None


# The checks below are on the path of calls that take a few microseconds on the device: one
# condition decides the usual case, what is wrong is worked out after it.

def _typed(t: torch.Tensor, name: str, ndim: int) -> int:
    """The moe_dtype of a contiguous CUDA tensor of `ndim` dimensions."""
    code = _DTYPES.get(t.dtype)
    if code is not None and t.is_cuda and t.is_contiguous() and t.dim() == ndim:
        return code
    _cuda(t, name)
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")


def _shaped(t: torch.Tensor, name: str, shape: tuple, dtype) -> torch.Tensor:
    """t, a contiguous CUDA tensor of just this shape and type."""
    if t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t
    _cuda(t, name, dtype)
    raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")


def _like(t: torch.Tensor, out: Optional[torch.Tensor], name: str, shape: tuple,
          stream) -> torch.Tensor:
    """`out`, of just this shape and t's type, or a new tensor. (t.new_empty() goes through torch's
    dispatcher twice: 2 us more between two launches.)"""
    return _new(shape, t.dtype, t.device, stream) if out is None else _shaped(
        out, name, shape, t.dtype)


def _slots(inv: torch.Tensor, name: str = "inv"):
    if inv.dtype is not torch.int32 or not inv.is_cuda or not inv.is_contiguous():
        _cuda(inv, name, torch.int32)
    if inv.dim() != 2:
        raise ValueError(f"{name} must be [T, k], got {tuple(inv.shape)}")
    return inv.shape


MOE_DISPATCH_SMALL_SLOTS = 12288


def moe_dispatch(x, ids, num_experts: int, x_perm=None, inv=None, offsets=None,
                 scratch: Optional[Scratch] = None, stream=None):
    """Rows of x [T, H] sorted by expert. ids int32 [T, k], -1 for a dropped slot. Returns
    (x_perm [T*k, H], inv int32 [T, k], offsets int32 [E + 1]): rows of expert e are
    x_perm[offsets[e]:offsets[e + 1]], inv the row of each slot (-1 - row of a dropped one, whose
    row holds zeros). Pass a scratch to read back (moe_read_device_status) whether an id was
    neither -1 nor an expert."""
    dt = _typed(x, "x", 2)
    T, H = x.shape
    if _slots(ids, "ids")[0] != T:
        raise ValueError(f"ids must have {T} rows, got {tuple(ids.shape)}")
    k = ids.shape[1]
    x_perm = _like(x, x_perm, "x_perm", (T * k, H), stream)
    inv = _like(ids, inv, "inv", (T, k), stream)
    offsets = _like(ids, offsets, "offsets", (num_experts + 1,), stream)
    if scratch is None and T * k > MOE_DISPATCH_SMALL_SLOTS:
        scratch = alloc_dispatch_scratch(T, num_experts, k, x.device, stream)
    _check(_lib.moe_dispatch(x.data_ptr(), ids.data_ptr(), T, H, num_experts, k, dt,
                             x_perm.data_ptr(), inv.data_ptr(),
                             offsets.data_ptr(), scratch.ptr if scratch else None,
                             scratch.nbytes if scratch else 0, _stream(stream)), "moe_dispatch")
    return x_perm, inv, offsets


def moe_dispatch_rows(x, inv, x_perm=None, stream=None):
    """moe_dispatch's x_perm again, by the inv it returned."""
    dt = _typed(x, "x", 2)
    T, k = _slots(inv)
    H = x.shape[1]
    if x.shape[0] != T:
        raise ValueError(f"x must have {T} rows, got {tuple(x.shape)}")
    x_perm = _like(x, x_perm, "x_perm", (T * k, H), stream)
    _check(_lib.moe_dispatch_rows(x.data_ptr(), inv.data_ptr(), T, H, k, dt, x_perm.data_ptr(), _stream(stream)),
           "moe_dispatch_rows")
    return x_perm


def moe_dispatch_backward(dx_perm, inv, dx=None, stream=None):
    """Gradient of moe_dispatch: dx [T, H], each token's kept rows of dx_perm [T*k, H] summed."""
    dt = _typed(dx_perm, "dx_perm", 2)
    T, k = _slots(inv)
    H = dx_perm.shape[1]
    _shaped(dx_perm, "dx_perm", (T * k, H), dx_perm.dtype)
    dx = _like(dx_perm, dx, "dx", (T, H), stream)
    _check(_lib.moe_dispatch_backward(dx_perm.data_ptr(), inv.data_ptr(), T, H, k, dt, dx.data_ptr(),
                                      _stream(stream)), "moe_dispatch_backward")
    return dx


def moe_combine(rows, inv, scales=None, y=None, stream=None):
    """Back to token order: y [T, H] = sum of each token's kept rows [T*k, H], weighted by scales
    fp32 [T, k] (None: 1)."""
    dt = _typed(rows, "rows", 2)
    T, k = _slots(inv)
    H = rows.shape[1]
    _shaped(rows, "rows", (T * k, H), rows.dtype)
    if scales is not None:
        _shaped(scales, "scales", (T, k), torch.float32)
    y = _like(rows, y, "y", (T, H), stream)
    _check(_lib.moe_combine(rows.data_ptr(), inv.data_ptr(), _ptr(scales), T, H, k, dt, y.data_ptr(),
                            _stream(stream)), "moe_combine")
    return y


def moe_combine_backward(dy, rows, inv, scales=None, drows=None, dscales=None, stream=None):
    """Gradients of moe_combine: (drows [T*k, H], dscales fp32 [T, k])."""
    dt = _typed(dy, "dy", 2)
    T, k = _slots(inv)
    H = dy.shape[1]
    _shaped(dy, "dy", (T, H), dy.dtype)
    _shaped(rows, "rows", (T * k, H), dy.dtype)
    if scales is not None:
        _shaped(scales, "scales", (T, k), torch.float32)
    drows = _like(rows, drows, "drows", (T * k, H), stream)
    dscales = (_new((T, k), torch.float32, dy.device, stream) if dscales is None
               else _shaped(dscales, "dscales", (T, k), torch.float32))
    _check(_lib.moe_combine_backward(dy.data_ptr(), rows.data_ptr(), inv.data_ptr(), _ptr(scales), T, H, k, dt,
                                     drows.data_ptr(), dscales.data_ptr(), _stream(stream)),
           "moe_combine_backward")
    return drows, dscales


MOE_CKPT_BLOCK = 32


class Checkpoint:
    """What moe_swiglu_ckpt keeps of gu [R, 2I]: the e4m3 codes q [R, 2I] and the exponent bytes
    q_scales [R, 2 * ceil(I / 32)] (scale 2^(byte - 127)), in one buffer `buf` (uint8; to be saved
    between the passes). Unpacks and indexes as (q, q_scales)."""
    __slots__ = ("buf", "R", "I")

    def __init__(self, buf: torch.Tensor, R: int, I: int):
        if buf.dtype is not torch.uint8 or buf.numel() < self.nbytes(R, I):
            raise ValueError(f"a checkpoint of [{R}, {2 * I}] takes {self.nbytes(R, I)} bytes (uint8)")
        self.buf, self.R, self.I = buf, R, I

    @staticmethod
    def scales_at(R: int, I: int) -> int:
        return (R * 2 * I + 15) // 16 * 16

    @staticmethod
    def nbytes(R: int, I: int) -> int:
        return Checkpoint.scales_at(R, I) + R * 2 * (-(-I // MOE_CKPT_BLOCK))

    @property
    def q(self) -> torch.Tensor:
        return self.buf[:self.R * 2 * self.I].view(self.R, 2 * self.I)

    @property
    def q_scales(self) -> torch.Tensor:
        return self.buf[self.scales_at(self.R, self.I):self.nbytes(self.R, self.I)].view(
            self.R, 2 * (-(-self.I // MOE_CKPT_BLOCK)))

    def __len__(self):
        return 2

    def __getitem__(self, i):
        return (self.q, self.q_scales)[i]


def _ckpt_ptrs(ckpt, R: int, I: int):
    """Addresses of the codes and the scales of a Checkpoint, or of a pair of tensors."""
    if type(ckpt) is Checkpoint:
        if ckpt.R != R or ckpt.I != I or not ckpt.buf.is_cuda or not ckpt.buf.is_contiguous():
            raise ValueError(f"the checkpoint must be of [{R}, {2 * I}], contiguous, on the GPU")
        at = ckpt.buf.data_ptr()
        return at, at + Checkpoint.scales_at(R, I)
    q, qs = ckpt
    return (_shaped(q, "q", (R, 2 * I), torch.uint8).data_ptr(),
            _shaped(qs, "q_scales", (R, 2 * (-(-I // MOE_CKPT_BLOCK))), torch.uint8).data_ptr())


def moe_swiglu_ckpt(gu, h=None, ckpt=None, stream=None):
    """SwiGLU that keeps its input in 8 bits. gu [R, 2I], gate then up. Returns (h [R, I], a
    Checkpoint, for moe_swiglu_ckpt_backward). ckpt: a Checkpoint, or the pair (q, q_scales), to
    write to."""
    dt = _typed(gu, "gu", 2)
    R, I2 = gu.shape
    if I2 % 2:
        raise ValueError(f"gu must have an even number of columns, got {I2}")
    I = I2 // 2
    h = _like(gu, h, "h", (R, I), stream)
    if ckpt is None:
        ckpt = Checkpoint(_new(Checkpoint.nbytes(R, I), torch.uint8, gu.device, stream), R, I)
    q, qs = _ckpt_ptrs(ckpt, R, I)
    _check(_lib.moe_swiglu_ckpt(gu.data_ptr(), R, I, dt, h.data_ptr(), q, qs, _stream(stream)),
           "moe_swiglu_ckpt")
    return h, ckpt


def moe_swiglu_ckpt_backward(dh, ckpt, dgu=None, h=None, want_h: bool = False, stream=None):
    """Gradient of moe_swiglu_ckpt at the kept values: (dgu [R, 2I], h [R, I] again or None)."""
    dt = _typed(dh, "dh", 2)
    R, I = dh.shape
    q, qs = _ckpt_ptrs(ckpt, R, I)
    dgu = _like(dh, dgu, "dgu", (R, 2 * I), stream)
    if h is not None:
        _shaped(h, "h", (R, I), dh.dtype)
    elif want_h:
        h = _new((R, I), dh.dtype, dh.device, stream)
    _check(_lib.moe_swiglu_ckpt_backward(dh.data_ptr(), q, qs, R, I, dt, dgu.data_ptr(), _ptr(h),
                                         _stream(stream)), "moe_swiglu_ckpt_backward")
    return dgu, h


def _offsets(offsets, E):
    return _shaped(offsets, "offsets", (E + 1,), torch.int32)


def moe_experts_matmul(x, w, offsets, y=None, scratch: Optional[Scratch] = None, stream=None):
    """y [R, N]: each row of x [R, K] times its expert's w[e]^T (w [E, N, K]); rows
    [offsets[e], offsets[e + 1]) are expert e's, rows of no expert are zeros in y."""
    dt = _typed(x, "x", 2)
    _shaped(w, "w", (w.shape[0], w.shape[1], x.shape[1]) if w.dim() == 3 else (0, 0, 0), x.dtype)
    E, N, K = w.shape
    R = x.shape[0]
    y = _like(x, y, "y", (R, N), stream)
    if scratch is None:
        scratch = _split_scratch(0, R, E, N, K, x.device, stream)
    _check(_lib.moe_experts_matmul(x.data_ptr(), w.data_ptr(), _offsets(offsets, E).data_ptr(), R,
                                   E, N, K, dt, y.data_ptr(), scratch.ptr if scratch else None,
                                   scratch.nbytes if scratch else 0, _stream(stream)),
           "moe_experts_matmul")
    return y


def moe_experts_matmul_dx(dy, w, offsets, dx=None, scratch: Optional[Scratch] = None, stream=None):
    """Gradient of moe_experts_matmul to its rows: dx [R, K] = each row of dy [R, N] times its
    expert's w[e]."""
    dt = _typed(dy, "dy", 2)
    _shaped(w, "w", (w.shape[0], dy.shape[1], w.shape[2]) if w.dim() == 3 else (0, 0, 0), dy.dtype)
    E, N, K = w.shape
    R = dy.shape[0]
    dx = _like(dy, dx, "dx", (R, K), stream)
    if scratch is None:
        scratch = _split_scratch(1, R, E, N, K, dy.device, stream)
    _check(_lib.moe_experts_matmul_dx(dy.data_ptr(), w.data_ptr(), _offsets(offsets, E).data_ptr(),
                                      R, E, N, K, dt, dx.data_ptr(),
                                      scratch.ptr if scratch else None,
                                      scratch.nbytes if scratch else 0, _stream(stream)),
           "moe_experts_matmul_dx")
    return dx


def moe_experts_matmul_dw(dy, x, offsets, dw=None, dw_dtype=None, accumulate: bool = False,
                          scratch: Optional[Scratch] = None, stream=None):
    """Gradient of moe_experts_matmul to the weights: dw [E, N, K] = for each expert, dy^T x over
    its rows. dw is of the inputs' type, or fp32 (dw_dtype, or a dw given); accumulate adds to a
    given fp32 dw."""
    dt = _typed(dy, "dy", 2)
    _cuda(offsets, "offsets", torch.int32)
    E = offsets.numel() - 1
    _offsets(offsets, E)
    R, N = dy.shape
    _shaped(x, "x", (R, x.shape[-1]), dy.dtype)
    K = x.shape[1]
    if accumulate and dw is None:
        raise ValueError("accumulate needs the dw to add to")
    if dw is None:
        dw = _new((E, N, K), dw_dtype or dy.dtype, dy.device, stream)
    out = _typed(dw, "dw", 3)
    _shaped(dw, "dw", (E, N, K), dw_dtype or dw.dtype)
    if scratch is None:
        n = _lib.moe_experts_split_bytes(2, R, E, N, K) or _lib.moe_experts_workspace_bytes(E)
        scratch = Scratch(_new(max(n, 1), torch.uint8, dy.device, stream, result=False))
    _check(_lib.moe_experts_matmul_dw(dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), R, E, N, K,
                                      dt, out, int(accumulate), dw.data_ptr(), scratch.ptr, scratch.nbytes,
                                      _stream(stream)), "moe_experts_matmul_dw")
    return dw


def moe_read_timeouts(stream=None):
    """Synchronise; read and clear whether a wait of the experts' products (on 16-bit or 4-bit operands),
    of the gate or of moe_layer_few ran out in any call on the current GPU since the last read (its
    results are incomplete then), whether or not the call was given a scratch. Returns (status,
    flags)."""
    flags = ctypes.c_int32(0)
    st = _lib.moe_read_timeouts(_stream(stream), ctypes.byref(flags))
    return st, flags.value


def moe_selftest_experts_wait(stream=None):
    """Enqueue the self-test of moe_read_timeouts: a bounded wait that runs out after about 2 s."""
    _check(_lib.moe_selftest_experts_wait(_stream(stream)), "moe_selftest_experts_wait")


def moe_selftest_fp4_wait(stream=None):
    """The same of the products on 4-bit operands."""
    _check(_lib.moe_selftest_fp4_wait(_stream(stream)), "moe_selftest_fp4_wait")


def moe_selftest_few_wait(stream=None):
    """The same of moe_layer_few."""
    _check(_lib.moe_selftest_few_wait(_stream(stream)), "moe_selftest_few_wait")


def moe_route_backward(logits, ids, dscales, method: int, routed_scaling_factor: float = 1.0,
                       dlogits=None, stream=None):
    """Gradient of moe_route's scales to its logits: dlogits fp32 [T, E] from logits [T, E], the ids
    [T, k] it chose and dscales [T, k]."""
    _cuda(logits, "logits", torch.float32)
    T, k = _slots(ids, "ids")
    E = logits.shape[-1]
    _shaped(logits, "logits", (T, E), torch.float32)
    _shaped(dscales, "dscales", (T, k), torch.float32)
    dlogits = _like(logits, dlogits, "dlogits", (T, E), stream)
    p = MoeRouteParams(E, k, method, 1, 1, routed_scaling_factor)
    _check(_lib.moe_route_backward(logits.data_ptr(), ids.data_ptr(), dscales.data_ptr(), T, ctypes.byref(p),
                                   dlogits.data_ptr(), _stream(stream)), "moe_route_backward")
    return dlogits


# ------------------------------------------------------------------ 4-bit operands

_FP4_BLOCK = {MOE_FP4_MX: 32, MOE_FP4_NV: 16}


class Fp4:
    """A tensor [rows, K] or [planes, rows, K] in microscaled 4-bit floating point. codes: uint8
    [..., K / 2], two e2m1 numbers a byte, the lower channel in the low half. scales: uint8
    [..., S], one for each block of 32 (MOE_FP4_MX: 2^(byte - 127)) or 16 (MOE_FP4_NV: e4m3) channels,
    S = K / block rounded up to a multiple of 16; what fills a row up is not looked at. g: f32, the
    factor of all of a matrix (1 element) or of each plane (MOE_FP4_NV; None: 1)."""
    __slots__ = ("codes", "scales", "format", "g")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, format: int,
                 g: Optional[torch.Tensor] = None):
        if format not in _FP4_BLOCK:
            raise ValueError(f"format must be MOE_FP4_MX or MOE_FP4_NV, got {format}")
        if codes.dim() not in (2, 3):
            raise ValueError(f"codes must be [rows, K / 2] or [planes, rows, K / 2], got {tuple(codes.shape)}")
        shape = codes.shape
        _shaped(codes, "codes", shape, torch.uint8)
        _shaped(scales, "scales", shape[:-1] + (self.scale_columns(2 * shape[-1], format),), torch.uint8)
        if g is not None:
            if format != MOE_FP4_NV:
                raise ValueError("only MOE_FP4_NV has a g")
            _shaped(g, "g", (shape[0] if len(shape) == 3 else 1,), torch.float32)
            if g.device != codes.device:
                raise ValueError("g must be on the codes' device")
        if scales.device != codes.device:
            raise ValueError("scales must be on the codes' device")
        self.codes, self.scales, self.format, self.g = codes, scales, format, g

    @classmethod
    def _of(cls, codes, scales, format, g) -> "Fp4":
        """Of parts that this module has made or checked."""
        q = cls.__new__(cls)
        q.codes, q.scales, q.format, q.g = codes, scales, format, g
        return q

    @staticmethod
    def scale_columns(K: int, format: int) -> int:
        return (K // _FP4_BLOCK[format] + 15) // 16 * 16

    @property
    def shape(self) -> tuple:
        return tuple(self.codes.shape[:-1]) + (2 * self.codes.shape[-1],)


def _new_fp4(shape, format: int, g, device, stream, out: Optional[Fp4]) -> Fp4:
    if format not in _FP4_BLOCK:
        raise ValueError(f"format must be MOE_FP4_MX or MOE_FP4_NV, got {format}")
    if shape[-1] % 32:
        raise ValueError(f"4-bit rows must be a multiple of 32 channels, got {shape[-1]}")
    if out is not None:
        if out.shape != tuple(shape) or out.format != format or out.codes.device != device:
            raise ValueError(f"out must be of {tuple(shape)} and the same format, got {out.shape}")
        return Fp4(out.codes, out.scales, format, g)
    if g is not None:
        if format != MOE_FP4_NV:
            raise ValueError("only MOE_FP4_NV has a g")
        _shaped(g, "g", (shape[0] if len(shape) == 3 else 1,), torch.float32)
        if g.device != device:
            raise ValueError("g must be on the rows' device")
    head, K = tuple(shape[:-1]), shape[-1]
    return Fp4._of(_new(head + (K // 2,), torch.uint8, device, stream),
                   _new(head + (Fp4.scale_columns(K, format),), torch.uint8, device, stream), format, g)


def _written_fp4(q: Fp4, out: Optional[Fp4]) -> Fp4:
    """What a conversion returns: `out`, where one was given, with the g that its new values stand for."""
    if out is None:
        return q
    out.g = q.g
    return out


def moe_quantize_fp4(x, format: int, g: Optional[torch.Tensor] = None, out: Optional[Fp4] = None,
                     stream=None) -> Fp4:
    """x [rows, K] or [planes, rows, K] in 4 bits (MOE_FP4_MX or MOE_FP4_NV). g (MOE_FP4_NV): f32, one
    value or one for each plane, by which values are divided first: amax / (6 * 448) uses all of the
    scales' range; kept in the result. out: an Fp4 whose codes and scales are written and whose g becomes
    this one; returned."""
    dt = _typed(x, "x", 3 if x.dim() == 3 else 2)
    q = _new_fp4(x.shape, format, g, x.device, stream, out)
    planes = x.shape[0] if x.dim() == 3 else 1
    _check(_lib.moe_quantize_fp4(x.data_ptr(), planes, x.shape[-2], x.shape[-1], dt, format, _ptr(g),
                                 q.codes.data_ptr(), q.scales.data_ptr(), _stream(stream)),
           "moe_quantize_fp4")
    return _written_fp4(q, out)


def moe_swiglu_fp4(gu, format: int, g: Optional[torch.Tensor] = None, out: Optional[Fp4] = None,
                   stream=None) -> Fp4:
    """SwiGLU of gu [R, 2I] (gate, then up), its result [R, I] in 4 bits, as moe_quantize_fp4's."""
    dt = _typed(gu, "gu", 2)
    R, I2 = gu.shape
    if I2 % 2:
        raise ValueError(f"gu must have an even number of columns, got {I2}")
    q = _new_fp4((R, I2 // 2), format, g, gu.device, stream, out)
    _check(_lib.moe_swiglu_fp4(gu.data_ptr(), R, I2 // 2, dt, format, _ptr(g), q.codes.data_ptr(),
                               q.scales.data_ptr(), _stream(stream)), "moe_swiglu_fp4")
    return _written_fp4(q, out)


def moe_dequantize_fp4(q: Fp4, dtype=torch.bfloat16, out=None, stream=None):
    """The values that q stands for, in bfloat16, float16 or float32."""
    if out is None:
        out = _new(q.shape, dtype, q.codes.device, stream)
    else:
        _shaped(out, "out", q.shape, dtype)
    shape = q.shape
    dt = _typed(out, "out", len(shape))
    planes = shape[0] if len(shape) == 3 else 1
    _check(_lib.moe_dequantize_fp4(q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.g), planes, shape[-2],
                                   shape[-1], q.format, dt, out.data_ptr(), _stream(stream)),
           "moe_dequantize_fp4")
    return out


def moe_experts_matmul_fp4(x: Fp4, w: Fp4, offsets, dtype=torch.bfloat16, y=None, stream=None):
    """moe_experts_matmul with both operands in 4 bits of the same format: y [R, N] of `dtype` (bfloat16
    or float16) from x [R, K] and w [E, N, K]."""
    if len(x.shape) != 2 or len(w.shape) != 3 or x.shape[1] != w.shape[2] or x.format != w.format:
        raise ValueError(f"x must be [R, K] and w [E, N, K] of one format, got {x.shape} and {w.shape}")
    E, N, K = w.shape
    R = x.shape[0]
    if y is None:
        y = _new((R, N), dtype, x.codes.device, stream)
    else:
        _shaped(y, "y", (R, N), dtype)
    _check(_lib.moe_experts_matmul_fp4(x.codes.data_ptr(), x.scales.data_ptr(), _ptr(x.g),
                                       w.codes.data_ptr(), w.scales.data_ptr(), _ptr(w.g),
                                       _offsets(offsets, E).data_ptr(), R, E, N, K, x.format,
                                       _typed(y, "y", 2), y.data_ptr(), _stream(stream)),
           "moe_experts_matmul_fp4")
    return y


def alloc_few_scratch(problem: MoeProblem, device="cuda", stream=None) -> Scratch:
    """Workspace of moe_layer_few, for calls on `stream` (None: the current one)."""
    n = _lib.moe_layer_few_workspace_bytes(ctypes.byref(problem))
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_layer_few_workspace_bytes")
    return Scratch(_new(n, torch.uint8, device, stream, result=False))


@functools.lru_cache(maxsize=256)
def _few_plan(T, H, I, E, k, shared_I, method, n_group, topk_group, rsf):
    """What the library is told of a layer's sizes and routing, and the workspace's size."""
    p = MoeProblem(T, H, I, E, k, shared_I)
    r = MoeRouteParams(E, k, method, n_group, topk_group, rsf)
    return ctypes.byref(p), ctypes.byref(r), _lib.moe_layer_few_workspace_bytes(ctypes.byref(p))


def _few_weights(w, name: str, shape: tuple, format: int, dtype) -> MoeWeights:
    """A weight of moe_layer_few: an Fp4 of `format`, or a tensor of `dtype`, of just this shape."""
    if format == MOE_WEIGHTS_16BIT:
        if isinstance(w, Fp4):
            raise ValueError(f"{name} must be a tensor of {dtype} as the other weights are")
        return MoeWeights(_shaped(w, name, shape, dtype).data_ptr(), None, None)
    if not isinstance(w, Fp4) or w.format != format or w.shape != shape:
        raise ValueError(f"{name} must be {shape} in 4 bits of the same format as w13, got "
                         f"{tuple(getattr(w, 'shape', ()))}")
    return MoeWeights(w.codes.data_ptr(), w.scales.data_ptr(), _ptr(w.g))


def moe_layer_few(x, wg, w13, w2, method: int, top_k: int, bias: Optional[torch.Tensor] = None,
                  n_group: int = 1, topk_group: int = 1, routed_scaling_factor: float = 1.0,
                  w13_s=None, w2_s=None, y=None, ids=None, scales=None,
                  scratch: Optional[Scratch] = None, stream=None):
    """The whole layer for up to MOE_FEW_TOKENS tokens, in two kernels: gate, routing, the chosen experts
    (and the shared one) and the weighted sum. x [T, H] and wg [E, H] in bfloat16 or float16; w13
    [E, 2I, H] and w2 [E, H, I] (w13_s [2Is, H], w2_s [H, Is]) of the same type, or all Fp4 of one
    format. A wg with E + 1 rows carries the shared expert's gate in its last row. Routing parameters as
    moe_route's (and groups of any two or more experts). Returns (y [T, H], ids int32 [T, k], scales fp32 [T, k]). moe_read_timeouts says whether
    a wait ran out."""
    code = _typed(x, "x", 2)
    if code == MOE_DTYPE_F32:
        raise ValueError("x must be bfloat16 or float16, got torch.float32")
    T, H = x.shape
    format = w13.format if isinstance(w13, Fp4) else MOE_WEIGHTS_16BIT
    if len(w13.shape) != 3:
        raise ValueError(f"w13 must be [E, 2I, {H}], got {tuple(w13.shape)}")
    E, I = w13.shape[0], w13.shape[1] // 2
    if wg.dim() != 2 or wg.shape[0] - E not in (0, 1):
        raise ValueError(f"wg must be [{E} or {E + 1}, {H}], got {tuple(wg.shape)}")
    gate = wg.shape[0] - E
    _shaped(wg, "wg", (E + gate, H), x.dtype)
    a = _few_weights(w13, "w13", (E, 2 * I, H), format, x.dtype)
    b = _few_weights(w2, "w2", (E, H, I), format, x.dtype)
    a_s = b_s = None
    shared_I = 0
    if w13_s is not None or w2_s is not None:
        if w13_s is None or w2_s is None:
            raise ValueError("w13_s and w2_s belong together")
        shared_I = w13_s.shape[0] // 2
        a_s = ctypes.byref(_few_weights(w13_s, "w13_s", (2 * shared_I, H), format, x.dtype))
        b_s = ctypes.byref(_few_weights(w2_s, "w2_s", (H, shared_I), format, x.dtype))
    if bias is not None:
        _shaped(bias, "bias", (E,), torch.float32)
    y = _like(x, y, "y", (T, H), stream)
    ids = (_new((T, top_k), torch.int32, x.device, stream) if ids is None
           else _shaped(ids, "ids", (T, top_k), torch.int32))
    scales = (_new((T, top_k), torch.float32, x.device, stream) if scales is None
              else _shaped(scales, "scales", (T, top_k), torch.float32))
    p, r, n = _few_plan(T, H, I, E, top_k, shared_I, method, n_group, topk_group, routed_scaling_factor)
    if scratch is None:
        buf = _new(n, torch.uint8, x.device, stream, result=False)
    else:
        buf, n = scratch.buf, scratch.nbytes
    st = _lib.moe_layer_few(p, r, x.data_ptr(), wg.data_ptr(), gate, _ptr(bias), ctypes.byref(a),
                            ctypes.byref(b), a_s, b_s, format, code, ids.data_ptr(), scales.data_ptr(),
                            y.data_ptr(), buf.data_ptr(), n, _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_layer_few")
    return y, ids, scales


__all__ = [n for n in dir() if n.startswith(("moe_", "MOE_", "Moe"))] + [
    "make_problem", "alloc_workspace", "Workspace", "load_library", "EXPORTED", "LIB_PATH",
    "Checkpoint", "Scratch", "Fp4", "alloc_dispatch_scratch", "alloc_few_scratch", "alloc_experts_scratch"]
