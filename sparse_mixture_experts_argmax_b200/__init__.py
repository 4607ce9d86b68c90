"""Python binding of libswitchlayer.so, the sm_100a Switch-layer forward pass.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory (tensors) and the current stream.
There is no fallback: if the shared library is missing or cannot be loaded,
every call raises.

The C entry points are exposed under their C names (``switch_layer_forward``,
``switch_layer_capacity`` ...); ``forward`` is a convenience wrapper that
allocates the outputs and the workspace with torch and calls
``switch_layer_forward``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SWL_LIBRARY=checked loads the range-checked build (see build.py)
LIB_PATH = os.path.join(_HERE, "libswitchlayer_checked.so"
                        if os.environ.get("SWL_LIBRARY", "") == "checked"
                        else "libswitchlayer.so")

SWL_F32, SWL_BF16 = 0, 1
SWL_WS_HOST_IO = 1
SWL_WS_TOP2 = 2
SWL_WS_NTLB = 4
SWL_NUM_STAGES = 5
STATUS = {0: "SWL_OK", 1: "SWL_ERR_INVALID_ARG", 2: "SWL_ERR_UNSUPPORTED",
          3: "SWL_ERR_WORKSPACE", 4: "SWL_ERR_CUDA", 5: "SWL_ERR_DEVICE"}

# Every symbol declared in include/switch_layer.h.
EXPORTS = ("switch_layer_capacity", "switch_layer_workspace_size", "switch_layer_forward",
           "switch_layer_forward_timed", "switch_layer_forward_host_io",
           "switch_layer_device_status", "switch_layer_status_string",
           "switch_layer_stage_name", "switch_layer_launch_count",
           "switch_layer_forward_noalloc", "switch_layer_set_router_mode",
           "switch_layer_router_mode", "switch_layer_describe_plan",
           "switch_layer_noalloc_status", "switch_layer_shard_record_bytes",
           "switch_layer_forward_shard_begin", "switch_layer_forward_shard_end",
           "switch_layer_set_wait_limit_ns", "switch_layer_set_stall_test",
           "switch_layer_forward_top2", "switch_layer_forward_ntlb", "switch_layer_ep_max_recv_rows",
           "switch_layer_ep_workspace_size", "switch_layer_ep_counts",
           "switch_layer_ep_dispatch", "switch_layer_ep_experts", "switch_layer_ep_combine",
           "switch_layer_variant_workspace_size", "switch_layer_forward_variant",
           "switch_layer_backward_workspace_size", "switch_layer_backward",
           "switch_layer_adamw_step", "switch_layer_norm_residual",
           "switch_layer_norm_residual_backward_workspace_size",
           "switch_layer_norm_residual_backward", "switch_layer_grouped_workspace_size",
           "switch_layer_grouped_matmul", "switch_layer_grouped_matmul_backward")
SWL_ACT_RELU, SWL_ACT_GEGLU = 0, 1


class Variant(ctypes.Structure):
    """struct swl_variant of include/switch_layer.h."""
    _fields_ = [("top_k", ctypes.c_int), ("normalize", ctypes.c_int),
                ("activation", ctypes.c_int), ("router_noise", ctypes.c_void_p)]


class AdamwTensor(ctypes.Structure):
    """struct swl_adamw_tensor of include/switch_layer.h."""
    _fields_ = [("n", ctypes.c_int64), ("dtype", ctypes.c_int), ("state_bits", ctypes.c_int),
                ("weight_decay", ctypes.c_double), ("param", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("master", ctypes.c_void_p)]


class Adamw(ctypes.Structure):
    """struct swl_adamw of include/switch_layer.h."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("seed", ctypes.c_uint32)]


class Norm(ctypes.Structure):
    """struct swl_norm of include/switch_layer.h."""
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("w_pre", ctypes.c_void_p),
                ("b_pre", ctypes.c_void_p), ("w_post", ctypes.c_void_p),
                ("b_post", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class NormGrads(ctypes.Structure):
    """struct swl_norm_grads of include/switch_layer.h."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "dy", "dgate", "dw_pre", "db_pre",
                                               "dw_post", "db_post", "dscale")]


SWL_NORM_RMS, SWL_NORM_LAYER = 0, 1
SWL_ADAMW_BLOCK = 256
SWL_ROUTER_TENSOR = 0
SWL_ROUTER_FFMA = 1
SWL_NOALLOC_MAX_BYTES = 64 << 20


class SwitchLayerError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s (%s)%s" % (STATUS.get(status, "status %d" % status),
                                        _status_string(status),
                                        (": " + what) if what else ""))


_lib: Optional[ctypes.CDLL] = None

_i64, _i32, _dbl, _vp, _sz = (ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p,
                              ctypes.c_size_t)
_FWD_ARGS = [_i64, _i64, _i64, _i64, _i32,            # T, d, d_ff, N, dtype
             _vp, _vp, _vp, _vp, _vp, _vp, _dbl,       # x, W_r, W1, b1, W2, b2, cf
             _vp, _vp, _vp, _vp, _vp,                  # out, expert_idx, gate, pos, aux
             _vp, _vp, _sz, _vp]                       # b_r, workspace, bytes, stream


def lib() -> ctypes.CDLL:
    """Load libswitchlayer.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("%s is missing: build it with "
                           "`python -m sparse_mixture_experts_argmax_b200.build`"
                           % os.path.basename(LIB_PATH))
    L = ctypes.CDLL(LIB_PATH)
    L.switch_layer_capacity.restype = _i64
    L.switch_layer_capacity.argtypes = [_i64, _i64, _dbl]
    L.switch_layer_workspace_size.restype = _i32
    L.switch_layer_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i32, _dbl, _i32,
                                              ctypes.POINTER(_sz)]
    L.switch_layer_forward.restype = _i32
    L.switch_layer_forward.argtypes = _FWD_ARGS
    L.switch_layer_forward_timed.restype = _i32
    L.switch_layer_forward_timed.argtypes = _FWD_ARGS + [ctypes.POINTER(_vp)]
    L.switch_layer_forward_host_io.restype = _i32
    L.switch_layer_forward_host_io.argtypes = _FWD_ARGS
    L.switch_layer_device_status.restype = _i32
    L.switch_layer_device_status.argtypes = [_vp, _vp]
    L.switch_layer_status_string.restype = ctypes.c_char_p
    L.switch_layer_status_string.argtypes = [_i32]
    L.switch_layer_stage_name.restype = ctypes.c_char_p
    L.switch_layer_stage_name.argtypes = [_i32]
    L.switch_layer_launch_count.restype = ctypes.c_uint64
    L.switch_layer_launch_count.argtypes = []
    L.switch_layer_set_router_mode.restype = ctypes.c_int
    L.switch_layer_set_router_mode.argtypes = [_i32]
    L.switch_layer_router_mode.restype = ctypes.c_int
    L.switch_layer_router_mode.argtypes = []
    L.switch_layer_describe_plan.restype = _i32
    L.switch_layer_describe_plan.argtypes = [_i64, _i64, _i64, _i64, _i32, _dbl, _i32,
                                             ctypes.c_char_p, _sz]
    L.switch_layer_forward_noalloc.restype = _i32
    L.switch_layer_forward_noalloc.argtypes = _FWD_ARGS[:17] + [_vp, _vp]
    L.switch_layer_noalloc_status.restype = _i32
    L.switch_layer_noalloc_status.argtypes = [_vp]
    L.switch_layer_ep_max_recv_rows.restype = _i64
    L.switch_layer_ep_max_recv_rows.argtypes = [_i64, _i32, _i64, _dbl]
    L.switch_layer_ep_workspace_size.restype = _i32
    L.switch_layer_ep_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, _i64, _dbl,
                                                 ctypes.POINTER(_sz)]
    L.switch_layer_ep_counts.restype = _i32
    L.switch_layer_ep_counts.argtypes = [_i64, _i32, _i32, _i64, _dbl, _vp,
                                         ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
    L.switch_layer_ep_dispatch.restype = _i32
    L.switch_layer_ep_dispatch.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _dbl,
                                           _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.switch_layer_ep_experts.restype = _i32
    L.switch_layer_ep_experts.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _dbl,
                                          _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                          _vp]
    L.switch_layer_ep_combine.restype = _i32
    L.switch_layer_ep_combine.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _dbl,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.switch_layer_backward_workspace_size.restype = _i32
    L.switch_layer_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i32, _dbl,
                                                       ctypes.POINTER(_sz)]
    L.switch_layer_backward.restype = _i32
    L.switch_layer_backward.argtypes = ([_i64, _i64, _i64, _i64, _i32] + [_vp] * 7 + [_dbl] +
                                        [_vp] * 5 + [_sz, _vp, ctypes.c_float] + [_vp] * 8 +
                                        [_sz, _vp])
    L.switch_layer_variant_workspace_size.restype = _i32
    L.switch_layer_variant_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i32, _dbl,
                                                      ctypes.POINTER(Variant),
                                                      ctypes.POINTER(_sz)]
    L.switch_layer_forward_variant.restype = _i32
    L.switch_layer_forward_variant.argtypes = (_FWD_ARGS[:18] + [ctypes.POINTER(Variant)] +
                                               _FWD_ARGS[18:])
    L.switch_layer_forward_top2.restype = _i32
    L.switch_layer_forward_top2.argtypes = _FWD_ARGS[:12] + [_i32] + _FWD_ARGS[12:]
    L.switch_layer_forward_ntlb.restype = _i32
    L.switch_layer_forward_ntlb.argtypes = _FWD_ARGS
    L.switch_layer_set_wait_limit_ns.restype = _i32
    L.switch_layer_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.switch_layer_set_stall_test.restype = _i32
    L.switch_layer_set_stall_test.argtypes = [_i32]
    L.switch_layer_shard_record_bytes.restype = _sz
    L.switch_layer_shard_record_bytes.argtypes = [_i64]
    L.switch_layer_forward_shard_begin.restype = _i32
    L.switch_layer_forward_shard_begin.argtypes = [_i64, _i64, _i64, _i64, _i32, _i64,
                                                   _vp, _vp, _vp, _dbl, _vp, _vp, _vp, _vp,
                                                   _vp, _sz, _vp]
    L.switch_layer_forward_shard_end.restype = _i32
    L.switch_layer_forward_shard_end.argtypes = [_i64, _i64, _i64, _i64, _i32, _i64, _i32,
                                                 _i32, _vp, _vp, _vp, _vp, _vp, _vp, _dbl,
                                                 _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.switch_layer_grouped_workspace_size.restype = _i32
    L.switch_layer_grouped_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i32,
                                                      ctypes.POINTER(_sz)]
    L.switch_layer_grouped_matmul.restype = _i32
    L.switch_layer_grouped_matmul.argtypes = ([_i64, _i64, _i64, _i64, _i32] + [_vp] * 6 +
                                              [_sz, _vp])
    L.switch_layer_grouped_matmul_backward.restype = _i32
    L.switch_layer_grouped_matmul_backward.argtypes = ([_i64, _i64, _i64, _i64, _i32] +
                                                       [_vp] * 8 + [_sz, _vp])
    L.switch_layer_norm_residual.restype = _i32
    L.switch_layer_norm_residual.argtypes = [_i64, _i64, _i32, _vp, _vp, _vp,
                                             ctypes.POINTER(Norm), _vp, _vp, _vp]
    L.switch_layer_norm_residual_backward_workspace_size.restype = _i32
    L.switch_layer_norm_residual_backward_workspace_size.argtypes = [_i64, _i64, _i32,
                                                                     ctypes.POINTER(_sz)]
    L.switch_layer_norm_residual_backward.restype = _i32
    L.switch_layer_norm_residual_backward.argtypes = [_i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp,
                                                      ctypes.POINTER(Norm),
                                                      ctypes.POINTER(NormGrads), _vp, _sz, _vp]
    L.switch_layer_adamw_step.restype = _i32
    L.switch_layer_adamw_step.argtypes = [ctypes.POINTER(AdamwTensor), _i32,
                                          ctypes.POINTER(Adamw), _vp, _vp, _vp, _vp]
    _lib = L
    return L


def _status_string(status: int) -> str:
    try:
        return lib().switch_layer_status_string(status).decode()
    except Exception:  # pragma: no cover - only while reporting another failure
        return "?"


def _check(status: int, what: str = "") -> None:
    if status != 0:
        raise SwitchLayerError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# torch's own short ways to the current device and its stream's handle make no Stream object;
# they are not public, so under a torch without them the public ones stand in.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream_handle(stream) -> int:
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return SWL_F32
    if dt == torch.bfloat16:
        return SWL_BF16
    raise TypeError("activation dtype must be float32 or bfloat16, got %s" % dt)


# ---------------------------------------------------------------------------
# C entry points, same names
# ---------------------------------------------------------------------------
def switch_layer_capacity(T: int, N: int, capacity_factor: float) -> int:
    return int(lib().switch_layer_capacity(T, N, capacity_factor))


def switch_layer_workspace_size(T, d, d_ff, N, dtype: int, capacity_factor: float,
                                flags: int = 0) -> int:
    n = _sz(0)
    _check(lib().switch_layer_workspace_size(T, d, d_ff, N, dtype, capacity_factor, flags,
                                             ctypes.byref(n)), "workspace_size")
    return int(n.value)


def _shape_of(x, W1, W_r):
    T, d = x.shape
    N, d_ff, d2 = W1.shape
    if d2 != d or tuple(W_r.shape) != (N, d):
        raise ValueError("shape mismatch: x %s, W_r %s, W1 %s" % (tuple(x.shape),
                                                                  tuple(W_r.shape),
                                                                  tuple(W1.shape)))
    return T, d, d_ff, N


def _require(t: torch.Tensor, name: str, dtype=None, device="cuda"):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if device == "cuda" and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device == "cpu" and t.is_cuda:
        raise ValueError("%s must be a host tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def switch_layer_forward(x, W_r, W1, b1, W2, b2, capacity_factor, out, expert_idx, gate,
                         pos_in_expert, aux_loss, b_r=None, workspace=None, stream=None,
                         stage_events: Optional[Sequence] = None) -> None:
    """Enqueue one forward pass (all tensors on the GPU; see include/switch_layer.h)."""
    T, d, d_ff, N = _shape_of(x, W1, W_r)
    act = x.dtype
    for t, n in ((x, "x"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (b2, "b2"), (out, "out")):
        _require(t, n, act)
    _require(W_r, "W_r", torch.float32)
    if b_r is not None:
        _require(b_r, "b_r", torch.float32)
    _require(expert_idx, "expert_idx", torch.int32)
    _require(pos_in_expert, "pos_in_expert", torch.int32)
    _require(gate, "gate", torch.float32)
    _require(aux_loss, "aux_loss", torch.float32)
    _require(workspace, "workspace", torch.uint8)
    args = (T, d, d_ff, N, dtype_code(act), _ptr(x), _ptr(W_r), _ptr(W1), _ptr(b1), _ptr(W2),
            _ptr(b2), float(capacity_factor), _ptr(out), _ptr(expert_idx), _ptr(gate),
            _ptr(pos_in_expert), _ptr(aux_loss), _ptr(b_r), _ptr(workspace),
            workspace.numel(), _stream_handle(stream))
    if stage_events is None:
        _check(lib().switch_layer_forward(*args), "forward")
    else:
        if len(stage_events) != SWL_NUM_STAGES + 1:
            raise ValueError("need %d stage events" % (SWL_NUM_STAGES + 1))
        for e in stage_events:          # torch creates the CUDA event on first record
            if not e.cuda_event:
                e.record()
        evs = (_vp * (SWL_NUM_STAGES + 1))(*[ctypes.c_void_p(int(e.cuda_event))
                                             for e in stage_events])
        _check(lib().switch_layer_forward_timed(*args, evs), "forward_timed")


def switch_layer_forward_top2(x, W_r, W1, b1, W2, b2, capacity_factor, normalize, out,
                              expert_idx, gate, pos_in_expert, aux_loss, b_r=None,
                              workspace=None, stream=None) -> None:
    """Enqueue one forward pass of the top-2 variant (expert_idx, gate,
    pos_in_expert are [T, 2]; workspace sized with SWL_WS_TOP2)."""
    T, d, d_ff, N = _shape_of(x, W1, W_r)
    act = x.dtype
    for t, n in ((x, "x"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (b2, "b2"), (out, "out")):
        _require(t, n, act)
    _require(W_r, "W_r", torch.float32)
    if b_r is not None:
        _require(b_r, "b_r", torch.float32)
    for t, n, dt in ((expert_idx, "expert_idx", torch.int32), (gate, "gate", torch.float32),
                     (pos_in_expert, "pos_in_expert", torch.int32)):
        _require(t, n, dt)
        if t.numel() != 2 * T:
            raise ValueError("%s must hold [T, 2] values" % n)
    _require(aux_loss, "aux_loss", torch.float32)
    _require(workspace, "workspace", torch.uint8)
    _check(lib().switch_layer_forward_top2(
        T, d, d_ff, N, dtype_code(act), _ptr(x), _ptr(W_r), _ptr(W1), _ptr(b1), _ptr(W2),
        _ptr(b2), float(capacity_factor), 1 if normalize else 0, _ptr(out), _ptr(expert_idx),
        _ptr(gate), _ptr(pos_in_expert), _ptr(aux_loss), _ptr(b_r), _ptr(workspace),
        workspace.numel(), _stream_handle(stream)), "forward_top2")


def switch_layer_forward_ntlb(x, W_r, W1, b1, W2, b2, capacity_factor, out, expert_idx, gate,
                              pos_in_expert, aux_loss, b_r=None, workspace=None,
                              stream=None) -> None:
    """Enqueue one forward pass of the No-Token-Left-Behind variant (expert_idx,
    gate, pos_in_expert are [T, 2]; workspace sized with SWL_WS_NTLB)."""
    T, d, d_ff, N = _shape_of(x, W1, W_r)
    act = x.dtype
    for t, n in ((x, "x"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (b2, "b2"), (out, "out")):
        _require(t, n, act)
    _require(W_r, "W_r", torch.float32)
    if b_r is not None:
        _require(b_r, "b_r", torch.float32)
    for t, n, dt in ((expert_idx, "expert_idx", torch.int32), (gate, "gate", torch.float32),
                     (pos_in_expert, "pos_in_expert", torch.int32)):
        _require(t, n, dt)
        if t.numel() != 2 * T:
            raise ValueError("%s must hold [T, 2] values" % n)
    _require(aux_loss, "aux_loss", torch.float32)
    _require(workspace, "workspace", torch.uint8)
    _check(lib().switch_layer_forward_ntlb(
        T, d, d_ff, N, dtype_code(act), _ptr(x), _ptr(W_r), _ptr(W1), _ptr(b1), _ptr(W2),
        _ptr(b2), float(capacity_factor), _ptr(out), _ptr(expert_idx), _ptr(gate),
        _ptr(pos_in_expert), _ptr(aux_loss), _ptr(b_r), _ptr(workspace), workspace.numel(),
        _stream_handle(stream)), "forward_ntlb")


def switch_layer_forward_host_io(x_host, W_r, W1, b1, W2, b2, capacity_factor, out_host,
                                 expert_idx_host, gate_host, pos_host, aux_host, b_r=None,
                                 workspace=None, stream=None) -> None:
    """Enqueue H2D(x) -> forward -> D2H(outputs); host tensors should be pinned."""
    T, d, d_ff, N = _shape_of(x_host, W1, W_r)
    act = x_host.dtype
    _require(x_host, "x_host", act, device="cpu")
    _require(out_host, "out_host", act, device="cpu")
    for t, n in ((W1, "W1"), (b1, "b1"), (W2, "W2"), (b2, "b2")):
        _require(t, n, act)
    _require(W_r, "W_r", torch.float32)
    _require(expert_idx_host, "expert_idx_host", torch.int32, device="cpu")
    _require(pos_host, "pos_host", torch.int32, device="cpu")
    _require(gate_host, "gate_host", torch.float32, device="cpu")
    _require(aux_host, "aux_host", torch.float32, device="cpu")
    _require(workspace, "workspace", torch.uint8)
    _check(lib().switch_layer_forward_host_io(
        T, d, d_ff, N, dtype_code(act), _ptr(x_host), _ptr(W_r), _ptr(W1), _ptr(b1), _ptr(W2),
        _ptr(b2), float(capacity_factor), _ptr(out_host), _ptr(expert_idx_host),
        _ptr(gate_host), _ptr(pos_host), _ptr(aux_host), _ptr(b_r), _ptr(workspace),
        workspace.numel(), _stream_handle(stream)), "forward_host_io")


def switch_layer_device_status(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().switch_layer_device_status(_ptr(workspace), _stream_handle(stream)))


def switch_layer_status_string(status: int) -> str:
    return _status_string(status)


def switch_layer_stage_name(k: int) -> Optional[str]:
    r = lib().switch_layer_stage_name(k)
    return None if r is None else r.decode()


def switch_layer_launch_count() -> int:
    return int(lib().switch_layer_launch_count())


def switch_layer_set_router_mode(mode: int) -> None:
    """SWL_ROUTER_TENSOR (default) or SWL_ROUTER_FFMA for bf16 layers (process-wide)."""
    _check(lib().switch_layer_set_router_mode(int(mode)), "switch_layer_set_router_mode")


def switch_layer_router_mode() -> int:
    return int(lib().switch_layer_router_mode())


def switch_layer_describe_plan(T, d, d_ff, N, dtype: int, capacity_factor: float,
                               num_sms: int = 148) -> dict:
    """The kernels a forward call of this shape would launch (host-only), as a dict
    of the C entry point's key=value pairs (integers converted)."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().switch_layer_describe_plan(T, d, d_ff, N, dtype, capacity_factor, num_sms,
                                            buf, len(buf)), "describe_plan")
    out = {}
    for kv in buf.value.decode().split(","):
        k, v = kv.split("=", 1)
        out[k] = int(v) if v.lstrip("-").isdigit() else v
    return out


def switch_layer_set_wait_limit_ns(ns: int) -> None:
    """Failure-path test hook: bound of every wait inside the kernels (0: 2 s)."""
    _check(lib().switch_layer_set_wait_limit_ns(int(ns)), "set_wait_limit_ns")


def switch_layer_set_stall_test(on: bool) -> None:
    """Failure-path test hook: make the expert FFN's first GEMM2 wait run out."""
    _check(lib().switch_layer_set_stall_test(1 if on else 0), "set_stall_test")


def switch_layer_ep_max_recv_rows(N, world, T_total, capacity_factor) -> int:
    return int(lib().switch_layer_ep_max_recv_rows(N, world, T_total, capacity_factor))


def switch_layer_ep_workspace_size(T, d, d_ff, N, dtype, world, T_total, capacity_factor) -> int:
    n = _sz(0)
    _check(lib().switch_layer_ep_workspace_size(T, d, d_ff, N, dtype, world, T_total,
                                                capacity_factor, ctypes.byref(n)),
           "ep_workspace_size")
    return int(n.value)


def switch_layer_ep_counts(N, world, rank, T_total, capacity_factor, gathered_host):
    """(send rows per peer, receive rows per peer) from a host copy of the records."""
    _require(gathered_host, "gathered_host", torch.uint8, device="cpu")
    send = (_i64 * world)()
    recv = (_i64 * world)()
    _check(lib().switch_layer_ep_counts(N, world, rank, int(T_total), float(capacity_factor),
                                        _ptr(gathered_host), send, recv), "ep_counts")
    return [int(v) for v in send], [int(v) for v in recv]


def switch_layer_ep_dispatch(x, d_ff, N, world, rank, T_total, capacity_factor, gathered,
                             expert_idx, pos_in_expert, aux_loss, send_rows, workspace,
                             stream=None) -> None:
    T, d = x.shape
    _check(lib().switch_layer_ep_dispatch(
        T, d, d_ff, N, dtype_code(x.dtype), world, rank, int(T_total), float(capacity_factor),
        _ptr(gathered), _ptr(x), _ptr(expert_idx), _ptr(pos_in_expert), _ptr(aux_loss),
        _ptr(send_rows), _ptr(workspace), workspace.numel(), _stream_handle(stream)),
        "ep_dispatch")


def switch_layer_ep_experts(T, d, d_ff, N, act_dtype, world, rank, T_total, capacity_factor,
                            gathered, recv_rows, W1_local, b1_local, W2_local, b2_local, ret_rows,
                            workspace, stream=None) -> None:
    for t, n in ((W1_local, "W1_local"), (b1_local, "b1_local"), (W2_local, "W2_local"),
                 (b2_local, "b2_local")):
        _require(t, n, act_dtype)
    _check(lib().switch_layer_ep_experts(
        T, d, d_ff, N, dtype_code(act_dtype), world, rank, int(T_total), float(capacity_factor),
        _ptr(gathered), _ptr(recv_rows), recv_rows.shape[0], _ptr(W1_local), _ptr(b1_local),
        _ptr(W2_local), _ptr(b2_local), _ptr(ret_rows), _ptr(workspace), workspace.numel(),
        _stream_handle(stream)), "ep_experts")


def switch_layer_ep_combine(T, d, d_ff, N, act_dtype, world, rank, T_total, capacity_factor,
                            back_rows, expert_idx, gate, pos_in_expert, out, workspace,
                            stream=None) -> None:
    _check(lib().switch_layer_ep_combine(
        T, d, d_ff, N, dtype_code(act_dtype), world, rank, int(T_total), float(capacity_factor),
        _ptr(back_rows), _ptr(expert_idx), _ptr(gate), _ptr(pos_in_expert), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream_handle(stream)), "ep_combine")


def switch_layer_shard_record_bytes(N: int) -> int:
    return int(lib().switch_layer_shard_record_bytes(N))


def switch_layer_forward_shard_begin(x, W_r, capacity_factor, T_total, expert_idx, gate,
                                     pos_in_expert, record, d_ff, b_r=None, workspace=None,
                                     stream=None) -> None:
    """Step 1 of a forward over one rank's token range of a global batch."""
    T, d = x.shape
    N = W_r.shape[0]
    _require(x, "x")
    _require(W_r, "W_r", torch.float32)
    if b_r is not None:
        _require(b_r, "b_r", torch.float32)
    _require(record, "record", torch.uint8)
    _require(workspace, "workspace", torch.uint8)
    if record.numel() != switch_layer_shard_record_bytes(N):
        raise ValueError("record must hold %d bytes" % switch_layer_shard_record_bytes(N))
    _check(lib().switch_layer_forward_shard_begin(
        T, d, d_ff, N, dtype_code(x.dtype), int(T_total), _ptr(x), _ptr(W_r), _ptr(b_r),
        float(capacity_factor), _ptr(expert_idx), _ptr(gate), _ptr(pos_in_expert),
        _ptr(record), _ptr(workspace), workspace.numel(), _stream_handle(stream)),
        "forward_shard_begin")


def switch_layer_forward_shard_end(x, W1, b1, W2, b2, capacity_factor, T_total, rank, world,
                                   gathered, out, expert_idx, gate, pos_in_expert, aux_loss,
                                   workspace=None, stream=None) -> None:
    """Step 3 of a forward over one rank's token range of a global batch."""
    T, d = x.shape
    N, d_ff, _ = W1.shape
    act = x.dtype
    for t, n in ((x, "x"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (b2, "b2"), (out, "out")):
        _require(t, n, act)
    _require(gathered, "gathered", torch.uint8)
    _require(workspace, "workspace", torch.uint8)
    if gathered.numel() != world * switch_layer_shard_record_bytes(N):
        raise ValueError("gathered must hold world * record bytes")
    _check(lib().switch_layer_forward_shard_end(
        T, d, d_ff, N, dtype_code(act), int(T_total), int(rank), int(world), _ptr(gathered),
        _ptr(x), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), float(capacity_factor), _ptr(out),
        _ptr(expert_idx), _ptr(gate), _ptr(pos_in_expert), _ptr(aux_loss), _ptr(workspace),
        workspace.numel(), _stream_handle(stream)), "forward_shard_end")


# ---------------------------------------------------------------------------
# convenience: allocate outputs + workspace with torch and run
# ---------------------------------------------------------------------------
def alloc_workspace(T, d, d_ff, N, act_dtype: torch.dtype, capacity_factor: float,
                    host_io: bool = False, device="cuda", top2: bool = False,
                    ntlb: bool = False) -> torch.Tensor:
    n = switch_layer_workspace_size(T, d, d_ff, N, dtype_code(act_dtype), capacity_factor,
                                    (SWL_WS_HOST_IO if host_io else 0) |
                                    (SWL_WS_TOP2 if top2 else 0) |
                                    (SWL_WS_NTLB if ntlb else 0))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def alloc_outputs(T, d, act_dtype, device="cuda") -> dict:
    return {
        "out": torch.empty((T, d), dtype=act_dtype, device=device),
        "expert_idx": torch.empty(T, dtype=torch.int32, device=device),
        "gate": torch.empty(T, dtype=torch.float32, device=device),
        "pos_in_expert": torch.empty(T, dtype=torch.int32, device=device),
        "aux_loss": torch.empty(1, dtype=torch.float32, device=device),
    }


def forward(inputs: dict, capacity_factor: float, workspace: Optional[torch.Tensor] = None,
            outputs: Optional[dict] = None, stream=None, check: bool = True) -> dict:
    """Run the layer on ``inputs`` (keys x, W_r, b_r, W1, b1, W2, b2; CUDA tensors)."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N, d_ff, _ = W1.shape
    if workspace is None:
        workspace = alloc_workspace(T, d, d_ff, N, x.dtype, capacity_factor, device=x.device)
    if outputs is None:
        outputs = alloc_outputs(T, d, x.dtype, device=x.device)
    switch_layer_forward(x, inputs["W_r"], W1, inputs["b1"], inputs["W2"], inputs["b2"],
                         capacity_factor, outputs["out"], outputs["expert_idx"], outputs["gate"],
                         outputs["pos_in_expert"], outputs["aux_loss"], b_r=inputs.get("b_r"),
                         workspace=workspace, stream=stream)
    if check:
        _check(switch_layer_device_status(workspace, stream), "device status")
    return outputs


def forward_shard(inputs: dict, capacity_factor: float, T_total: int, rank: int, world: int,
                  exchange, workspace: Optional[torch.Tensor] = None,
                  outputs: Optional[dict] = None, stream=None, check: bool = True) -> dict:
    """One rank's part of a forward over a global batch: ``inputs`` holds this
    rank's token range (x) and the full weights; ``exchange(record)`` returns
    the records of all ranks in rank order (an all-gather)."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N, d_ff, _ = W1.shape
    if workspace is None:
        workspace = alloc_workspace(max(T, 1), d, d_ff, N, x.dtype, capacity_factor,
                                    device=W1.device)
    if outputs is None:
        outputs = alloc_outputs(T, d, x.dtype, device=W1.device)
    record = torch.empty(switch_layer_shard_record_bytes(N), dtype=torch.uint8,
                         device=W1.device)
    switch_layer_forward_shard_begin(x, inputs["W_r"], capacity_factor, T_total,
                                     outputs["expert_idx"], outputs["gate"],
                                     outputs["pos_in_expert"], record, d_ff,
                                     b_r=inputs.get("b_r"), workspace=workspace, stream=stream)
    gathered = exchange(record)
    switch_layer_forward_shard_end(x, W1, inputs["b1"], inputs["W2"], inputs["b2"],
                                   capacity_factor, T_total, rank, world, gathered,
                                   outputs["out"], outputs["expert_idx"], outputs["gate"],
                                   outputs["pos_in_expert"], outputs["aux_loss"],
                                   workspace=workspace, stream=stream)
    if check:
        _check(switch_layer_device_status(workspace, stream), "device status")
    return outputs


def forward_top2(inputs: dict, capacity_factor: float, normalize: bool = True,
                 workspace: Optional[torch.Tensor] = None, stream=None,
                 check: bool = True) -> dict:
    """Run the top-2 variant on ``inputs`` (CUDA tensors); [T, 2] routing outputs."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N, d_ff, _ = W1.shape
    if workspace is None:
        workspace = alloc_workspace(T, d, d_ff, N, x.dtype, capacity_factor, device=x.device,
                                    top2=True)
    o = {"out": torch.empty((T, d), dtype=x.dtype, device=x.device),
         "expert_idx": torch.empty((T, 2), dtype=torch.int32, device=x.device),
         "gate": torch.empty((T, 2), dtype=torch.float32, device=x.device),
         "pos_in_expert": torch.empty((T, 2), dtype=torch.int32, device=x.device),
         "aux_loss": torch.empty(1, dtype=torch.float32, device=x.device)}
    switch_layer_forward_top2(x, inputs["W_r"], W1, inputs["b1"], inputs["W2"], inputs["b2"],
                              capacity_factor, normalize, o["out"], o["expert_idx"], o["gate"],
                              o["pos_in_expert"], o["aux_loss"], b_r=inputs.get("b_r"),
                              workspace=workspace, stream=stream)
    if check:
        _check(switch_layer_device_status(workspace, stream), "device status")
    return o


def forward_ntlb(inputs: dict, capacity_factor: float,
                 workspace: Optional[torch.Tensor] = None, stream=None,
                 check: bool = True) -> dict:
    """Run the No-Token-Left-Behind variant on ``inputs`` (CUDA tensors); [T, 2]
    routing outputs."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N, d_ff, _ = W1.shape
    if workspace is None:
        workspace = alloc_workspace(T, d, d_ff, N, x.dtype, capacity_factor, device=x.device,
                                    ntlb=True)
    o = {"out": torch.empty((T, d), dtype=x.dtype, device=x.device),
         "expert_idx": torch.empty((T, 2), dtype=torch.int32, device=x.device),
         "gate": torch.empty((T, 2), dtype=torch.float32, device=x.device),
         "pos_in_expert": torch.empty((T, 2), dtype=torch.int32, device=x.device),
         "aux_loss": torch.empty(1, dtype=torch.float32, device=x.device)}
    switch_layer_forward_ntlb(x, inputs["W_r"], W1, inputs["b1"], inputs["W2"], inputs["b2"],
                              capacity_factor, o["out"], o["expert_idx"], o["gate"],
                              o["pos_in_expert"], o["aux_loss"], b_r=inputs.get("b_r"),
                              workspace=workspace, stream=stream)
    if check:
        _check(switch_layer_device_status(workspace, stream), "device status")
    return o


def forward_ep(inputs: dict, capacity_factor: float, N: int, T_total: int, rank: int,
               world: int, allgather, alltoall, stream=None, check: bool = True) -> dict:
    """One rank's part of an expert-parallel forward pass.  ``inputs``: this
    rank's token range x, the full W_r (and b_r), and the weights of this
    rank's experts W1/b1/W2/b2 ([N / world, ...]).  ``allgather(record)``
    returns every rank's record in rank order (device); ``alltoall(rows,
    send_counts, recv_counts)`` exchanges row blocks between ranks (rows [sum
    send, d] -> [sum recv, d])."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    d_ff = W1.shape[1]
    dev = W1.device
    ws = torch.empty(switch_layer_ep_workspace_size(T, d, d_ff, N, dtype_code(x.dtype), world,
                                                    T_total, capacity_factor),
                     dtype=torch.uint8, device=dev)
    o = alloc_outputs(T, d, x.dtype, device=dev)
    record = torch.empty(switch_layer_shard_record_bytes(N), dtype=torch.uint8, device=dev)
    switch_layer_forward_shard_begin(x, inputs["W_r"], capacity_factor, T_total, o["expert_idx"],
                                     o["gate"], o["pos_in_expert"], record, d_ff,
                                     b_r=inputs.get("b_r"), workspace=ws, stream=stream)
    gathered = allgather(record)
    send_c, recv_c = switch_layer_ep_counts(N, world, rank, T_total, capacity_factor,
                                            gathered.cpu())
    send = torch.empty((sum(send_c), d), dtype=x.dtype, device=dev)
    switch_layer_ep_dispatch(x, d_ff, N, world, rank, T_total, capacity_factor, gathered,
                             o["expert_idx"], o["pos_in_expert"], o["aux_loss"], send, ws,
                             stream)
    recv = alltoall(send, send_c, recv_c)
    ret = torch.empty_like(recv)
    switch_layer_ep_experts(T, d, d_ff, N, x.dtype, world, rank, T_total, capacity_factor,
                            gathered, recv, W1, inputs["b1"], inputs["W2"], inputs["b2"], ret, ws,
                            stream)
    back = alltoall(ret, recv_c, send_c)
    switch_layer_ep_combine(T, d, d_ff, N, x.dtype, world, rank, T_total, capacity_factor, back,
                            o["expert_idx"], o["gate"], o["pos_in_expert"], o["out"], ws, stream)
    if check:
        _check(switch_layer_device_status(ws, stream), "device status")
    return o


def make_variant(top_k: int = 1, normalize: bool = True, activation: str = "relu",
                 router_noise: Optional[torch.Tensor] = None) -> Variant:
    if router_noise is not None:
        _require(router_noise, "router_noise", torch.float32)
    return Variant(int(top_k), 1 if normalize else 0,
                   {"relu": SWL_ACT_RELU, "geglu": SWL_ACT_GEGLU}[activation],
                   None if router_noise is None else router_noise.data_ptr())


def switch_layer_variant_workspace_size(T, d, d_ff, N, dtype, capacity_factor,
                                        variant: Variant) -> int:
    n = _sz(0)
    _check(lib().switch_layer_variant_workspace_size(T, d, d_ff, N, dtype, capacity_factor,
                                                     ctypes.byref(variant), ctypes.byref(n)),
           "variant_workspace_size")
    return int(n.value)


def forward_variant(inputs: dict, capacity_factor: float, top_k: int = 1, normalize: bool = True,
                    activation: str = "relu", router_noise: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None,
                    check: bool = True) -> dict:
    """Run a layer variant (top-2 routing, GEGLU experts, router input jitter)."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N = W1.shape[0]
    d_ff = W1.shape[1] // (2 if activation == "geglu" else 1)
    v = make_variant(top_k, normalize, activation, router_noise)
    if workspace is None:
        workspace = torch.empty(max(256, switch_layer_variant_workspace_size(
            T, d, d_ff, N, dtype_code(x.dtype), capacity_factor, v)), dtype=torch.uint8,
            device=x.device)
    shape_k = (T, top_k) if top_k == 2 else (T,)
    o = {"out": torch.empty((T, d), dtype=x.dtype, device=x.device),
         "expert_idx": torch.empty(shape_k, dtype=torch.int32, device=x.device),
         "gate": torch.empty(shape_k, dtype=torch.float32, device=x.device),
         "pos_in_expert": torch.empty(shape_k, dtype=torch.int32, device=x.device),
         "aux_loss": torch.empty(1, dtype=torch.float32, device=x.device)}
    for t, n in ((x, "x"), (W1, "W1"), (inputs["b1"], "b1"), (inputs["W2"], "W2"),
                 (inputs["b2"], "b2")):
        _require(t, n, x.dtype)
    _require(inputs["W_r"], "W_r", torch.float32)
    _check(lib().switch_layer_forward_variant(
        T, d, d_ff, N, dtype_code(x.dtype), _ptr(x), _ptr(inputs["W_r"]), _ptr(W1),
        _ptr(inputs["b1"]), _ptr(inputs["W2"]), _ptr(inputs["b2"]), float(capacity_factor),
        _ptr(o["out"]), _ptr(o["expert_idx"]), _ptr(o["gate"]), _ptr(o["pos_in_expert"]),
        _ptr(o["aux_loss"]), _ptr(inputs.get("b_r")), ctypes.byref(v), _ptr(workspace),
        workspace.numel(), _stream_handle(stream)), "forward_variant")
    if check:
        _check(switch_layer_device_status(workspace, stream), "device status")
    return o


def backward(inputs: dict, capacity_factor: float, fwd: dict, fwd_workspace: torch.Tensor,
             dout: torch.Tensor, daux: float = 0.0, stream=None, check: bool = True) -> dict:
    """Gradients of sum(dout * out) + daux * aux for a forward call made with
    ``fwd_workspace`` (its outputs ``fwd``): dx, dW_r, db_r, dW1, db1, dW2, db2."""
    x, W1 = inputs["x"], inputs["W1"]
    T, d = x.shape
    N, d_ff, _ = W1.shape
    dev = x.device
    n = _sz(0)
    _check(lib().switch_layer_backward_workspace_size(T, d, d_ff, N, dtype_code(x.dtype),
                                                      float(capacity_factor), ctypes.byref(n)),
           "backward_workspace_size")
    bws = torch.empty(max(256, int(n.value)), dtype=torch.uint8, device=dev)
    g = {"dx": torch.empty_like(x), "dW_r": torch.empty_like(inputs["W_r"]),
         "db_r": torch.empty(N, dtype=torch.float32, device=dev),
         "dW1": torch.empty_like(W1), "db1": torch.empty_like(inputs["b1"]),
         "dW2": torch.empty_like(inputs["W2"]), "db2": torch.empty_like(inputs["b2"])}
    _require(dout, "dout", x.dtype)
    _check(lib().switch_layer_backward(
        T, d, d_ff, N, dtype_code(x.dtype), _ptr(x), _ptr(inputs["W_r"]), _ptr(inputs.get("b_r")),
        _ptr(W1), _ptr(inputs["b1"]), _ptr(inputs["W2"]), _ptr(inputs["b2"]),
        float(capacity_factor), _ptr(fwd["out"]), _ptr(fwd["expert_idx"]), _ptr(fwd["gate"]),
        _ptr(fwd["pos_in_expert"]), _ptr(fwd_workspace), fwd_workspace.numel(), _ptr(dout),
        float(daux), _ptr(g["dx"]), _ptr(g["dW_r"]), _ptr(g["db_r"]), _ptr(g["dW1"]),
        _ptr(g["db1"]), _ptr(g["dW2"]), _ptr(g["db2"]), _ptr(bws), bws.numel(),
        _stream_handle(stream)), "backward")
    if check:
        _check(switch_layer_device_status(fwd_workspace, stream), "device status")
    return g


# ---------------------------------------------------------------------------
# the operators around the layer: shared checks
# ---------------------------------------------------------------------------
def _at(t: Optional[torch.Tensor], name: str, dtype, shape, dev) -> Optional[int]:
    """The address of a contiguous CUDA tensor of this type, shape and device (None: None)."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or
            not t.is_contiguous()):
        _require(t, name, dtype)
    if t.device != dev:
        raise ValueError("%s is on %s: all tensors must be on %s" % (name, t.device, dev))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


_HERE_ALREADY = contextlib.nullcontext()


def _on(dev: torch.device):
    """A context in which ``dev`` is the current device (the library launches there)."""
    if dev.index is None or dev.index == _current_device():
        return _HERE_ALREADY
    return torch.cuda.device(dev)


def _allocating_on(stream, dev: torch.device):
    """A context in which torch allocates for ``stream`` (None: the current one), so that
    memory freed after the call is not handed out before the stream is done with it."""
    if stream is None:
        return _HERE_ALREADY
    if not isinstance(stream, torch.cuda.Stream):
        h = int(stream)          # 0 and 1 are both the legacy default stream
        stream = (torch.cuda.default_stream(dev) if h in (0, 1) else
                  torch.cuda.ExternalStream(h, device=dev))
    return torch.cuda.stream(stream)


# ---------------------------------------------------------------------------
# products grouped by expert
# ---------------------------------------------------------------------------
def switch_layer_grouped_workspace_size(R, K, O, N, dtype: int) -> int:
    n = _sz(0)
    _check(lib().switch_layer_grouped_workspace_size(R, K, O, N, dtype, ctypes.byref(n)),
           "grouped_workspace_size")
    return int(n.value)


def _grouped_workspace(workspace, R, K, O, N, dt, dev):
    if workspace is None:
        return torch.empty(switch_layer_grouped_workspace_size(R, K, O, N, dtype_code(dt)),
                           dtype=torch.uint8, device=dev)
    _require(workspace, "workspace", torch.uint8)
    if workspace.device != dev:
        raise ValueError("workspace is on %s: all tensors must be on %s" % (workspace.device, dev))
    return workspace


def grouped_matmul(x: torch.Tensor, offsets: torch.Tensor, W: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   check: bool = True) -> torch.Tensor:
    """y [R, O]: ``y[r] = W[e] x[r] + bias[e]`` for the rows offsets[e] <= r < offsets[e + 1]
    (see switch_layer_grouped_matmul in include/switch_layer.h).  Rows of no group keep what
    ``out`` holds (zeros when it is allocated here)."""
    if x.dim() != 2 or W.dim() != 3:
        raise ValueError("x must be [R, K] and W [N, O, K]")
    dev, dt = x.device, x.dtype
    R, K = x.shape
    N, O, _ = W.shape
    px = _at(x, "x", dt, (R, K), dev)
    pw = _at(W, "W", dt, (N, O, K), dev)
    po = _at(offsets, "offsets", torch.int32, (N + 1,), dev)
    pb = _at(bias, "bias", dt, (N, O), dev)
    with _allocating_on(stream, dev):
        if out is None:
            out = torch.zeros((R, O), dtype=dt, device=dev)
        ws = _grouped_workspace(workspace, R, K, O, N, dt, dev)
    with _on(dev):
        _check(lib().switch_layer_grouped_matmul(
            R, K, O, N, dtype_code(dt), px, po, pw, pb, _at(out, "out", dt, (R, O), dev),
            ws.data_ptr(), ws.numel(), _stream_handle(stream)), "grouped_matmul")
        if check:
            _check(switch_layer_device_status(ws, stream), "device status")
    return out


def grouped_matmul_backward(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                            W: torch.Tensor, dx: Optional[torch.Tensor] = None,
                            dW: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None,
                            check: bool = True) -> dict:
    """dx, dW and db of ``grouped_matmul`` for the gradient ``dy`` of its result.  With none
    of the three given, all are allocated; otherwise only the given ones are computed (the
    others are None in the result).  Rows of no group keep what ``dx`` holds (zeros when it
    is allocated here)."""
    if dy.dim() != 2 or x.dim() != 2 or W.dim() != 3:
        raise ValueError("dy must be [R, O], x [R, K] and W [N, O, K]")
    dev, dt = dy.device, dy.dtype
    R, K = x.shape
    N, O, _ = W.shape
    pdy = _at(dy, "dy", dt, (R, O), dev)
    px = _at(x, "x", dt, (R, K), dev)
    pw = _at(W, "W", dt, (N, O, K), dev)
    po = _at(offsets, "offsets", torch.int32, (N + 1,), dev)
    with _allocating_on(stream, dev):
        if dx is None and dW is None and db is None:
            dx = torch.zeros((R, K), dtype=dt, device=dev)
            dW = torch.empty((N, O, K), dtype=dt, device=dev)
            db = torch.empty((N, O), dtype=dt, device=dev)
        ws = _grouped_workspace(workspace, R, K, O, N, dt, dev)
    with _on(dev):
        _check(lib().switch_layer_grouped_matmul_backward(
            R, K, O, N, dtype_code(dt), pdy, px, po, pw, _at(dx, "dx", dt, (R, K), dev),
            _at(dW, "dW", dt, (N, O, K), dev), _at(db, "db", dt, (N, O), dev), ws.data_ptr(),
            ws.numel(), _stream_handle(stream)), "grouped_matmul_backward")
        if check:
            _check(switch_layer_device_status(ws, stream), "device status")
    return {"dx": dx, "dW": dW, "db": db}


# ---------------------------------------------------------------------------
# the norms around a block
# ---------------------------------------------------------------------------
_NORM_KINDS = {"rms": SWL_NORM_RMS, "layer": SWL_NORM_LAYER}


def _norm_struct(d, dev, kind, eps, w_pre, b_pre, w_post, b_post, scale) -> Norm:
    if kind not in _NORM_KINDS:
        raise ValueError("kind must be 'rms' or 'layer', got %r" % (kind,))
    f, shape = torch.float32, (d,)
    return Norm(_NORM_KINDS[kind], eps, _at(w_pre, "w_pre", f, shape, dev),
                _at(b_pre, "b_pre", f, shape, dev), _at(w_post, "w_post", f, shape, dev),
                _at(b_post, "b_post", f, shape, dev), _at(scale, "scale", f, shape, dev))


def norm_residual(x: torch.Tensor, y: Optional[torch.Tensor] = None,
                  w_pre: Optional[torch.Tensor] = None, b_pre: Optional[torch.Tensor] = None,
                  w_post: Optional[torch.Tensor] = None, b_post: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  kind: str = "rms", eps: float = 1e-6, r: Optional[torch.Tensor] = None,
                  h: Optional[torch.Tensor] = None, stream=None) -> dict:
    """The norms around a block (see switch_layer_norm_residual in include/switch_layer.h):
    ``r = x + gate * scale * norm(y; w_post, b_post)`` and ``h = norm(r; w_pre, b_pre)``.
    Without ``y`` ``r`` is ``x`` itself; without ``w_pre`` ``h`` is None.  ``r`` and ``h`` are
    allocated unless given (``r=x`` adds in place)."""
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    dev, dt, shape = x.device, x.dtype, x.shape
    T, d = shape
    n = _norm_struct(d, dev, kind, eps, w_pre, b_pre, w_post, b_post, scale)
    if y is None and r is not None:
        raise ValueError("r needs y")
    if w_pre is None and h is not None:
        raise ValueError("h needs w_pre")
    if (r is None and y is not None) or (h is None and w_pre is not None):
        with _allocating_on(stream, dev):
            r = torch.empty_like(x) if r is None and y is not None else r
            h = torch.empty_like(x) if h is None and w_pre is not None else h
    args = (T, d, dtype_code(dt), _at(x, "x", dt, shape, dev), _at(y, "y", dt, shape, dev),
            _at(gate, "gate", torch.float32, (T,), dev), ctypes.byref(n),
            _at(r, "r", dt, shape, dev), _at(h, "h", dt, shape, dev))
    if T > 0:
        with _on(dev):
            _check(lib().switch_layer_norm_residual(*args, _stream_handle(stream)),
                   "norm_residual")
    return {"r": x if y is None else r, "h": h}


def norm_residual_backward(dr: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                           r: torch.Tensor, y: Optional[torch.Tensor] = None,
                           w_pre: Optional[torch.Tensor] = None,
                           b_pre: Optional[torch.Tensor] = None,
                           w_post: Optional[torch.Tensor] = None,
                           b_post: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None,
                           scale: Optional[torch.Tensor] = None, kind: str = "rms",
                           eps: float = 1e-6, stream=None) -> dict:
    """Gradients of ``sum(dr * r) + sum(dh * h)`` of ``norm_residual`` (its ``r`` and its
    inputs): dx, dy, dgate, dscale, dw_pre, db_pre, dw_post, db_post; None where the forward
    call had no such input.  ``dr`` None: zero."""
    if r.dim() != 2:
        raise ValueError("r must be [T, d]")
    dev, dt, shape = r.device, r.dtype, r.shape
    T, d = shape
    f = torch.float32
    n = _norm_struct(d, dev, kind, eps, w_pre, b_pre, w_post, b_post, scale)
    pr, py = _at(r, "r", dt, shape, dev), _at(y, "y", dt, shape, dev)
    pdr, pdh = _at(dr, "dr", dt, shape, dev), _at(dh, "dh", dt, shape, dev)
    pg = _at(gate, "gate", f, (T,), dev)
    nbytes = _sz(0)
    _check(lib().switch_layer_norm_residual_backward_workspace_size(T, d, dtype_code(dt),
                                                                    ctypes.byref(nbytes)),
           "norm_residual_backward_workspace_size")
    with _allocating_on(stream, dev):
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
        g = {"dx": torch.empty_like(r), "dy": None if y is None else torch.empty_like(r)}
        for k, t in (("dgate", gate), ("dscale", scale), ("dw_pre", w_pre), ("db_pre", b_pre),
                     ("dw_post", w_post), ("db_post", b_post)):
            g[k] = None if t is None else torch.empty_like(t)
    o = NormGrads(*[_ptr(g[k]) for k, _ in NormGrads._fields_])
    with _on(dev):
        _check(lib().switch_layer_norm_residual_backward(
            T, d, dtype_code(dt), pdr, pdh, pr, py, pg, ctypes.byref(n), ctypes.byref(o),
            ws.data_ptr(), ws.numel(), _stream_handle(stream)), "norm_residual_backward")
    return g


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
def _one_device(tensors) -> torch.device:
    """The device that all of these CUDA tensors are on (None entries are skipped)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors on %s and %s: all must be on one device" % (dev, t.device))
    return dev


def adamw_state(params: Sequence[torch.Tensor], state_bits: int = 32,
                master: bool = False) -> dict:
    """Zero states for ``adamw_step`` over ``params``: lists ``m``, ``v`` (and ``m_scale``,
    ``v_scale`` with 8-bit states, ``master`` fp32 copies of the bf16 parameters when
    ``master``), and ``step``, the device counter."""
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
    dev = _one_device(params)
    if dev is None:
        raise ValueError("adamw_state needs at least one parameter")
    for p in params:
        _require(p, "param")
        dtype_code(p.dtype)
    eight = state_bits == 8
    dt = torch.float8_e4m3fn if eight else torch.float32

    def zeros(n, t):
        return torch.zeros(n, dtype=torch.uint8 if t == torch.float8_e4m3fn else t,
                           device=dev).view(t)

    nb = [-(-p.numel() // SWL_ADAMW_BLOCK) for p in params]
    return {"m": [zeros(p.numel(), dt) for p in params],
            "v": [zeros(p.numel(), dt) for p in params],
            "m_scale": [zeros(n, torch.float32) if eight else None for n in nb],
            "v_scale": [zeros(n, torch.float32) if eight else None for n in nb],
            "master": [p.detach().float() if master and p.dtype == torch.bfloat16 else None
                       for p in params],
            "step": torch.zeros(2, dtype=torch.int32, device=dev)}


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], state: dict,
               lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
               grad_scale: Optional[torch.Tensor] = None,
               lr_scale: Optional[torch.Tensor] = None, seed: int = 0, stream=None) -> None:
    """One AdamW step over all ``params`` in place (see switch_layer_adamw_step in
    include/switch_layer.h).  ``state`` is adamw_state's; ``weight_decay`` is one number or
    one per tensor; ``grad_scale`` and ``lr_scale`` are fp32 device tensors of one element."""
    n = len(params)
    wds = weight_decay if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
    lists = [state[k] for k in ("m", "v", "m_scale", "v_scale", "master")]
    if len(grads) != n or len(wds) != n or any(len(x) != n for x in lists):
        raise ValueError("params, grads, weight_decay and every list of the state must hold "
                         "%d entries" % n)
    step = state["step"]
    _require(step, "step", torch.int32)
    if step.numel() != 2:
        raise ValueError("step must hold 2 values")
    dev = step.device
    table = (AdamwTensor * max(1, n))()

    def at(t, name, dtype, count):
        # _require, the size and the device in one pass (this call is made for every tensor)
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
            _require(t, name, dtype)
        if t.device != dev:
            raise ValueError("%s is on %s: all tensors must be on %s" % (name, t.device, dev))
        if t.numel() != count:
            raise ValueError("%s must hold %d values, got %d" % (name, count, t.numel()))
        return t.data_ptr()

    for i, (p, g, m, v, ms, vs, w) in enumerate(zip(params, grads, *lists)):
        e = table[i]
        if not isinstance(p, torch.Tensor):
            raise TypeError("param must be a torch.Tensor")
        dt, k = p.dtype, p.numel()
        e.n, e.dtype, e.weight_decay = k, dtype_code(dt), wds[i]
        e.param = at(p, "param", dt, k)
        e.grad = at(g, "grad", dt, k)
        st = torch.float32
        e.state_bits = 32
        if ms is not None or vs is not None:
            st = torch.float8_e4m3fn
            e.state_bits = 8
            nb = -(-k // SWL_ADAMW_BLOCK)
            e.m_scale = at(ms, "m_scale", torch.float32, nb)
            e.v_scale = at(vs, "v_scale", torch.float32, nb)
        e.m = at(m, "m", st, k)
        e.v = at(v, "v", st, k)
        if w is not None:
            e.master = at(w, "master", torch.float32, k)
    gs = None if grad_scale is None else at(grad_scale, "grad_scale", torch.float32, 1)
    ls = None if lr_scale is None else at(lr_scale, "lr_scale", torch.float32, 1)
    cfg = Adamw(lr, betas[0], betas[1], eps, int(seed) & 0xFFFFFFFF)
    with _on(dev):
        _check(lib().switch_layer_adamw_step(table, n, ctypes.byref(cfg), step.data_ptr(), gs, ls,
                                             _stream_handle(stream)), "adamw_step")
