"""Beam MoE block forward on B200 (sm_100a): Python binding of libbeam_moe.so.

Argument marshalling only: every step of the block runs in the library's CUDA
kernels. Functions take torch tensors for device buffers (torch provides
device memory and the current stream) and raise BeamMoeError on any non-OK
status. There is no fallback: if the library is missing, the first call
raises ImportError.

The entry points mirror include/beam_moe.h one to one:
beam_moe_workspace_size, beam_moe_route, beam_moe_forward,
beam_moe_forward_routed, beam_moe_forward_traced, beam_moe_check, and the
Trace wrapper of beam_moe_trace_*. The row and linear operators
(beam_moe_permute, beam_moe_combine, beam_moe_linear and their backward calls)
check their tensors' types, shapes, strides and device here as well, since the
library sees addresses only, and raise ValueError.
"""
import ctypes
import os

__all__ = ["BeamMoeCfg", "BeamMoeError", "Trace", "OP_ROUTE", "OP_FORWARD", "N_STAGES",
           "STAGE_NAMES", "lib", "beam_cfg", "beam_moe_workspace_size", "beam_moe_route",
           "beam_moe_route_noalloc", "BeamMoeNvfp4Experts", "OP_FORWARD_NVFP4", "nvfp4_experts",
           "beam_moe_forward_nvfp4", "beam_moe_nvfp4_quantize", "OP_FORWARD_HOST",
           "OP_FORWARD_NVFP4_HOST", "HOST_CHUNK", "beam_moe_forward_host",
           "beam_moe_forward_nvfp4_host", "BeamMoeEpCfg", "ep_cfg", "beam_moe_ep_workspace_size",
           "beam_moe_ep_route", "beam_moe_ep_plan", "beam_moe_ep_dispatch", "beam_moe_ep_experts",
           "beam_moe_ep_combine", "beam_moe_selftest_wait",
           "beam_moe_forward", "beam_moe_forward_routed", "beam_moe_forward_traced",
           "beam_moe_forward_stages", "beam_moe_workspace_layout", "BeamMoeWsLayout",
           "BeamMoeEpHandle", "beam_moe_ep_export", "beam_moe_ep_import",
           "beam_moe_ep_release", "EpPeers", "torch_gather",
           "BeamMoeRowsCfg", "rows_cfg", "beam_moe_permute_workspace_size", "beam_moe_permute",
           "beam_moe_permute_backward", "beam_moe_combine", "beam_moe_combine_backward",
           "BeamMoeLinearCfg", "linear_cfg", "beam_moe_linear_workspace_size", "beam_moe_linear",
           "beam_moe_linear_backward", "BF16", "FP16", "FP32", "ACTS",
           "beam_moe_check"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbeam_moe.so")

OP_ROUTE = 0
OP_FORWARD = 1
OP_FORWARD_NVFP4 = 2
OP_FORWARD_HOST = 3
OP_FORWARD_NVFP4_HOST = 4
HOST_CHUNK = 8192
BF16, FP16, FP32 = 0, 1, 2
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu")
N_STAGES = 7
STAGE_NAMES = ("router_gemm", "router_topk", "scan", "permute", "gateup_gemm", "down_gemm",
               "combine")


class BeamMoeCfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("bias_mode", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("router_tc", ctypes.c_int32)]


class BeamMoeWsLayout(ctypes.Structure):
    """Byte offsets of the intermediates inside a forward workspace."""
    _fields_ = [("counts", ctypes.c_int64), ("offsets", ctypes.c_int64), ("ids", ctypes.c_int64),
                ("w", ctypes.c_int64), ("pos", ctypes.c_int64), ("xp", ctypes.c_int64),
                ("h", ctypes.c_int64), ("y", ctypes.c_int64), ("router_splits", ctypes.c_int32),
                ("router_tc", ctypes.c_int32), ("pair_gateup", ctypes.c_int32),
                ("pair_down", ctypes.c_int32), ("light_rows", ctypes.c_int32)]


class BeamMoeNvfp4Experts(ctypes.Structure):
    """NVFP4 expert weights (device pointers) and tensor scales."""
    _fields_ = [("w13_codes", ctypes.c_void_p), ("w13_scales", ctypes.c_void_p),
                ("w2_codes", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p),
                ("w13_scale", ctypes.c_float), ("w2_scale", ctypes.c_float),
                ("x_scale", ctypes.c_float), ("h_scale", ctypes.c_float)]


class BeamMoeEpCfg(ctypes.Structure):
    """Expert parallelism: ranks, this rank, most tokens per rank, receive rows."""
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("t_max", ctypes.c_int64),
                ("recv_cap", ctypes.c_int64)]


class BeamMoeEpHandle(ctypes.Structure):
    """A workspace exported for other processes (CUDA IPC handle and offset)."""
    _fields_ = [("ipc", ctypes.c_uint8 * 64), ("offset", ctypes.c_int64),
                ("bytes", ctypes.c_int64), ("device", ctypes.c_int32), ("pid", ctypes.c_int32)]


class BeamMoeRowsCfg(ctypes.Structure):
    """Token rows of the permute and combine operators."""
    _fields_ = [("width", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class BeamMoeLinearCfg(ctypes.Structure):
    """The linear operator: sizes, activation and types."""
    _fields_ = [("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("act", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_fp32", ctypes.c_int32)]


class BeamMoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {lib().beam_moe_status_string(status).decode()} ({status})")


_lib = None
_P = ctypes.c_void_p
_CFG = ctypes.POINTER(BeamMoeCfg)
_EP = ctypes.POINTER(BeamMoeEpCfg)
_PP = ctypes.POINTER(ctypes.c_void_p)
_ROWS = ctypes.POINTER(BeamMoeRowsCfg)
_LIN = ctypes.POINTER(BeamMoeLinearCfg)
_SIGS = {
    "beam_moe_workspace_size": [_CFG, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "beam_moe_route": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "beam_moe_route_noalloc": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P],
    "beam_moe_forward": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                         ctypes.c_size_t, _P],
    "beam_moe_forward_stages": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                _P, ctypes.c_size_t, _P],
    "beam_moe_workspace_layout": [_CFG, ctypes.c_int64, ctypes.c_int,
                                  ctypes.POINTER(BeamMoeWsLayout)],
    "beam_moe_forward_routed": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P],
    "beam_moe_forward_traced": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P, _P],
    "beam_moe_forward_nvfp4": [_CFG, ctypes.c_int64, _P, _P, _P,
                               ctypes.POINTER(BeamMoeNvfp4Experts), _P, _P, _P, _P, _P,
                               ctypes.c_size_t, _P],
    "beam_moe_forward_nvfp4_traced": [_CFG, ctypes.c_int64, _P, _P, _P,
                                      ctypes.POINTER(BeamMoeNvfp4Experts), _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P, _P],
    "beam_moe_forward_host": [_CFG, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                              _P],
    "beam_moe_forward_nvfp4_host": [_CFG, ctypes.c_int64, _P, _P, _P,
                                    ctypes.POINTER(BeamMoeNvfp4Experts), _P, _P, ctypes.c_size_t,
                                    _P],
    "beam_moe_nvfp4_quantize": [ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_float, _P, _P, _P],
    "beam_moe_ep_workspace_size": [_CFG, _EP, ctypes.POINTER(ctypes.c_size_t)],
    "beam_moe_ep_route": [_CFG, _EP, ctypes.c_int64, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "beam_moe_ep_plan": [_CFG, _EP, _P, _P, _P, ctypes.POINTER(ctypes.c_int64)],
    "beam_moe_ep_dispatch": [_CFG, _EP, ctypes.c_int64, _P, _P, _PP, _P, ctypes.c_size_t, _P],
    "beam_moe_ep_experts": [_CFG, _EP, _P, _P, _P, _PP, _P, ctypes.c_size_t, _P],
    "beam_moe_ep_combine": [_CFG, _EP, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P],
    "beam_moe_ep_export": [_P, ctypes.c_size_t, ctypes.POINTER(BeamMoeEpHandle)],
    "beam_moe_ep_import": [ctypes.POINTER(BeamMoeEpHandle), ctypes.c_size_t,
                           ctypes.POINTER(ctypes.c_void_p)],
    "beam_moe_ep_release": [ctypes.POINTER(BeamMoeEpHandle), _P],
    "beam_moe_permute_workspace_size": [_ROWS, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)],
    "beam_moe_permute": [_ROWS, ctypes.c_int64, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "beam_moe_permute_backward": [_ROWS, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P],
    "beam_moe_combine": [_ROWS, ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int32, _P, _P, _P,
                         _P],
    "beam_moe_combine_backward": [_ROWS, ctypes.c_int64, ctypes.c_int64, _P, _P, ctypes.c_int32,
                                  _P, _P, _P, _P, _P],
    "beam_moe_linear_workspace_size": [_LIN, ctypes.c_int64, ctypes.c_int32,
                                       ctypes.POINTER(ctypes.c_size_t)],
    "beam_moe_linear": [_LIN, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                        _P],
    "beam_moe_linear_backward": [_LIN, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                 ctypes.c_size_t, _P],
    "beam_moe_trace_create": [ctypes.c_int32, ctypes.POINTER(_P)],
    "beam_moe_trace_destroy": [_P],
    "beam_moe_trace_reset": [_P],
    "beam_moe_trace_read": [_P, _P, ctypes.POINTER(ctypes.c_int32)],
    "beam_moe_check": [_P, ctypes.c_size_t, _P, ctypes.POINTER(ctypes.c_uint32)],
    "beam_moe_selftest_wait": [_P, ctypes.c_size_t, ctypes.c_int32, _P],
    "beam_moe_status_string": [ctypes.c_int],
}


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libbeam_moe.so not built at {LIB_PATH}; run "
                              "`python -m sparse_moe_layer_beam_b200._build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_char_p if name == "beam_moe_status_string" else ctypes.c_int
        _lib = L
    return _lib


def beam_cfg(H=5120, I=2560, E=256, G=8, Gk=4, K=8, renormalize=True, bias_mode=0, scale=2.5,
             router_tc=False):
    """Configuration struct; the defaults are the Beam block. router_tc opts in
    to the router GEMM on tensor cores (exact three-way bf16 split of the FP32
    weights); the default is FP32 FMAs on CUDA cores."""
    return BeamMoeCfg(H, I, E, G, Gk, K, 1 if renormalize else 0, bias_mode, scale,
                      1 if router_tc else 0)


def _check(status, where):
    if status != 0:
        raise BeamMoeError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def beam_moe_workspace_size(cfg, T, op=OP_FORWARD):
    n = ctypes.c_size_t(0)
    _check(lib().beam_moe_workspace_size(ctypes.byref(cfg), T, op, ctypes.byref(n)),
           "beam_moe_workspace_size")
    return n.value


def beam_moe_route(cfg, x, w_router, bias, topk_ids, topk_w, expert_counts, ws, stream=None):
    T = x.shape[0] if x is not None else 0
    _check(lib().beam_moe_route(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias),
                                _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "beam_moe_route")


def beam_moe_route_noalloc(cfg, x, w_router, bias, topk_ids, topk_w, expert_counts=None,
                           stream=None):
    """Routing with the library's fixed scratch instead of a workspace, for
    callers that cannot allocate device memory (at most 2048 tokens and 256
    experts; concurrent calls on one device race)."""
    T = x.shape[0]
    _check(lib().beam_moe_route_noalloc(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router),
                                        _ptr(bias), _ptr(topk_ids), _ptr(topk_w),
                                        _ptr(expert_counts), _stream(stream)),
           "beam_moe_route_noalloc")


def beam_moe_forward(cfg, x, w_router, bias, w13, w2, out, ws, topk_ids=None, topk_w=None,
                     expert_counts=None, stream=None):
    T = x.shape[0]
    _check(lib().beam_moe_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias),
                                  _ptr(w13), _ptr(w2), _ptr(out), _ptr(topk_ids), _ptr(topk_w),
                                  _ptr(expert_counts), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "beam_moe_forward")


def beam_moe_forward_traced(cfg, x, w_router, bias, w13, w2, out, ws, trace, topk_ids=None,
                            topk_w=None, expert_counts=None, stream=None):
    T = x.shape[0]
    _check(lib().beam_moe_forward_traced(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router),
                                         _ptr(bias), _ptr(w13), _ptr(w2), _ptr(out),
                                         _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts),
                                         _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(stream), trace.handle),
           "beam_moe_forward_traced")


def beam_moe_forward_stages(cfg, x, w_router, bias, w13, w2, out, last_stage, ws, stream=None):
    """The forward's stages 0..last_stage (0 router GEMM ... 6 combine), leaving
    the intermediates in ws (see beam_moe_workspace_layout)."""
    T = x.shape[0]
    _check(lib().beam_moe_forward_stages(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router),
                                         _ptr(bias), _ptr(w13), _ptr(w2), _ptr(out), last_stage,
                                         _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(stream)), "beam_moe_forward_stages")


def beam_moe_workspace_layout(cfg, T, op=OP_FORWARD):
    """BeamMoeWsLayout of a workspace for T tokens on the current device."""
    out = BeamMoeWsLayout()
    _check(lib().beam_moe_workspace_layout(ctypes.byref(cfg), T, op, ctypes.byref(out)),
           "beam_moe_workspace_layout")
    return out


def beam_moe_forward_routed(cfg, x, topk_ids, topk_w, w13, w2, out, ws, expert_counts=None,
                            stream=None):
    T = x.shape[0]
    _check(lib().beam_moe_forward_routed(ctypes.byref(cfg), T, _ptr(x), _ptr(topk_ids),
                                         _ptr(topk_w), _ptr(w13), _ptr(w2), _ptr(out),
                                         _ptr(expert_counts), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_forward_routed")


def nvfp4_experts(w13_codes, w13_scales, w2_codes, w2_scales, w13_scale, w2_scale, x_scale,
                  h_scale):
    return BeamMoeNvfp4Experts(_ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
                               _ptr(w2_scales), w13_scale, w2_scale, x_scale, h_scale)


def beam_moe_forward_host(cfg, x_host, w_router, bias, w13, w2, out_host, ws, stream=None):
    """Forward on host buffers (x_host, out_host: CPU tensors, pinned for overlap)."""
    T = x_host.shape[0]
    _check(lib().beam_moe_forward_host(ctypes.byref(cfg), T, _ptr(x_host), _ptr(w_router),
                                       _ptr(bias), _ptr(w13), _ptr(w2), _ptr(out_host), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_forward_host")


def beam_moe_forward_nvfp4_host(cfg, x_host, w_router, bias, experts, out_host, ws, stream=None):
    T = x_host.shape[0]
    _check(lib().beam_moe_forward_nvfp4_host(ctypes.byref(cfg), T, _ptr(x_host), _ptr(w_router),
                                             _ptr(bias), ctypes.byref(experts), _ptr(out_host),
                                             _ptr(ws), ws.numel() * ws.element_size(),
                                             _stream(stream)),
           "beam_moe_forward_nvfp4_host")


def beam_moe_forward_nvfp4(cfg, x, w_router, bias, experts, out, ws, topk_ids=None, topk_w=None,
                           expert_counts=None, stream=None, trace=None):
    T = x.shape[0]
    args = (ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias), ctypes.byref(experts),
            _ptr(out), _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(stream))
    if trace is None:
        _check(lib().beam_moe_forward_nvfp4(*args), "beam_moe_forward_nvfp4")
    else:
        _check(lib().beam_moe_forward_nvfp4_traced(*args, trace.handle),
               "beam_moe_forward_nvfp4_traced")


def beam_moe_nvfp4_quantize(v, g, codes, scales, stream=None):
    rows, K = v.shape
    _check(lib().beam_moe_nvfp4_quantize(rows, K, _ptr(v), g, _ptr(codes), _ptr(scales),
                                         _stream(stream)), "beam_moe_nvfp4_quantize")


def beam_moe_check(ws, stream=None):
    """Synchronizes the stream, returns the device status bits (0 = clean) and
    clears them. Raises BeamMoeError on a CUDA error."""
    flags = ctypes.c_uint32(0)
    st = lib().beam_moe_check(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream),
                              ctypes.byref(flags))
    if st not in (0, 6):
        raise BeamMoeError(st, "beam_moe_check")
    return flags.value


def beam_moe_selftest_wait(ws, limit_ms, stream=None):
    """Runs the device self-check of a bounded wait that runs out."""
    _check(lib().beam_moe_selftest_wait(_ptr(ws), ws.numel() * ws.element_size(), limit_ms,
                                        _stream(stream)), "beam_moe_selftest_wait")


class Trace:
    """Per-stage CUDA-event timing of traced forward calls."""

    def __init__(self, capacity):
        h = _P()
        _check(lib().beam_moe_trace_create(capacity, ctypes.byref(h)), "beam_moe_trace_create")
        self.handle = h
        self.capacity = capacity

    def reset(self):
        _check(lib().beam_moe_trace_reset(self.handle), "beam_moe_trace_reset")

    def read(self):
        """List (one entry per traced call) of per-stage milliseconds."""
        n = ctypes.c_int32(0)
        buf = (ctypes.c_float * (self.capacity * N_STAGES))()
        _check(lib().beam_moe_trace_read(self.handle, buf, ctypes.byref(n)), "beam_moe_trace_read")
        return [list(buf[i * N_STAGES:(i + 1) * N_STAGES]) for i in range(n.value)]

    def close(self):
        if self.handle:
            lib().beam_moe_trace_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------ row and linear operators

# These calls can be shorter on the GPU than on the host, so the checks are kept
# to one comparison each and what torch is asked for is asked once a call.

_NAMES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}
_I32 = 3
_types = None    # tensor types of each kind (bf16 also as its 16-bit pattern); set last
_device = None   # () -> current CUDA device
_raw_stream = None  # (device) -> its current stream


def _bind_torch():
    global _types, _device, _raw_stream
    import torch
    _device = torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    # last: another thread that finds the types finds the rest as well
    _types = (frozenset((torch.bfloat16, torch.int16, torch.uint16)),
              frozenset((torch.float16,)), frozenset((torch.float32,)),
              frozenset((torch.int32,)))


def _begin(name, t):
    """The current device, which tensor t (never None) has to be on."""
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    if _types is None:
        _bind_torch()
    if not t.is_cuda or t.get_device() != _device():
        raise ValueError(f"{name}: not on the current CUDA device")
    _rows(name, t)
    return t.get_device()


def _rows(name, t):
    """The first dimension of a tensor that is required."""
    if t is None or not t.dim():
        raise ValueError(f"{name}: a tensor of two dimensions is required")
    return t.shape[0]


def _tensor(name, t, kind, dev, shape):
    """Address of a contiguous tensor of this kind and shape on device dev;
    None passes."""
    if t is None:
        return None
    if (t.shape == shape and t.dtype in _types[kind] and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}; "
                     f"expected a contiguous tensor {shape} of a type among "
                     f"{sorted(map(str, _types[kind]))} on cuda:{dev}")


def _need(name, t):
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    return t


def _workspace(ws, dev):
    """(address, bytes) of a workspace on device dev."""
    if ws is None or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous tensor on cuda:{dev} is required")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _on(dev, stream):
    return _raw_stream(dev) if stream is None else stream


def rows_cfg(width, n_experts, top_k, dtype="bf16"):
    """Token rows of `width` elements of dtype ("bf16", "fp16", "fp32"), routed
    to top_k of n_experts."""
    return BeamMoeRowsCfg(width, n_experts, top_k, _NAMES[dtype])


def beam_moe_permute_workspace_size(cfg, T):
    n = ctypes.c_size_t(0)
    _check(lib().beam_moe_permute_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)),
           "beam_moe_permute_workspace_size")
    return n.value


def beam_moe_permute(cfg, x, topk_ids, xp, pos, offsets, ws, stream=None):
    """Token rows sorted by expert: x [T, H], topk_ids [T, K] int32 -> xp
    [T*K, H], pos [T, K] int32, offsets [E+1] int32."""
    dev = _begin("x", x)
    T, H, K, d = x.shape[0], cfg.width, cfg.top_k, cfg.dtype
    _check(lib().beam_moe_permute(
        cfg, T, _tensor("x", x, d, dev, (T, H)),
        _tensor("topk_ids", _need("topk_ids", topk_ids), _I32, dev, (T, K)),
        _tensor("xp", _need("xp", xp), d, dev, (T * K, H)),
        _tensor("pos", _need("pos", pos), _I32, dev, (T, K)),
        _tensor("offsets", _need("offsets", offsets), _I32, dev, (cfg.n_experts + 1,)),
        *_workspace(ws, dev), _on(dev, stream)), "beam_moe_permute")


def beam_moe_permute_backward(cfg, dxp, pos, dx, stream=None):
    """dx[t] = sum_k dxp[pos[t, k]]: dxp [rows, H], pos [T, K] -> dx [T, H]."""
    dev = _begin("dx", dx)
    T, rows, H, d = dx.shape[0], _rows("dxp", dxp), cfg.width, cfg.dtype
    _check(lib().beam_moe_permute_backward(
        cfg, T, rows, _tensor("dxp", dxp, d, dev, (rows, H)),
        _tensor("pos", _need("pos", pos), _I32, dev, (T, cfg.top_k)),
        _tensor("dx", dx, d, dev, (T, H)), _on(dev, stream)), "beam_moe_permute_backward")


def _y_kind(cfg, y):
    """FP32 for fp32 rows, else the configuration's dtype."""
    return FP32 if y.dtype in _types[FP32] else cfg.dtype


def beam_moe_combine(cfg, y, pos, w, out, stream=None):
    """out[t] = sum_k w[t, k] y[pos[t, k]]: y [rows, H] of cfg's dtype or fp32,
    w [T, K] fp32 or None (ones) -> out [T, H]."""
    dev = _begin("out", out)
    T, rows, H, K = out.shape[0], _rows("y", y), cfg.width, cfg.top_k
    kind = _y_kind(cfg, y)
    _check(lib().beam_moe_combine(
        cfg, T, rows, _tensor("y", y, kind, dev, (rows, H)), kind,
        _tensor("pos", _need("pos", pos), _I32, dev, (T, K)), _tensor("w", w, FP32, dev, (T, K)),
        _tensor("out", out, cfg.dtype, dev, (T, H)), _on(dev, stream)), "beam_moe_combine")


def beam_moe_combine_backward(cfg, dout, y, pos, w, dy, dw, stream=None):
    """dy[pos[t, k]] = w[t, k] dout[t] (dy as y, or None), dw[t, k] =
    <dout[t], y[pos[t, k]]> (fp32 [T, K], or None; y may be None without it)."""
    dev = _begin("dout", dout)
    like = y if y is not None else dy
    T, rows, H, K = dout.shape[0], _rows("y or dy", like), cfg.width, cfg.top_k
    kind = _y_kind(cfg, like)
    _check(lib().beam_moe_combine_backward(
        cfg, T, rows, _tensor("dout", dout, cfg.dtype, dev, (T, H)),
        _tensor("y", y, kind, dev, (rows, H)), kind,
        _tensor("pos", _need("pos", pos), _I32, dev, (T, K)), _tensor("w", w, FP32, dev, (T, K)),
        _tensor("dy", dy, kind, dev, (rows, H)), _tensor("dw", dw, FP32, dev, (T, K)),
        _on(dev, stream)), "beam_moe_combine_backward")


def linear_cfg(n_in, n_out, n_experts=1, act="none", dtype="bf16", out_fp32=False):
    """Y = act(X W^T + bias) + residual over n_experts' rows; act is one of
    ACTS, dtype "bf16" or "fp16" (y and residual fp32 with out_fp32)."""
    return BeamMoeLinearCfg(n_in, n_out, n_experts, ACTS.index(act), _NAMES[dtype],
                            1 if out_fp32 else 0)


def _weight_rows(cfg):
    return cfg.n_out * 2 if cfg.act == 5 else cfg.n_out


def beam_moe_linear_workspace_size(cfg, rows, backward=False):
    n = ctypes.c_size_t(0)
    _check(lib().beam_moe_linear_workspace_size(ctypes.byref(cfg), rows, 1 if backward else 0,
                                                ctypes.byref(n)),
           "beam_moe_linear_workspace_size")
    return n.value


def beam_moe_linear(cfg, x, w, y, ws, bias=None, residual=None, offsets=None, z=None,
                    stream=None):
    """y = act(x w_e^T + bias_e) + residual for the rows of every expert e: x
    [rows, n_in], w [E, N, n_in] (N = n_out, 2 n_out for swiglu), bias [E, N]
    fp32, residual [rows, n_out], offsets [E+1] int32 (None: one expert) -> y
    [rows, n_out] and, if given, z [rows, N] = x w_e^T + bias_e."""
    dev = _begin("x", x)
    rows, E, N, d = x.shape[0], cfg.n_experts, _weight_rows(cfg), cfg.dtype
    K, M, out = cfg.n_in, cfg.n_out, FP32 if cfg.out_fp32 else d
    _check(lib().beam_moe_linear(
        cfg, rows, _tensor("x", x, d, dev, (rows, K)),
        _tensor("w", _need("w", w), d, dev, (E, N, K)), _tensor("bias", bias, FP32, dev, (E, N)),
        _tensor("residual", residual, out, dev, (rows, M)),
        _tensor("offsets", offsets, _I32, dev, (E + 1,)),
        _tensor("y", _need("y", y), out, dev, (rows, M)), _tensor("z", z, d, dev, (rows, N)),
        *_workspace(ws, dev), _on(dev, stream)), "beam_moe_linear")


def beam_moe_linear_backward(cfg, dy, x, w, ws, dx=None, dw=None, dbias=None, z=None,
                             offsets=None, stream=None):
    """Gradients of beam_moe_linear: dy [rows, n_out], x, w and the forward's z
    -> dx [rows, n_in], dw [E, N, n_in], dbias [E, N] fp32 (each may be None)."""
    dev = _begin("dy", dy)
    rows, E, N, d = dy.shape[0], cfg.n_experts, _weight_rows(cfg), cfg.dtype
    K, M = cfg.n_in, cfg.n_out
    _check(lib().beam_moe_linear_backward(
        cfg, rows, _tensor("dy", dy, d, dev, (rows, M)), _tensor("x", x, d, dev, (rows, K)),
        _tensor("w", w, d, dev, (E, N, K)), _tensor("z", z, d, dev, (rows, N)),
        _tensor("offsets", offsets, _I32, dev, (E + 1,)), _tensor("dx", dx, d, dev, (rows, K)),
        _tensor("dw", dw, d, dev, (E, N, K)), _tensor("dbias", dbias, FP32, dev, (E, N)),
        *_workspace(ws, dev), _on(dev, stream)), "beam_moe_linear_backward")


# ------------------------------------------------------------ expert parallelism

def ep_cfg(world, rank, t_max, recv_cap):
    return BeamMoeEpCfg(world, rank, t_max, recv_cap)


def _addr(v):
    return v if isinstance(v, int) or v is None else v.data_ptr()


def _peers(peer_ws):
    return (ctypes.c_void_p * len(peer_ws))(*[_addr(p) for p in peer_ws])


def beam_moe_ep_workspace_size(cfg, ep):
    n = ctypes.c_size_t(0)
    _check(lib().beam_moe_ep_workspace_size(ctypes.byref(cfg), ctypes.byref(ep), ctypes.byref(n)),
           "beam_moe_ep_workspace_size")
    return n.value


def beam_moe_ep_route(cfg, ep, x, w_router, bias, counts, ws, stream=None):
    _check(lib().beam_moe_ep_route(ctypes.byref(cfg), ctypes.byref(ep), x.shape[0], _ptr(x),
                                   _ptr(w_router), _ptr(bias), _ptr(counts), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_ep_route")


def beam_moe_ep_plan(cfg, ep, counts_all):
    """counts_all: int32 array [world][E] (host). Returns (send_base [E],
    recv_counts [E/world], recv_rows)."""
    import numpy as np
    counts_all = np.ascontiguousarray(counts_all, dtype=np.int32)
    send_base = np.zeros(cfg.n_experts, dtype=np.int32)
    recv_counts = np.zeros(cfg.n_experts // ep.world, dtype=np.int32)
    rows = ctypes.c_int64(0)
    _check(lib().beam_moe_ep_plan(ctypes.byref(cfg), ctypes.byref(ep), counts_all.ctypes.data,
                                  send_base.ctypes.data, recv_counts.ctypes.data,
                                  ctypes.byref(rows)), "beam_moe_ep_plan")
    return send_base, recv_counts, rows.value


def beam_moe_ep_dispatch(cfg, ep, x, send_base, peer_ws, ws, stream=None):
    _check(lib().beam_moe_ep_dispatch(ctypes.byref(cfg), ctypes.byref(ep), x.shape[0], _ptr(x),
                                      _ptr(send_base), _peers(peer_ws), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_ep_dispatch")


def beam_moe_ep_experts(cfg, ep, recv_counts, w13, w2, peer_ws, ws, stream=None):
    """recv_counts: int32 array [E/world] (host); w13, w2: this rank's experts
    (tensors or device addresses)."""
    import numpy as np
    rc = np.ascontiguousarray(recv_counts, dtype=np.int32)
    _check(lib().beam_moe_ep_experts(ctypes.byref(cfg), ctypes.byref(ep), rc.ctypes.data,
                                     _addr(w13), _addr(w2), _peers(peer_ws), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_ep_experts")


def beam_moe_ep_combine(cfg, ep, T, out, ws, stream=None):
    _check(lib().beam_moe_ep_combine(ctypes.byref(cfg), ctypes.byref(ep), T, _ptr(out), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "beam_moe_ep_combine")


def beam_moe_ep_export(ws):
    """This rank's workspace as bytes another process can import."""
    h = BeamMoeEpHandle()
    _check(lib().beam_moe_ep_export(_ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(h)),
           "beam_moe_ep_export")
    return bytes(h)


def beam_moe_ep_import(blob, ws_bytes):
    """Device address of another process's exported workspace."""
    h = BeamMoeEpHandle.from_buffer_copy(blob)
    p = ctypes.c_void_p(0)
    _check(lib().beam_moe_ep_import(ctypes.byref(h), ws_bytes, ctypes.byref(p)),
           "beam_moe_ep_import")
    return p.value


def beam_moe_ep_release(blob, peer_ws):
    h = BeamMoeEpHandle.from_buffer_copy(blob)
    _check(lib().beam_moe_ep_release(ctypes.byref(h), peer_ws), "beam_moe_ep_release")


class EpPeers:
    """Every rank's workspace as an address this process can store to.

    gather(blob) must return the list of every rank's blob in rank order (an
    all-gather, e.g. torch.distributed.all_gather_object); export / import_ /
    release default to the library's CUDA IPC calls. This rank's own slot is
    its local workspace; every other slot is imported, and close() releases
    them (call it on every rank, after a barrier, before any rank frees its
    workspace)."""

    def __init__(self, ep, ws, gather, export=None, import_=None, release=None):
        self._release = release or beam_moe_ep_release
        mine = (export or beam_moe_ep_export)(ws)
        blobs = gather(mine)
        if len(blobs) != ep.world or blobs[ep.rank] != mine:
            raise ValueError("gather must return every rank's blob in rank order")
        nbytes = ws.numel() * ws.element_size()
        self.ptrs, self._opened = [], []
        try:
            for r, blob in enumerate(blobs):
                if r == ep.rank:
                    self.ptrs.append(ws.data_ptr())
                else:
                    p = (import_ or beam_moe_ep_import)(blob, nbytes)
                    self._opened.append((blob, p))
                    self.ptrs.append(p)
        except Exception:
            self.close()
            raise

    def close(self):
        while self._opened:
            blob, p = self._opened.pop()
            self._release(blob, p)


def torch_gather(group=None):
    """An all-gather of Python objects over a torch.distributed group."""
    import torch.distributed as dist

    def gather(obj):
        out = [None] * dist.get_world_size(group)
        dist.all_gather_object(out, obj, group=group)
        return out
    return gather
