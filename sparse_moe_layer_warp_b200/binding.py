"""Thin ctypes binding of ``libmoe_layer.so`` (C ABI declared in ``include/moe_layer.h``).

Argument marshalling only: torch tensors supply device pointers and the current CUDA
stream; every step of the layer runs in the library's kernels.  There is no fallback: if
the shared library is missing or fails to load, importing the functions raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_layer.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_ALIGNMENT = 3
MOE_ERR_WORKSPACE = 4
MOE_ERR_CUDA = 5
MOE_ERR_DEVICE_TIMEOUT = 6

MOE_F32 = 0
MOE_BF16 = 1

# every entry point the header declares (checked by tests against the built library)
EXPORTS = ("moe_layer_init", "moe_layer_destroy", "moe_workspace_size", "moe_workspace_init",
           "moe_route", "moe_route_from_logits", "moe_forward", "moe_forward_profiled",
           "moe_device_status", "moe_status_string", "moe_router_logits_static",
           "moe_router_stats", "moe_update_router_bias", "moe_forward_launch_count",
           "moe_selftest_wait_timeout", "moe_expert_health", "moe_backward",
           "moe_backward_workspace_size", "moe_saved_size", "moe_forward_save",
           "moe_backward_saved", "moe_backward_ex", "moe_set_option", "moe_layer_init_ep",
           "moe_forward_partial", "moe_ep_plan", "moe_ep_pack", "moe_ep_combine",
           "moe_gemm_clock", "moe_mxfp4_quantize", "moe_mxfp4_dequantize",
           "moe_mxfp4_tile_scales", "moe_layer_init_mxfp4", "moe_forward_few")
MXFP4_BLOCK = 32  # values that share a scale
MOE_BACKWARD_OVERWRITE = 1
MOE_OPTION_H_HANDOVER = 1
MOE_OPTION_SHARED_SIDE_SMS = 2
MOE_OPTION_ROW_GATHER_IN_GEMM = 3
MOE_OPTION_GEMM_CLOCK = 4
MOE_PROFILE_STAGES = 7
PROFILE_STAGE_NAMES = ("router_logits", "topk_gates_hist", "permute_scatter", "row_gather",
                       "expert_up_swiglu", "expert_down", "combine")


class moe_config(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int), ("d_model", ctypes.c_int),
                ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("d_ff", ctypes.c_int),
                ("n_shared", ctypes.c_int), ("dtype", ctypes.c_int),
                ("routed_scale", ctypes.c_float)]


class moe_weights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p)]


class moe_mxfp4_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_router", "router_bias", "w_gate", "w_up",
                                               "w_down", "scale_gate", "scale_up",
                                               "scale_down")]


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: status {status} ({status_string(status)})")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe_layer.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise OSError(f"{path} is missing: build it with `python -m "
                          "sparse_moe_layer_warp_b200.build`")
        lib = ctypes.CDLL(path)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.moe_layer_init.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights),
                                       ctypes.POINTER(P)]
        lib.moe_layer_destroy.argtypes = [P]
        lib.moe_workspace_size.argtypes = [P, I]
        lib.moe_workspace_size.restype = Z
        lib.moe_workspace_init.argtypes = [P, P, Z, P]
        lib.moe_route.argtypes = [P, P, I, P, P, P, P, P, P, P, P, Z, P]
        lib.moe_route_from_logits.argtypes = [P, P, I, P, P, P, P, P, P, P, Z, P]
        lib.moe_forward.argtypes = [P, P, I, P, P, Z, P]
        lib.moe_forward_profiled.argtypes = [P, P, I, P, P, Z, P, ctypes.POINTER(P), I]
        lib.moe_device_status.argtypes = [P, P, Z, P]
        lib.moe_gemm_clock.argtypes = [P, P, Z, ctypes.POINTER(ctypes.c_double), P]
        lib.moe_router_logits_static.argtypes = [P, P, I, P, P]
        lib.moe_router_stats.argtypes = [P, P, P, I, I, P, P, P, P, Z, P]
        lib.moe_update_router_bias.argtypes = [P, P, I, ctypes.c_float, P, P]
        lib.moe_selftest_wait_timeout.argtypes = [P, P, Z, I, P]
        lib.moe_expert_health.argtypes = [P, I, P, P, P, P, Z, P]
        lib.moe_backward.argtypes = [P, P, I, P, P, P, P, P, P, P, Z, P]
        lib.moe_backward_workspace_size.argtypes = [P, I]
        lib.moe_backward_workspace_size.restype = Z
        lib.moe_saved_size.argtypes = [P, I]
        lib.moe_saved_size.restype = Z
        lib.moe_forward_save.argtypes = [P, P, I, P, P, Z, P, Z, P]
        lib.moe_backward_saved.argtypes = [P, P, I, P, P, Z, P, P, P, P, P, P, Z, P]
        lib.moe_backward_ex.argtypes = [P, P, I, P, P, Z, ctypes.c_uint, P, P, P, P, P, P, Z, P]
        lib.moe_set_option.argtypes = [P, I, I]
        lib.moe_layer_init_ep.argtypes = [ctypes.POINTER(moe_config),
                                          ctypes.POINTER(moe_weights), I, I, ctypes.POINTER(P)]
        lib.moe_forward_partial.argtypes = [P, P, I, P, P, I, I, I, I, P, P, Z, P]
        lib.moe_ep_plan.argtypes = [P, P, I, I, P, P, P, P, P, Z, P]
        lib.moe_ep_pack.argtypes = [P, P, P, P, I, I, P, P, P, P, P, P]
        lib.moe_ep_combine.argtypes = [P, P, P, P, P, I, I, P, P]
        lib.moe_mxfp4_quantize.argtypes = [P, I, ctypes.c_longlong, I, P, P, P]
        lib.moe_mxfp4_dequantize.argtypes = [P, P, ctypes.c_longlong, I, P, I, P]
        lib.moe_mxfp4_tile_scales.argtypes = [P, ctypes.c_longlong, I, P, P]
        lib.moe_layer_init_mxfp4.argtypes = [ctypes.POINTER(moe_config),
                                             ctypes.POINTER(moe_mxfp4_weights),
                                             ctypes.POINTER(P)]
        lib.moe_forward_few.argtypes = [P, P, I, P, P, Z, P]
        lib.moe_forward_launch_count.argtypes = [P, I]
        lib.moe_forward_launch_count.restype = I
        lib.moe_status_string.argtypes = [I]
        lib.moe_status_string.restype = ctypes.c_char_p
        for name in ("moe_layer_init", "moe_layer_destroy", "moe_workspace_init", "moe_route",
                     "moe_route_from_logits", "moe_forward", "moe_forward_profiled",
                     "moe_device_status", "moe_router_logits_static", "moe_router_stats",
                     "moe_update_router_bias", "moe_selftest_wait_timeout",
                     "moe_expert_health", "moe_backward", "moe_forward_save",
                     "moe_backward_saved", "moe_backward_ex", "moe_set_option", "moe_layer_init_ep",
                     "moe_forward_partial", "moe_ep_plan", "moe_ep_pack", "moe_ep_combine",
                     "moe_gemm_clock", "moe_mxfp4_quantize", "moe_mxfp4_dequantize",
                     "moe_mxfp4_tile_scales", "moe_layer_init_mxfp4", "moe_forward_few"):
            getattr(lib, name).restype = I
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().moe_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoEError(fn, status)


def _dense(t) -> None:
    if not t.is_contiguous():
        raise ValueError(f"the library takes contiguous (dense row-major) tensors; got shape "
                         f"{tuple(t.shape)} with strides {tuple(t.stride())}")


def _addr(t) -> int:
    """Device address of a tensor handed to the C ABI.  The library reads and writes dense
    row-major device memory through raw pointers, so a strided view or a host tensor is
    refused here, before anything is launched."""
    _dense(t)
    if not t.is_cuda:
        raise ValueError(f"the library takes CUDA tensors; got one on {t.device}")
    return t.data_ptr()


def _p(t):
    return None if t is None else ctypes.c_void_p(_addr(t))


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class _Here:
    """The caller's device and stream are the call's: nothing to switch or to hand over."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False

    @staticmethod
    def new(t):
        return t


_HERE = _Here()


class _There:
    """A call's device and stream made current: what it allocates comes from the pool of the stream
    that writes it.  Memory that crosses between that stream and the caller's goes back to its pool
    only once the other is done with it: the caller's `tensors`, and results (`new`)."""

    def __init__(self, dev, stream, tensors):
        self.caller = None
        if stream is None:
            self.ctx = torch.cuda.device(dev)
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
        if stream.device.index != dev:
            raise ValueError(f"stream: of {stream.device}, the call's tensors are on cuda:{dev}")
        self.ctx = torch.cuda.stream(stream)
        self.caller = torch.cuda.current_stream(dev)
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)

    def __enter__(self):
        self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)

    def new(self, t):
        if self.caller is not None:
            t.record_stream(self.caller)
        return t


def _on(dev, stream, *tensors):
    """Context of a call on `stream` (None: the current one) of device `dev` that reads or writes the
    caller's `tensors`.  Switches only where needed: for a small matrix that takes longer than the
    kernel."""
    if dev == torch._C._cuda_getDevice() and (
            stream is None
            or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev)):
        return _HERE
    return _There(dev, stream, tensors)


def _call_here(dev, fn, *args) -> None:
    """Library call `fn` on the current stream of device `dev`, its last argument."""
    _check(fn, getattr(_lib or load_library(), fn)(
        *args, torch._C._cuda_getCurrentRawStream(dev)))


# ------------------------------------------------------------------ C-ABI mirrors
def moe_layer_init(cfg: moe_config, w_router, router_bias, w_gate, w_up, w_down):
    lib = load_library()
    w = moe_weights(_addr(w_router), None if router_bias is None else _addr(router_bias),
                    _addr(w_gate), _addr(w_up), _addr(w_down))
    h = ctypes.c_void_p()
    _check("moe_layer_init", lib.moe_layer_init(ctypes.byref(cfg), ctypes.byref(w),
                                                ctypes.byref(h)))
    return h


def moe_layer_init_ep(cfg: moe_config, expert_begin: int, expert_end: int, w_router,
                      router_bias, w_gate, w_up, w_down):
    """Handle over the routed experts [expert_begin, expert_end) of a bf16 layer (weights:
    those experts then the shared expert; the full router)."""
    lib = load_library()
    w = moe_weights(_addr(w_router), None if router_bias is None else _addr(router_bias),
                    _addr(w_gate), _addr(w_up), _addr(w_down))
    h = ctypes.c_void_p()
    _check("moe_layer_init_ep", lib.moe_layer_init_ep(ctypes.byref(cfg), ctypes.byref(w),
                                                      int(expert_begin), int(expert_end),
                                                      ctypes.byref(h)))
    return h


def moe_layer_init_mxfp4(cfg: moe_config, w_router, router_bias, w_gate, w_up, w_down):
    """Handle of a layer over MXFP4 expert weights: w_gate, w_up, w_down are (codes, tiled
    scales)."""
    lib = load_library()
    w = moe_mxfp4_weights(_addr(w_router), None if router_bias is None else _addr(router_bias),
                          *(_addr(t[0]) for t in (w_gate, w_up, w_down)),
                          *(_addr(t[1]) for t in (w_gate, w_up, w_down)))
    h = ctypes.c_void_p()
    _check("moe_layer_init_mxfp4", lib.moe_layer_init_mxfp4(ctypes.byref(cfg), ctypes.byref(w),
                                                            ctypes.byref(h)))
    return h


def moe_forward_partial(handle, x, n_tokens, topk_idx, topk_gate, expert_begin, expert_end,
                        shared_begin, shared_end, out, ws, stream=None) -> None:
    """fp32 partial output of an expert range (see include/moe_layer.h)."""
    _check("moe_forward_partial", load_library().moe_forward_partial(
        handle, _p(x), int(n_tokens), _p(topk_idx), _p(topk_gate), int(expert_begin),
        int(expert_end), int(shared_begin), int(shared_end), _p(out), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_ep_plan(handle, topk_idx, n_tokens, n_ranks, send_counts, send_offsets, send_perm,
                send_slot, ws, stream=None) -> None:
    _check("moe_ep_plan", load_library().moe_ep_plan(
        handle, _p(topk_idx), int(n_tokens), int(n_ranks), _p(send_counts), _p(send_offsets),
        _p(send_perm), _p(send_slot), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_ep_pack(handle, x, topk_idx, topk_gate, n_tokens, n_ranks, send_perm, send_offsets,
                x_send, idx_send, gate_send, stream=None) -> None:
    _check("moe_ep_pack", load_library().moe_ep_pack(
        handle, _p(x), _p(topk_idx), _p(topk_gate), int(n_tokens), int(n_ranks), _p(send_perm),
        _p(send_offsets), _p(x_send), _p(idx_send), _p(gate_send), _stream(stream)))


def moe_ep_combine(handle, back, send_slot, send_offsets, shared, n_tokens, n_ranks, out,
                   stream=None) -> None:
    _check("moe_ep_combine", load_library().moe_ep_combine(
        handle, _p(back), _p(send_slot), _p(send_offsets), _p(shared), int(n_tokens),
        int(n_ranks), _p(out), _stream(stream)))


def moe_layer_destroy(handle) -> None:
    _check("moe_layer_destroy", load_library().moe_layer_destroy(handle))


def moe_set_option(handle, option: int, value: int) -> None:
    """Launch-plan option of a handle (MOE_OPTION_H_HANDOVER; see include/moe_layer.h)."""
    _check("moe_set_option", load_library().moe_set_option(handle, int(option), int(value)))


def moe_workspace_size(handle, n_tokens: int) -> int:
    return int(load_library().moe_workspace_size(handle, int(n_tokens)))


def moe_workspace_init(handle, ws, stream=None) -> None:
    _check("moe_workspace_init", load_library().moe_workspace_init(
        handle, _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_route(handle, x, n_tokens, logits_out, topk_idx, topk_gate, expert_counts,
              expert_offsets, perm, slot_row, ws, stream=None) -> None:
    _check("moe_route", load_library().moe_route(
        handle, _p(x), int(n_tokens), _p(logits_out), _p(topk_idx), _p(topk_gate),
        _p(expert_counts), _p(expert_offsets), _p(perm), _p(slot_row), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_from_logits(handle, logits, n_tokens, topk_idx, topk_gate, expert_counts,
                          expert_offsets, perm, slot_row, ws, stream=None) -> None:
    _check("moe_route_from_logits", load_library().moe_route_from_logits(
        handle, _p(logits), int(n_tokens), _p(topk_idx), _p(topk_gate), _p(expert_counts),
        _p(expert_offsets), _p(perm), _p(slot_row), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_forward(handle, x, n_tokens, out, ws, stream=None) -> None:
    _check("moe_forward", load_library().moe_forward(
        handle, _p(x), int(n_tokens), _p(out), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_forward_few(handle, x, n_tokens, out, ws, stream=None) -> None:
    """The whole layer for a few tokens in one launch (see include/moe_layer.h)."""
    _check("moe_forward_few", load_library().moe_forward_few(
        handle, _p(x), int(n_tokens), _p(out), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


_DTYPE_CODE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _conversion(m, name, codes, scales):
    """(rows, cols, dtype code) of matrix m, whose codes and scales have to go with it."""
    if m.dtype not in _DTYPE_CODE:
        raise ValueError(f"{name}: expected fp32 or bf16, got {m.dtype}")
    n, cols = m.numel(), int(m.shape[-1])
    for what, t, per in (("codes", codes, 2), ("scales", scales, MXFP4_BLOCK)):
        _expect_bytes(what, t, n // per, m.device)
    return n // max(cols, 1), cols, _DTYPE_CODE[m.dtype]


def _expect_bytes(name, t, n, device):
    if t.dtype != torch.uint8 or t.numel() != n or t.device != device:
        raise ValueError(f"{name}: expected {n} bytes (uint8) on {device}, got {t.numel()} of "
                         f"{t.dtype} on {t.device}")


def moe_mxfp4_quantize(src, codes, scales, stream=None) -> None:
    """codes and scales of `src` [.., cols] (fp32 or bf16; see include/moe_layer.h)."""
    rows, cols, dtype = _conversion(src, "src", codes, scales)
    _check("moe_mxfp4_quantize", load_library().moe_mxfp4_quantize(
        _p(src), dtype, rows, cols, _p(codes), _p(scales), _stream(stream)))


def moe_mxfp4_dequantize(codes, scales, dst, stream=None) -> None:
    """The values that codes and scales stand for, into `dst` [.., cols] (fp32 or bf16)."""
    rows, cols, dtype = _conversion(dst, "dst", codes, scales)
    _check("moe_mxfp4_dequantize", load_library().moe_mxfp4_dequantize(
        _p(codes), _p(scales), rows, cols, _p(dst), dtype, _stream(stream)))


def moe_mxfp4_tile_scales(scales, tiled, stream=None) -> None:
    """`scales` [.., rows, cols / 32] in the order in which the layer's kernels load them."""
    kb = int(scales.shape[-1])
    _expect_bytes("scales", scales, scales.numel(), scales.device)
    _expect_bytes("tiled", tiled, scales.numel(), scales.device)
    _check("moe_mxfp4_tile_scales", load_library().moe_mxfp4_tile_scales(
        _p(scales), scales.numel() // max(kb, 1), kb * MXFP4_BLOCK, _p(tiled), _stream(stream)))


def moe_backward_workspace_size(handle, n_tokens: int) -> int:
    return int(load_library().moe_backward_workspace_size(handle, int(n_tokens)))


def moe_backward(handle, x, n_tokens, dout, dx, dw_router, dw_gate, dw_up, dw_down, ws,
                 stream=None) -> None:
    """Gradients of <forward(x), dout> (see include/moe_layer.h); fp32 outputs."""
    _check("moe_backward", load_library().moe_backward(
        handle, _p(x), int(n_tokens), _p(dout), _p(dx), _p(dw_router), _p(dw_gate), _p(dw_up),
        _p(dw_down), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_saved_size(handle, n_tokens: int) -> int:
    return int(load_library().moe_saved_size(handle, int(n_tokens)))


def moe_forward_save(handle, x, n_tokens, out, saved, ws, stream=None) -> None:
    """moe_forward that also keeps the fp32 pre-activations for moe_backward_saved."""
    _check("moe_forward_save", load_library().moe_forward_save(
        handle, _p(x), int(n_tokens), _p(out), _p(saved), saved.numel() * saved.element_size(),
        _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_backward_saved(handle, x, n_tokens, dout, saved, dx, dw_router, dw_gate, dw_up, dw_down,
                       ws, stream=None) -> None:
    """moe_backward reading the pre-activations kept by moe_forward_save."""
    _check("moe_backward_saved", load_library().moe_backward_saved(
        handle, _p(x), int(n_tokens), _p(dout), _p(saved), saved.numel() * saved.element_size(),
        _p(dx), _p(dw_router), _p(dw_gate), _p(dw_up), _p(dw_down), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_backward_ex(handle, x, n_tokens, dout, saved, flags, dx, dw_router, dw_gate, dw_up,
                    dw_down, ws, stream=None) -> None:
    """moe_backward with options: `saved` (or None) and flags (MOE_BACKWARD_OVERWRITE)."""
    nbytes = 0 if saved is None else saved.numel() * saved.element_size()
    _check("moe_backward_ex", load_library().moe_backward_ex(
        handle, _p(x), int(n_tokens), _p(dout), None if saved is None else _p(saved), nbytes,
        int(flags), _p(dx), _p(dw_router), _p(dw_gate), _p(dw_up), _p(dw_down), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_health(handle, n_tokens, act_rms, param_norm, ratios, ws, stream=None) -> None:
    """Expert health signals of the last forward on `ws` (see include/moe_layer.h)."""
    _check("moe_expert_health", load_library().moe_expert_health(
        handle, int(n_tokens), _p(act_rms), _p(param_norm), _p(ratios), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_selftest_wait_timeout(handle, ws, limit_us: int, stream=None) -> None:
    """Launch the library's timeout self-test kernel (see include/moe_layer.h)."""
    _check("moe_selftest_wait_timeout", load_library().moe_selftest_wait_timeout(
        handle, _p(ws), ws.numel() * ws.element_size(), int(limit_us), _stream(stream)))


def moe_forward_launch_count(handle, n_tokens: int) -> int:
    """Kernel launches of one moe_forward of n_tokens tokens (-1: invalid arguments)."""
    return int(load_library().moe_forward_launch_count(handle, int(n_tokens)))


def moe_forward_profiled(handle, x, n_tokens, out, ws, events, stream=None) -> None:
    """`events`: MOE_PROFILE_STAGES + 1 torch.cuda.Event(enable_timing=True) objects."""
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event on its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check("moe_forward_profiled", load_library().moe_forward_profiled(
        handle, _p(x), int(n_tokens), _p(out), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream), arr, len(events)))


def moe_router_logits_static(handle, x, n_tokens, logits_out, stream=None, *, d_model=None,
                             n_experts=None, dtype=None) -> None:
    """Router logits with the library's own static scratch (no workspace argument), for
    callers that cannot allocate device memory; see include/moe_layer.h for the limits.
    With d_model, n_experts and dtype given (MoELayer passes them), x and logits_out are
    checked to hold n_tokens rows before the library reads and writes them."""
    if d_model is not None:
        if x.dtype != dtype or x.numel() < int(n_tokens) * int(d_model):
            raise ValueError(f"x: expected at least {int(n_tokens)} x {int(d_model)} elements "
                             f"of {dtype}, got {tuple(x.shape)} of {x.dtype}")
        if (logits_out.dtype != torch.float32 or
                logits_out.numel() < int(n_tokens) * int(n_experts)):
            raise ValueError(f"logits_out: expected at least {int(n_tokens)} x {int(n_experts)}"
                             f" fp32 elements, got {tuple(logits_out.shape)} of "
                             f"{logits_out.dtype}")
    _check("moe_router_logits_static", load_library().moe_router_logits_static(
        handle, _p(x), int(n_tokens), _p(logits_out), _stream(stream)))


def moe_router_stats(handle, logits, topk_idx, n_tokens, n_groups, p_mean, f_sel, scalars, ws,
                     stream=None) -> None:
    _check("moe_router_stats", load_library().moe_router_stats(
        handle, _p(logits), _p(topk_idx), int(n_tokens), int(n_groups), _p(p_mean), _p(f_sel),
        _p(scalars), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_update_router_bias(handle, expert_counts, n_tokens, gamma, bias, stream=None) -> None:
    _check("moe_update_router_bias", load_library().moe_update_router_bias(
        handle, _p(expert_counts), int(n_tokens), float(gamma), _p(bias), _stream(stream)))


def moe_device_status(handle, ws, stream=None) -> int:
    return int(load_library().moe_device_status(handle, _p(ws), ws.numel() * ws.element_size(),
                                                 _stream(stream)))


def moe_gemm_clock(handle, ws, stream=None) -> tuple:
    """(up, down) effective SM clock in MHz of the expert GEMMs run with MOE_OPTION_GEMM_CLOCK
    since the last call (0.0 when none ran); clears the sums."""
    mhz = (ctypes.c_double * 2)()
    _check("moe_gemm_clock", load_library().moe_gemm_clock(
        handle, _p(ws), ws.numel() * ws.element_size(), mhz, _stream(stream)))
    return float(mhz[0]), float(mhz[1])


# ------------------------------------------------------------------ MXFP4 matrices
def mxfp4_quantize(w, stream=None):
    """(codes [.., cols / 2], scales [.., cols / 32]), uint8, of `w` [.., cols] (fp32 or bf16,
    contiguous, cols a multiple of 32): MXFP4, one power-of-two scale for 32 neighbours.  On `stream`
    (default: the current one), which the caller orders after whatever wrote w, and which outlives the
    tensors if it was made elsewhere (ExternalStream): they are recorded on it."""
    dtype = _DTYPE_CODE.get(w.dtype)
    if dtype is None:
        raise ValueError(f"w: expected fp32 or bf16, got {w.dtype}")
    *lead, cols = w.shape or (1,)
    if cols % MXFP4_BLOCK:
        raise ValueError(f"w: the last dimension must be a multiple of {MXFP4_BLOCK}, got shape "
                         f"{tuple(w.shape)}")
    p, dev = _addr(w), w.get_device()
    with _on(dev, stream, w) as on:
        codes = on.new(w.new_empty((*lead, cols // 2), dtype=torch.uint8))
        scales = on.new(w.new_empty((*lead, cols // MXFP4_BLOCK), dtype=torch.uint8))
        if n := w.numel():
            _call_here(dev, "moe_mxfp4_quantize", p, dtype, n // cols, cols, codes.data_ptr(),
                       scales.data_ptr())
    return codes, scales


def mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, stream=None):
    """The values [.., cols] that codes [.., cols / 2] and scales [.., cols / 32] stand for, on `stream`
    as mxfp4_quantize."""
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype: expected fp32 or bf16, got {dtype}")
    *lead, half = codes.shape or (1,)
    if half % (MXFP4_BLOCK // 2):
        raise ValueError(f"codes: the last dimension must be a multiple of {MXFP4_BLOCK // 2}, "
                         f"got shape {tuple(codes.shape)}")
    cols = 2 * half
    if codes.dtype != torch.uint8:
        raise ValueError(f"codes: expected uint8, got {codes.dtype}")
    _expect(scales, (*lead, cols // MXFP4_BLOCK), torch.uint8, "scales")
    _dense(scales)
    p_codes, p_scales, dev = _addr(codes), _addr(scales), codes.get_device()
    if scales.get_device() != dev:
        raise ValueError(f"scales: on {scales.device}, codes on {codes.device}")
    with _on(dev, stream, codes, scales) as on:
        out = on.new(codes.new_empty((*lead, cols), dtype=dtype))
        if n := out.numel():
            _call_here(dev, "moe_mxfp4_dequantize", p_codes, p_scales, n // cols, cols,
                       out.data_ptr(), _DTYPE_CODE[dtype])
    return out


# ------------------------------------------------------------------ convenience wrapper
def _expect(t, shape, dtype, name):
    """The C ABI sees only pointers: a tensor of another shape or type would be read or
    written out of its bounds, so the class below checks every tensor it passes."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected shape {tuple(shape)} of {dtype}, got "
                         f"{tuple(t.shape)} of {t.dtype}")


def _expect_on(device, **tensors):
    """A layer's kernels run on one device: an address of another one means nothing there."""
    for name, t in tensors.items():
        for part in t if isinstance(t, tuple) else (t,):
            if part is not None and part.device != device:
                raise ValueError(f"{name}: on {part.device}, the layer on {device}")


class MoELayer:
    """Owns a handle and a workspace; holds references to the weight tensors.

    Calls run on `stream` (None: the current one), which the caller orders after whatever wrote
    their inputs; results, and a workspace that a call has to allocate, come from that stream's
    pool.  A stream made elsewhere (ExternalStream) outlives the tensors of its calls, which are
    recorded on it.  Calls of a layer share its workspace: on several streams the caller orders them.  A
    workspace that a captured call uses lives as long as the layer, so its graph may be replayed
    after calls of any size; the graph needs the layer to live."""

    def __init__(self, w_router, router_bias, w_gate, w_up, w_down, top_k: int,
                 max_tokens: int, n_shared: int = 1, routed_scale: float = 1.0):
        if w_router.dtype not in (torch.bfloat16, torch.float32) or w_router.dim() != 2:
            raise ValueError("w_router: expected a [E, d] bf16 or fp32 tensor")
        dt = MOE_BF16 if w_router.dtype == torch.bfloat16 else MOE_F32
        E, d = w_router.shape
        f = w_gate.shape[1]
        G = int(E) + int(n_shared)
        _expect(w_gate, (G, f, d), w_router.dtype, "w_gate")
        _expect(w_up, (G, f, d), w_router.dtype, "w_up")
        _expect(w_down, (G, d, f), w_router.dtype, "w_down")
        if router_bias is not None:
            _expect(router_bias, (E,), torch.float32, "router_bias")
        _expect_on(w_router.device, router_bias=router_bias, w_gate=w_gate, w_up=w_up,
                   w_down=w_down)
        self.cfg = moe_config(int(max_tokens), int(d), int(E), int(top_k), int(f),
                              int(n_shared), dt, float(routed_scale))
        self.tensors = (w_router, router_bias, w_gate, w_up, w_down)
        _addr(w_router)
        with _on(w_router.get_device(), None):  # the handle is of this device
            self.handle = moe_layer_init(self.cfg, *self.tensors)
        self._start(w_router)

    def _start(self, w_router):
        self.device = w_router.device
        self.dtype = w_router.dtype
        self.ws = None
        self.ws_need = {}  # bytes by number of tokens
        self.bw_ws = None
        self._ws_streams = {"ws": set(), "bw_ws": set()}  # (raw) streams that use each
        self._ws_clear = {"ws": False, "bw_ws": False}  # cleared by a call that was not captured
        self._ws_captured = {"ws": False, "bw_ws": False}  # used by a captured call
        self._kept = []  # replaced workspaces that graphs use
        self._streams = set()  # (raw) streams that read self.tensors
        self.E, self.k, self.d = (int(self.cfg.n_experts), int(self.cfg.top_k),
                                  int(self.cfg.d_model))

    def _on(self, stream, *tensors):
        return _on(self.device.index, stream, *tensors)

    def _read(self):
        """A call on the current stream reads self.tensors: a layer dropped before the call is done (it
        may hold the last reference to them) gives them back only afterwards."""
        raw = torch._C._cuda_getCurrentRawStream(self.device.index)
        if raw not in self._streams:
            self._streams.add(raw)
            here = torch.cuda.current_stream()
            for t in self.tensors:
                for part in t if isinstance(t, tuple) else (t,):
                    if part is not None:
                        part.record_stream(here)
        return raw

    def _expect(self, t, shape, dtype, name):
        _expect(t, shape, dtype, name)
        if t.get_device() != self.device.index:
            raise ValueError(f"{name}: on {t.device}, the layer on {self.device}")

    def _rows(self, x, name="x"):
        """Token count of a [T, d] activation of the layer's type."""
        if x.dim() != 2:
            raise ValueError(f"{name}: expected a [T, {self.d}] tensor, got {tuple(x.shape)}")
        self._expect(x, (x.shape[0], self.d), self.dtype, name)
        return int(x.shape[0])

    def router_logits_static(self, x, logits_out=None, stream=None):
        """Router logits [T, E] fp32 through the workspace-free entry point."""
        T = self._rows(x)
        if logits_out is not None:
            self._expect(logits_out, (T, self.E), torch.float32, "logits_out")
        with self._on(stream, x, logits_out) as on:
            if logits_out is None:
                logits_out = on.new(torch.empty((T, self.E), dtype=torch.float32,
                                                device=self.device))
            self._read()
            moe_router_logits_static(self.handle, x, T, logits_out, d_model=self.d,
                                     n_experts=self.E, dtype=self.dtype)
        return logits_out

    def set_option(self, option: int, value: int) -> None:
        moe_set_option(self.handle, option, value)

    def workspace(self, n_tokens: int, stream=None):
        """The workspace, large enough for calls of up to n_tokens tokens and ready for a call on any
        stream."""
        with self._on(stream):
            before, clear = self.ws, self._ws_clear["ws"]
            ws = self._workspace(n_tokens)
            if (ws is not before or not clear) and not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()  # it was cleared just now
        return ws

    def _workspace(self, n_tokens: int):
        need = self.ws_need.get(n_tokens)
        if need is None:
            need = self.ws_need[n_tokens] = moe_workspace_size(self.handle, n_tokens)
        return self._reserve("ws", need)

    def _reserve(self, name, need):
        """self.ws or self.bw_ws for a call on the current stream, replaced if it is smaller than need
        bytes."""
        ws, users, raw = getattr(self, name), self._ws_streams[name], self._read()
        capturing = torch.cuda.is_current_stream_capturing()
        if ws is None or ws.numel() < need:
            # The old one goes back to the pool of the stream that allocated it, once every stream
            # that used it is done (record_stream below), or never, if a graph has its address.
            if self._ws_captured[name]:
                self._kept.append(ws)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            setattr(self, name, ws)
            users.clear()
            users.add(raw)
            self._ws_clear[name] = self._ws_captured[name] = False
        elif raw not in users:
            ws.record_stream(torch.cuda.current_stream())
            users.add(raw)
        if not self._ws_clear[name]:
            # before the first call that uses it; a captured clearing only runs with its graph
            moe_workspace_init(self.handle, ws)
            self._ws_clear[name] = not capturing
        if capturing:
            self._ws_captured[name] = True
        return ws

    def forward(self, x, out=None, stream=None):
        T = self._rows(x)
        if out is not None:
            self._expect(out, x.shape, x.dtype, "out")
        with self._on(stream, x, out) as on:
            out = on.new(torch.empty_like(x)) if out is None else out
            moe_forward(self.handle, x, T, out, self._workspace(T))
        return out

    def forward_few(self, x, out=None, stream=None):
        """forward for at most 64 tokens in one launch (bf16 or MXFP4 weights; limits, and from which
        batch on a bf16 layer's forward is faster, in include/moe_layer.h)."""
        T = self._rows(x)
        if out is not None:
            self._expect(out, x.shape, x.dtype, "out")
        with self._on(stream, x, out) as on:
            out = on.new(torch.empty_like(x)) if out is None else out
            moe_forward_few(self.handle, x, T, out, self._workspace(T))
        return out

    def to_mxfp4(self, max_tokens: int | None = None) -> "MoELayerMXFP4":
        """A serving layer with this bf16 layer's router and its expert weights in MXFP4."""
        if self.dtype != torch.bfloat16:
            raise ValueError("to_mxfp4: a bf16 layer is needed")
        w_router, bias, w_gate, w_up, w_down = self.tensors
        return MoELayerMXFP4(w_router, bias, mxfp4_quantize(w_gate), mxfp4_quantize(w_up),
                             mxfp4_quantize(w_down), top_k=self.k,
                             max_tokens=max_tokens or int(self.cfg.max_tokens),
                             n_shared=int(self.cfg.n_shared),
                             routed_scale=float(self.cfg.routed_scale))

    def route(self, x=None, logits=None, want_logits=False, stream=None):
        if x is not None:
            T = self._rows(x)
        else:
            T = int(logits.shape[0])
            self._expect(logits, (T, self.E), torch.float32, "logits")
        with self._on(stream, x, logits) as on:
            def new(*shape, dtype=torch.int32):
                return on.new(torch.empty(shape, dtype=dtype, device=self.device))

            r = dict(idx=new(T, self.k), gates=new(T, self.k, dtype=torch.float32),
                     counts=new(self.E), offsets=new(self.E + 1), perm=new(T * self.k),
                     slot_row=new(T, self.k))
            ws = self._workspace(T)
            if logits is not None:
                moe_route_from_logits(self.handle, logits, T, r["idx"], r["gates"], r["counts"],
                                      r["offsets"], r["perm"], r["slot_row"], ws)
            else:
                lg = new(T, self.E, dtype=torch.float32) if want_logits else None
                moe_route(self.handle, x, T, lg, r["idx"], r["gates"], r["counts"], r["offsets"],
                          r["perm"], r["slot_row"], ws)
                if lg is not None:
                    r["logits"] = lg
        return r

    def router_stats(self, logits, topk_idx, n_groups, stream=None):
        """p_mean [E], f_sel [E] and scalars [L_EP, routing confidence] (device tensors)."""
        T = int(logits.shape[0])
        self._expect(logits, (T, self.E), torch.float32, "logits")
        self._expect(topk_idx, (T, self.k), torch.int32, "topk_idx")
        with self._on(stream, logits, topk_idx) as on:
            p_mean, f_sel, scalars = (
                on.new(torch.empty(n, dtype=torch.float32, device=self.device))
                for n in (self.E, self.E, 2))
            moe_router_stats(self.handle, logits, topk_idx, T, n_groups, p_mean, f_sel, scalars,
                             self._workspace(T))
        return p_mean, f_sel, scalars

    def forward_save(self, x, out=None, saved=None, stream=None):
        """Training forward (bf16): (out, saved) with `saved` the fp32 pre-activations that
        backward(..., saved=saved) reads instead of recomputing them."""
        T = self._rows(x)
        if out is not None:
            self._expect(out, x.shape, x.dtype, "out")
        with self._on(stream, x, out, saved) as on:
            ws = self._workspace(T)
            if out is None:
                out = on.new(torch.empty_like(x))
            if saved is None:
                saved = on.new(torch.empty(moe_saved_size(self.handle, T) // 4,
                                           dtype=torch.float32, device=self.device))
            moe_forward_save(self.handle, x, T, out, saved, ws)
        return out, saved

    def backward(self, x, dout, stream=None, grads=None, saved=None, overwrite=False):
        """dict of fp32 gradients dx, dw_router, dw_gate, dw_up, dw_down (device tensors); the
        weight gradients are added to `grads`' tensors when given (new zeroed ones if not),
        or set when `overwrite`.  With `saved` (from forward_save of the same x) the
        pre-activations are not recomputed."""
        T = self._rows(x)
        self._expect(dout, x.shape, x.dtype, "dout")
        with self._on(stream, x, dout, saved, *(grads or {}).values()) as on:
            g = self._backward(x, T, dout, grads, saved, overwrite)
            for name in g:
                if grads is None or name == "dx":
                    on.new(g[name])
        return g

    def _backward(self, x, T, dout, grads, saved, overwrite):
        bw_ws = self._reserve("bw_ws", moe_backward_workspace_size(self.handle, T))
        G = self.E + int(self.cfg.n_shared)
        f = int(self.cfg.d_ff)
        kw = dict(dtype=torch.float32, device=self.device)
        if grads is not None:
            g = dict(grads)
            g["dx"] = torch.empty((T, self.d), **kw)
        elif overwrite:  # every element is written
            g = dict(dx=torch.empty((T, self.d), **kw),
                     dw_router=torch.empty((self.E, self.d), **kw),
                     dw_gate=torch.empty((G, f, self.d), **kw),
                     dw_up=torch.empty((G, f, self.d), **kw),
                     dw_down=torch.empty((G, self.d, f), **kw))
        else:  # the weight gradients accumulate: start them at zero
            g = dict(dx=torch.empty((T, self.d), **kw),
                     dw_router=torch.zeros((self.E, self.d), **kw),
                     dw_gate=torch.zeros((G, f, self.d), **kw),
                     dw_up=torch.zeros((G, f, self.d), **kw),
                     dw_down=torch.zeros((G, self.d, f), **kw))
        for name, shape in (("dw_router", (self.E, self.d)), ("dw_gate", (G, f, self.d)),
                            ("dw_up", (G, f, self.d)), ("dw_down", (G, self.d, f))):
            self._expect(g[name], shape, torch.float32, name)
        if overwrite:
            moe_backward_ex(self.handle, x, T, dout, saved, MOE_BACKWARD_OVERWRITE, g["dx"],
                            g["dw_router"], g["dw_gate"], g["dw_up"], g["dw_down"], bw_ws)
        elif saved is not None:
            moe_backward_saved(self.handle, x, T, dout, saved, g["dx"], g["dw_router"],
                               g["dw_gate"], g["dw_up"], g["dw_down"], bw_ws)
        else:
            moe_backward(self.handle, x, T, dout, g["dx"], g["dw_router"], g["dw_gate"],
                         g["dw_up"], g["dw_down"], bw_ws)
        return g

    def expert_health(self, n_tokens, stream=None):
        """act_rms [G], param_norm [G], ratios [2] of the last forward of n_tokens tokens."""
        G = self.E + int(self.cfg.n_shared)
        with self._on(stream) as on:
            act, par, ratios = (on.new(torch.empty(n, dtype=torch.float32, device=self.device))
                                for n in (G, G, 2))
            moe_expert_health(self.handle, n_tokens, act, par, ratios, self._workspace(n_tokens))
        return act, par, ratios

    def gemm_clock_mhz(self, stream=None) -> tuple:
        """(up, down) effective SM clock of the forward's expert GEMMs since the last call, for
        forwards run with MOE_OPTION_GEMM_CLOCK set (see moe_gemm_clock)."""
        with self._on(stream):
            return moe_gemm_clock(self.handle, self.ws)

    def device_status(self, stream=None) -> int:
        """Device status of the forward's and the backward's workspaces (0: no bounded wait
        gave up in either)."""
        st = 0
        with self._on(stream):
            for ws in (self.ws, self.bw_ws):
                if ws is not None:
                    st = st or moe_device_status(self.handle, ws)
        return st

    def close(self):
        if self.handle is not None:
            moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MoELayerMXFP4(MoELayer):
    """MoELayer over MXFP4 expert weights, for serving: w_gate, w_up [E + n_shared, f, d] and
    w_down [E + n_shared, d, f] are (codes, scales) as mxfp4_quantize returns them; the router and
    the activations are bf16.  forward, forward_few, route and router_stats as in MoELayer; training
    calls and expert_health are refused by the library (MoEError).

    The layer reads the caller's codes in place, but a copy of the scales, tiled once when it is
    made.  Weights written anew into the same tensors would change the one and not the other: other
    weights need another layer.  Codes start on a 32-byte boundary."""

    def __init__(self, w_router, router_bias, w_gate, w_up, w_down, top_k: int,
                 max_tokens: int, n_shared: int = 1, routed_scale: float = 1.0):
        if w_router.dtype != torch.bfloat16 or w_router.dim() != 2:
            raise ValueError("w_router: expected a [E, d] bf16 tensor")
        E, d = w_router.shape
        G = int(E) + int(n_shared)
        if len(w_gate) != 2 or w_gate[0].dim() != 3:
            raise ValueError("w_gate: expected (codes [G, f, d / 2], scales [G, f, d / 32])")
        f = int(w_gate[0].shape[1])
        for name, w, rows, cols in (("w_gate", w_gate, f, d), ("w_up", w_up, f, d),
                                    ("w_down", w_down, d, f)):
            codes, scales = w
            _expect(codes, (G, rows, cols // 2), torch.uint8, f"{name} codes")
            _expect(scales, (G, rows, cols // MXFP4_BLOCK), torch.uint8, f"{name} scales")
        if router_bias is not None:
            _expect(router_bias, (E,), torch.float32, "router_bias")
        self.cfg = moe_config(int(max_tokens), int(d), int(E), int(top_k), int(f),
                              int(n_shared), MOE_BF16, float(routed_scale))
        self.handle = None
        _expect_on(w_router.device, router_bias=router_bias, w_gate=tuple(w_gate),
                   w_up=tuple(w_up), w_down=tuple(w_down))
        tiled = []
        _addr(w_router)
        with _on(w_router.get_device(), None):
            for codes, scales in (w_gate, w_up, w_down):
                t = torch.empty_like(scales)
                moe_mxfp4_tile_scales(scales, t)
                tiled.append((codes, t))
            torch.cuda.current_stream().synchronize()  # calls may come on any stream
            self.tensors = (w_router, router_bias, *tiled)
            self.handle = moe_layer_init_mxfp4(self.cfg, *self.tensors)
        self._start(w_router)

    def to_mxfp4(self, max_tokens: int | None = None):
        raise ValueError("to_mxfp4: the layer holds MXFP4 weights already")
