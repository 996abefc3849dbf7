"""Quantized recurrent-state decode step for B200 (sm_100a): Python binding.

A thin ctypes layer over the C ABI of ``librsq.so`` (declared in include/rsq.h).
The functions keep the C names (``rsq_create``, ``rsq_decode_step``, ...) and
only marshal arguments: tensors become device pointers, streams become
``cudaStream_t`` handles.  Every step of the decode path runs in the library's
CUDA kernels; there is no fallback, and importing this package on a machine
where the library cannot be loaded raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import sys

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librsq.so")

RSQ_GDN, RSQ_MAMBA2, RSQ_GLA, RSQ_KDA = 0, 1, 2, 3
RSQ_RTN, RSQ_SR, RSQ_BDR, RSQ_SR_BDR = 0, 1, 2, 3
RSQ_SR8, RSQ_SR8_BDR = 5, 7   # stochastic rounding with 8-bit uniforms (RSQ_SR: 16-bit)
RSQ_F32, RSQ_BF16 = 0, 1
RSQ_NORM_GATE, RSQ_GATE_NORM = 0, 1
RSQ_OK, RSQ_E_INVAL, RSQ_E_UNSUPPORTED, RSQ_E_CUDA, RSQ_E_NOMEM, RSQ_E_NONFINITE = range(6)
RSQ_MAX_HEADS = 512


class RsqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("rsq status %d (%s): %s" % (status, _status_name(status), message))
        self.status = status


rsq_alloc_fn = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
rsq_release_fn = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p)


class rsq_config(ctypes.Structure):
    _fields_ = [("family", ctypes.c_int), ("batch", ctypes.c_int), ("heads", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("ngroups", ctypes.c_int),
                ("head_bits", ctypes.POINTER(ctypes.c_int8)), ("rounding", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("seed", ctypes.c_uint64), ("window", ctypes.c_int),
                ("key_axis", ctypes.c_int), ("alloc", rsq_alloc_fn), ("release", rsq_release_fn),
                ("alloc_user", ctypes.c_void_p)]


class rsq_state(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class rsq_gdn_inputs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class rsq_mamba2_inputs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("Bm", ctypes.c_void_p), ("Cm", ctypes.c_void_p),
                ("dt", ctypes.c_void_p), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("decay", ctypes.c_void_p)]


class rsq_window(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("a_scale", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("b_scale", ctypes.c_void_p)]


class rsq_diag_inputs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class rsq_scan_config(ctypes.Structure):
    _fields_ = [("family", ctypes.c_int), ("in_dtype", ctypes.c_int), ("sequences", ctypes.c_int),
                ("heads", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("ngroups", ctypes.c_int), ("ragged", ctypes.c_int), ("tokens", ctypes.c_int64)]


class rsq_scan_inputs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("Bm", ctypes.c_void_p), ("Cm", ctypes.c_void_p),
                ("dt", ctypes.c_void_p), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("decay", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64)]


class rsq_scan_grads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dBm", ctypes.c_void_p), ("dCm", ctypes.c_void_p),
                ("ddt", ctypes.c_void_p), ("dlog_decay", ctypes.c_void_p), ("dA", ctypes.c_void_p),
                ("dD", ctypes.c_void_p), ("dstate_in", ctypes.c_void_p)]


class rsq_norm_config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int), ("group", ctypes.c_int),
                ("order", ctypes.c_int), ("x_dtype", ctypes.c_int), ("side_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("side_stride", ctypes.c_int64)]


_EXPORTS = ["rsq_create", "rsq_destroy", "rsq_state_bytes", "rsq_head_offset", "rsq_decode_step",
            "rsq_quantize", "rsq_dequantize", "rsq_state_drift", "rsq_check_flags",
            "rsq_allocate_bits", "rsq_reduction_partials", "rsq_status_string", "rsq_last_error",
            "rsq_version", "rsq_decode_step_noalloc", "rsq_decode_step_copy_scale",
            "rsq_column_absmax", "rsq_window_bytes", "rsq_decode_step_window", "rsq_debug_waits",
            "rsq_scan_workspace", "rsq_scan", "rsq_scan_backward", "rsq_scan_check", "rsq_norm_workspace",
            "rsq_gated_norm", "rsq_gated_norm_backward", "rsq_residual_norm",
            "rsq_residual_norm_backward"]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("librsq.so not built (run python -m ssm_decode_02_b200.build): %s" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, C = ctypes.c_void_p, ctypes.c_int
    sig = {
        "rsq_create": ([ctypes.POINTER(rsq_config), ctypes.POINTER(P)], C),
        "rsq_destroy": ([P], None),
        "rsq_state_bytes": ([P, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_head_offset": ([P, C, ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_decode_step": ([P, ctypes.POINTER(rsq_state), ctypes.POINTER(rsq_state), P, P,
                             ctypes.c_uint32, P], C),
        "rsq_quantize": ([P, P, ctypes.POINTER(rsq_state), ctypes.c_uint32, P], C),
        "rsq_dequantize": ([P, ctypes.POINTER(rsq_state), P, P], C),
        "rsq_state_drift": ([P, ctypes.POINTER(rsq_state), P, ctypes.POINTER(rsq_state), P, P], C),
        "rsq_check_flags": ([P, ctypes.POINTER(C), P], C),
        "rsq_allocate_bits": ([P, C, C, C, C, P], C),
        "rsq_reduction_partials": ([C], C),
        "rsq_status_string": ([C], ctypes.c_char_p),
        "rsq_last_error": ([], ctypes.c_char_p),
        "rsq_version": ([], ctypes.c_char_p),
        "rsq_decode_step_noalloc": ([ctypes.POINTER(rsq_config), ctypes.POINTER(rsq_state),
                                     ctypes.POINTER(rsq_state), P, P, ctypes.c_uint32, P], C),
        "rsq_decode_step_copy_scale": ([P, ctypes.POINTER(rsq_state), ctypes.POINTER(rsq_state), P, P,
                                        P, ctypes.c_uint32, P], C),
        "rsq_column_absmax": ([P, ctypes.POINTER(rsq_state), P, P], C),
        "rsq_window_bytes": ([P, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                              ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_decode_step_window": ([P, ctypes.POINTER(rsq_state), ctypes.POINTER(rsq_state),
                                    ctypes.POINTER(rsq_window), ctypes.POINTER(rsq_window), P, P,
                                    ctypes.c_uint32, P], C),
        "rsq_host_input_layout": ([P, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                                   ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_pipe_create": ([P, ctypes.POINTER(P)], C),
        "rsq_pipe_destroy": ([P], None),
        "rsq_pipe_step": ([P, ctypes.POINTER(rsq_state), ctypes.POINTER(rsq_state), ctypes.POINTER(rsq_window),
                           ctypes.POINTER(rsq_window), P, P, ctypes.c_uint32], C),
        "rsq_pipe_sync": ([P], C),
        "rsq_pipe_streams": ([P, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P)], C),
        "rsq_debug_waits": ([P, ctypes.c_uint32, C], C),
        "rsq_scan_workspace": ([ctypes.POINTER(rsq_scan_config), C, ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_scan": ([ctypes.POINTER(rsq_scan_config), ctypes.POINTER(rsq_scan_inputs), P, P, P, P, P,
                      ctypes.c_size_t, P], C),
        "rsq_scan_backward": ([ctypes.POINTER(rsq_scan_config), ctypes.POINTER(rsq_scan_inputs), P, P, P, P,
                               ctypes.POINTER(rsq_scan_grads), P, ctypes.c_size_t, P], C),
        "rsq_scan_check": ([P, P], C),
        "rsq_norm_workspace": ([ctypes.POINTER(rsq_norm_config), ctypes.POINTER(ctypes.c_size_t)], C),
        "rsq_gated_norm": ([ctypes.POINTER(rsq_norm_config)] + [P] * 5, C),
        "rsq_gated_norm_backward": ([ctypes.POINTER(rsq_norm_config)] + [P] * 8 + [ctypes.c_size_t, P], C),
        "rsq_residual_norm": ([ctypes.POINTER(rsq_norm_config)] + [P] * 7, C),
        "rsq_residual_norm_backward": ([ctypes.POINTER(rsq_norm_config)] + [P] * 11 + [ctypes.c_size_t, P], C),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


lib = _load()


def _status_name(s: int) -> str:
    return lib.rsq_status_string(int(s)).decode()


def _check(status: int) -> int:
    if status != RSQ_OK:
        raise RsqError(status, lib.rsq_last_error().decode())
    return status


def _ptr(t) -> int | None:
    """Host address of a numpy array (host arguments); ints pass through; None stays None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return int(t.ctypes.data)
    if hasattr(t, "data_ptr"):
        return int(t.data_ptr())
    raise TypeError("cannot take the address of %r" % type(t))


def _dptr(t) -> int | None:
    """Device address of a CUDA tensor argument; a CPU or non-contiguous tensor is
    refused here instead of reaching the kernel.  Ints (raw device addresses) pass
    through; None stays None."""
    if t is None or isinstance(t, int):
        return t
    if not hasattr(t, "data_ptr"):
        raise TypeError("expected a CUDA tensor, got %r" % type(t))
    if not getattr(t, "is_cuda", False):
        raise ValueError("expected a CUDA tensor, got one on %s" % getattr(t, "device", "the host"))
    if not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return int(t.data_ptr())


def _workspace(t) -> tuple[int | None, int]:
    if t is None:
        return None, 0
    return _arg(t, 0, None, _current_device(), "workspace"), t.numel() * t.element_size()


def _current_device() -> int | None:
    """torch's current device; None before it has one, when no argument can be a tensor on it."""
    global _current_device
    torch = sys.modules.get("torch")
    if torch is None or not torch.cuda.is_initialized():
        return None
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


_torch_types = None


def _types() -> dict:
    """torch dtypes by rsq_dtype; int32 by its name.  None before torch is loaded."""
    global _torch_types
    if _torch_types is None:
        torch = sys.modules.get("torch")
        if torch is None:
            return dict.fromkeys((RSQ_F32, RSQ_BF16, "int32"))
        _torch_types = {RSQ_F32: torch.float32, RSQ_BF16: torch.bfloat16, "int32": torch.int32}
    return _torch_types


def _refuse(t, count: int, want, name: str) -> None:
    """Says what is wrong with an argument that _arg does not take."""
    if not hasattr(t, "data_ptr"):
        raise TypeError("%s: expected a CUDA tensor, got %r" % (name, type(t)))
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor, got one on %s" % (name, t.device))
    if t.numel() < count or (want is not None and t.dtype is not want):
        raise ValueError("%s: expected at least %d elements of %s, got %s of %s" % (name, count, want, tuple(t.shape), t.dtype))
    raise ValueError("%s is on cuda:%d, the current device is cuda:%s" % (name, t.get_device(), _current_device()))


def _fits(t, count: int, want, here, name: str) -> None:
    """Refuses a tensor of fewer than count elements, of another type than want (None: the
    library's to refuse) or of another GPU than `here`, whose stream the call uses: the kernels
    take sizes and types from the configuration alone, and read float16 bits as bfloat16.
    Addresses pass."""
    if t is None or isinstance(t, int):
        return
    try:
        if t.numel() >= count and (t.dtype is want or want is None) and t.get_device() == here:
            return
    except AttributeError:
        pass
    _refuse(t, count, want, name)


def _arg(t, count: int, want, here, name: str) -> int | None:
    """_fits, and the address of a contiguous tensor."""
    if t is None or isinstance(t, int):
        return t
    try:
        if t.numel() >= count and (t.dtype is want or want is None) and t.get_device() == here and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _dptr(t)
    _refuse(t, count, want, name)
    return p


def _arg_rows(t, rows: int, width: int, stride: int, want, here, name: str) -> int | None:
    """As _arg, for rows that may lie apart: as `stride` (0: packed) says, since the kernels go by
    the configuration, whichever tensors it was made from."""
    if t is None or isinstance(t, int):
        return t
    stride = stride or width
    try:
        if stride == width and t.is_contiguous():
            return _arg(t, rows * width, want, here, name)
        if (t.dim() == 2 and t.stride(0) == stride and t.stride(1) == 1 and t.shape[0] >= rows and t.shape[1] >= width
                and (t.dtype is want or want is None) and t.get_device() == here):
            return t.data_ptr()
    except AttributeError:
        pass
    _fits(t, rows * width, want, here, name)
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s: expected a contiguous last dimension" % name)
    if rows < 2 and t.is_contiguous():
        return t.data_ptr()
    inner = 1
    for d in range(t.dim() - 1, 0, -1):     # the columns of a row, as far as they are packed
        if t.shape[d] > 1 and t.stride(d) != inner:
            break
        inner *= t.shape[d]
    else:
        if t.dim() > 1 and inner >= width and (rows < 2 or (t.stride(0) == stride and t.shape[0] >= rows)):
            return t.data_ptr()
    raise ValueError("%s: the configuration has %d rows of %d columns, %d elements apart; got shape %s with strides %s"
                     % (name, rows, width, stride, tuple(t.shape), tuple(t.stride())))


def _dtype_of(t) -> int:
    """rsq_dtype of a tensor or a torch dtype."""
    import torch
    d = t if isinstance(t, torch.dtype) else t.dtype
    if d == torch.float32:
        return RSQ_F32
    if d == torch.bfloat16:
        return RSQ_BF16
    raise ValueError("expected float32 or bfloat16, got %s" % d)


def _hptr(t) -> int:
    """Host address of a host buffer argument (numpy array or CPU tensor); a CUDA
    tensor is refused here."""
    if getattr(t, "is_cuda", False):
        raise ValueError("expected a host buffer, got a CUDA tensor")
    if isinstance(t, np.ndarray) and not t.flags.c_contiguous:
        raise ValueError("expected a contiguous host buffer")
    if hasattr(t, "is_contiguous") and not t.is_contiguous():
        raise ValueError("expected a contiguous host buffer")
    p = _ptr(t)
    if not p:
        raise ValueError("null host buffer")
    return p


_raw_stream = None


def _stream(stream) -> int | None:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            # the handle alone: torch.cuda.current_stream() builds an object around it, 3 us a call
            _raw_stream = ((lambda: get(torch._C._cuda_getDevice())) if get and torch.cuda.is_initialized()
                           else (lambda: int(torch.cuda.current_stream().cuda_stream)))
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ---------------------------------------------------------------------------
# C functions under their own names (argument marshalling only)
# ---------------------------------------------------------------------------
def rsq_create(family: int, batch: int, heads: int, dk: int, dv: int, *, head_bits=None,
               rounding: int = RSQ_SR8, in_dtype: int = RSQ_BF16, seed: int = 0,
               ngroups: int = 1, window: int = 0, key_axis: int = 0, alloc=None, release=None) -> int:
    """``alloc`` / ``release``: rsq_alloc_fn / rsq_release_fn objects (the
    allocator hook; the caller keeps them alive as long as the context)."""
    cfg, bits_arr = _config(family, batch, heads, dk, dv, head_bits, rounding, in_dtype, seed, ngroups,
                            window, key_axis)
    if alloc is not None:
        cfg.alloc = alloc
    if release is not None:
        cfg.release = release
    out = ctypes.c_void_p()
    _check(lib.rsq_create(ctypes.byref(cfg), ctypes.byref(out)))
    return int(out.value)


def _config(family, batch, heads, dk, dv, head_bits, rounding, in_dtype, seed, ngroups, window=0,
            key_axis=0):
    bits_arr = None
    if head_bits is not None:
        bits_arr = (ctypes.c_int8 * heads)(*[int(b) for b in head_bits])
    cfg = rsq_config(int(family), int(batch), int(heads), int(dk), int(dv), int(ngroups),
                     ctypes.cast(bits_arr, ctypes.POINTER(ctypes.c_int8)) if bits_arr else None,
                     int(rounding), int(in_dtype), int(seed) & (2 ** 64 - 1), int(window),
                     int(key_axis))
    return cfg, bits_arr


def rsq_decode_step_noalloc(family: int, batch: int, heads: int, dk: int, dv: int, state_in,
                            state_out, inputs, out, step: int, *, head_bits=None,
                            rounding: int = RSQ_SR8, in_dtype: int = RSQ_BF16, seed: int = 0,
                            ngroups: int = 1, stream=None) -> None:
    """Decode step without a context and without any device allocation (the
    kernel's flag word lives in a static device array; see include/rsq.h)."""
    cfg, keep = _config(family, batch, heads, dk, dv, head_bits, rounding, in_dtype, seed, ngroups)
    si, so = _state(state_in), _state(state_out)
    _check(lib.rsq_decode_step_noalloc(ctypes.byref(cfg), ctypes.byref(si), ctypes.byref(so),
                                       ctypes.byref(inputs), _dptr(out), int(step) & 0xFFFFFFFF,
                                       _stream(stream)))
    del keep


def rsq_destroy(ctx: int) -> None:
    lib.rsq_destroy(ctx)


def rsq_state_bytes(ctx: int) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.rsq_state_bytes(ctx, ctypes.byref(a), ctypes.byref(b)))
    return int(a.value), int(b.value)


def rsq_head_offset(ctx: int, h: int) -> int:
    o = ctypes.c_size_t()
    _check(lib.rsq_head_offset(ctx, int(h), ctypes.byref(o)))
    return int(o.value)


def _state(st) -> rsq_state:
    return rsq_state(_dptr(st.codes), _dptr(st.scales))


def rsq_decode_step(ctx: int, state_in, state_out, inputs, out, step: int, stream=None) -> None:
    """inputs: rsq_gdn_inputs / rsq_mamba2_inputs / rsq_diag_inputs (see gdn_inputs,
    mamba2_inputs, diag_inputs)."""
    si, so = _state(state_in), _state(state_out)
    _check(lib.rsq_decode_step(ctx, ctypes.byref(si), ctypes.byref(so), ctypes.byref(inputs),
                               _dptr(out), int(step) & 0xFFFFFFFF, _stream(stream)))


def rsq_decode_step_copy_scale(ctx: int, state_in, state_out, inputs, copy_absmax, out, step: int,
                               stream=None) -> None:
    """Decode step whose scales come from copy_absmax ([B][H][dv], column maxima of an
    unquantized copy of the state) instead of the state's own columns."""
    si, so = _state(state_in), _state(state_out)
    _check(lib.rsq_decode_step_copy_scale(ctx, ctypes.byref(si), ctypes.byref(so), ctypes.byref(inputs),
                                          _dptr(copy_absmax), _dptr(out), int(step) & 0xFFFFFFFF,
                                          _stream(stream)))


def rsq_column_absmax(ctx: int, state, absmax, stream=None) -> None:
    """Column maxima of |S^| of a stored state into absmax ([B][H][dv] float32, device)."""
    si = _state(state)
    _check(lib.rsq_column_absmax(ctx, ctypes.byref(si), _dptr(absmax), _stream(stream)))


def rsq_window_bytes(ctx: int) -> tuple[int, int, int]:
    a, b, sc = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.rsq_window_bytes(ctx, ctypes.byref(a), ctypes.byref(b), ctypes.byref(sc)))
    return int(a.value), int(b.value), int(sc.value)


def _window(win) -> rsq_window:
    return rsq_window(_dptr(win.a), _dptr(win.a_scale), _dptr(win.b), _dptr(win.b_scale))


def rsq_decode_step_window(ctx: int, state_in, state_out, win_in, win_out, inputs, out, step: int,
                           stream=None) -> None:
    si, so = _state(state_in), _state(state_out)
    wi, wo = _window(win_in), _window(win_out)
    _check(lib.rsq_decode_step_window(ctx, ctypes.byref(si), ctypes.byref(so), ctypes.byref(wi),
                                      ctypes.byref(wo), ctypes.byref(inputs), _dptr(out),
                                      int(step) & 0xFFFFFFFF, _stream(stream)))


def rsq_host_input_layout(ctx: int) -> tuple[list[int], list[int], int]:
    """(offsets, sizes, total) of the packed host input buffer of one step."""
    off = (ctypes.c_size_t * 6)()
    size = (ctypes.c_size_t * 6)()
    total = ctypes.c_size_t()
    _check(lib.rsq_host_input_layout(ctx, off, size, ctypes.byref(total)))
    return list(off), list(size), int(total.value)


def rsq_pipe_create(ctx: int) -> int:
    out = ctypes.c_void_p()
    _check(lib.rsq_pipe_create(ctx, ctypes.byref(out)))
    return int(out.value)


def rsq_pipe_destroy(pipe: int) -> None:
    lib.rsq_pipe_destroy(pipe)


def rsq_pipe_step(pipe: int, state_in, state_out, host_inputs, host_out, step: int, win_in=None,
                  win_out=None) -> None:
    """host_inputs: the packed host buffer (pack_host_inputs); host_out: host float [B][H][dv]."""
    si, so = _state(state_in), _state(state_out)
    wi = ctypes.byref(_window(win_in)) if win_in is not None else None
    wo = ctypes.byref(_window(win_out)) if win_out is not None else None
    _check(lib.rsq_pipe_step(pipe, ctypes.byref(si), ctypes.byref(so), wi, wo, _hptr(host_inputs),
                             _hptr(host_out), int(step) & 0xFFFFFFFF))


def rsq_pipe_sync(pipe: int) -> None:
    _check(lib.rsq_pipe_sync(pipe))


def rsq_pipe_streams(pipe: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib.rsq_pipe_streams(pipe, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return int(a.value), int(b.value), int(c.value)


def rsq_quantize(ctx: int, S, state_out, step: int, stream=None) -> None:
    so = _state(state_out)
    _check(lib.rsq_quantize(ctx, _dptr(S), ctypes.byref(so), int(step) & 0xFFFFFFFF, _stream(stream)))


def rsq_dequantize(ctx: int, state_in, S_out, stream=None) -> None:
    si = _state(state_in)
    _check(lib.rsq_dequantize(ctx, ctypes.byref(si), _dptr(S_out), _stream(stream)))


def rsq_state_drift(q_ctx: int, q_state, f_ctx: int, f_state, sums, stream=None) -> None:
    a, b = _state(q_state), _state(f_state)
    _check(lib.rsq_state_drift(q_ctx, ctypes.byref(a), f_ctx, ctypes.byref(b), _dptr(sums),
                               _stream(stream)))


def rsq_check_flags(ctx: int, stream=None) -> int:
    """Returns 1 if a non-finite column was seen since the last check (and clears it)."""
    seen = ctypes.c_int(0)
    st = lib.rsq_check_flags(ctx, ctypes.byref(seen), _stream(stream))
    if st not in (RSQ_OK, RSQ_E_NONFINITE):
        _check(st)
    return int(seen.value)


def rsq_debug_waits(ctx: int, wait_iters: int, withhold: int) -> None:
    """Failure-detection tests: limit the kernels' bounded waits and withhold an
    exchange-barrier arrival (see rsq.h)."""
    _check(lib.rsq_debug_waits(ctx, int(wait_iters), int(withhold)))


def rsq_allocate_bits(score, n_high: int, high_bits: int = 8, low_bits: int = 4) -> np.ndarray:
    s = np.ascontiguousarray(score, dtype=np.float64)
    out = np.zeros(s.shape[0], dtype=np.int8)
    _check(lib.rsq_allocate_bits(_ptr(s), s.shape[0], int(n_high), int(high_bits), int(low_bits),
                                 _ptr(out)))
    return out


def rsq_reduction_partials(dk: int) -> int:
    return int(lib.rsq_reduction_partials(int(dk)))


def rsq_scan_workspace(cfg: rsq_scan_config, backward: bool = False) -> int:
    n = ctypes.c_size_t()
    _check(lib.rsq_scan_workspace(ctypes.byref(cfg), int(backward), ctypes.byref(n)))
    return int(n.value)


def _scan_args(c, inputs, out, cu_seqlens, states, grads=None) -> list:
    """Checks the tensors behind a call's arguments, whose sizes, types and device the kernels
    take from the configuration; the addresses of cu_seqlens, the states and out."""
    types, here = _types(), _current_device()
    f32, bf16 = types[RSQ_F32], types[RSQ_BF16]
    tokens, gates = c.tokens, c.tokens * c.heads
    x_row, b_row = c.heads * c.dv, c.ngroups * c.dk
    x, Bm, Cm, dt, A, D, decay = getattr(inputs, "tensors", (None,) * 7)
    for name, t, row in (("x", x, x_row), ("Bm", Bm, b_row), ("Cm", Cm, b_row)):
        if t is not None and not isinstance(t, int):
            _fits(t, tokens * row, bf16, here, name)
            if t.numel() != t.shape[0] * row:
                raise ValueError("%s: expected %d elements a token, got %s" % (name, row, tuple(t.shape)))
    rest = [("dt", dt, gates, f32), ("decay", decay, gates, f32), ("A", A, c.heads, f32), ("D", D, c.heads, f32)]
    state = c.sequences * x_row * c.dk
    if grads is not None:
        dx, dBm, dCm, ddt, dlog, dA, dD, dstate = getattr(grads, "tensors", (None,) * 8)
        rest += [("dx", dx, tokens * x_row, bf16), ("dBm", dBm, tokens * b_row, bf16), ("dCm", dCm, tokens * b_row, bf16),
                 ("ddt", ddt, gates, f32), ("dlog_decay", dlog, gates, f32), ("dA", dA, c.heads, f32), ("dD", dD, c.heads, f32),
                 ("dstate_in", dstate, state, f32)]
    for name, t, count, want in rest:
        if t is not None:
            _fits(t, count, want, here, name)
    return [_arg(cu_seqlens, c.sequences + 1, types["int32"], here, "cu_seqlens"), _arg(states[0], state, f32, here, "state_in"),
            _arg(states[1], state, f32, here, "the second state"), _arg(out, tokens * x_row, bf16, here, "out or dout")]


def rsq_scan(cfg: rsq_scan_config, inputs: rsq_scan_inputs, out, *, cu_seqlens=None, state_in=None,
             state_out=None, workspace=None, stream=None) -> None:
    cu, first, last, to = _scan_args(cfg, inputs, out, cu_seqlens, (state_in, state_out))
    ws, n = _workspace(workspace)
    _check(lib.rsq_scan(ctypes.byref(cfg), ctypes.byref(inputs), cu, first, last, to, ws, n, _stream(stream)))


def rsq_scan_backward(cfg: rsq_scan_config, inputs: rsq_scan_inputs, dout, grads: rsq_scan_grads, *,
                      cu_seqlens=None, state_in=None, dstate_out=None, workspace=None, stream=None) -> None:
    cu, first, last, given = _scan_args(cfg, inputs, dout, cu_seqlens, (state_in, dstate_out), grads)
    ws, n = _workspace(workspace)
    _check(lib.rsq_scan_backward(ctypes.byref(cfg), ctypes.byref(inputs), cu, first, given, last, ctypes.byref(grads), ws, n,
                                 _stream(stream)))


def rsq_scan_check(workspace, stream=None) -> None:
    """Raises when a kernel of the last call with this workspace gave up a wait.  None, the
    workspace of calls that need none: nothing waits."""
    if workspace is None:
        return
    _check(lib.rsq_scan_check(_dptr(workspace), _stream(stream)))


def rsq_norm_workspace(cfg: rsq_norm_config) -> int:
    n = ctypes.c_size_t()
    _check(lib.rsq_norm_workspace(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def rsq_gated_norm(cfg: rsq_norm_config, x, z, w, y, stream=None) -> None:
    """x and z may be row-strided, as the configuration says (norm_config reads their strides)."""
    types, here, rows, width = _types(), _current_device(), cfg.rows, cfg.width
    args = (_arg_rows(x, rows, width, cfg.x_stride, types.get(cfg.x_dtype), here, "x"),
            _arg_rows(z, rows, width, cfg.side_stride, types.get(cfg.side_dtype), here, "z"),
            _arg(w, width, types[RSQ_F32], here, "w"), _arg(y, rows * width, types.get(cfg.y_dtype), here, "y"))
    _check(lib.rsq_gated_norm(ctypes.byref(cfg), *args, _stream(stream)))


def rsq_gated_norm_backward(cfg: rsq_norm_config, x, z, w, dy, dx, dz, dw, workspace=None, stream=None) -> None:
    types, here, rows, width = _types(), _current_device(), cfg.rows, cfg.width
    n, tx, ts, f32 = rows * width, types.get(cfg.x_dtype), types.get(cfg.side_dtype), types[RSQ_F32]
    ws, ws_bytes = _workspace(workspace)
    args = (_arg_rows(x, rows, width, cfg.x_stride, tx, here, "x"), _arg_rows(z, rows, width, cfg.side_stride, ts, here, "z"),
            _arg(w, width, f32, here, "w"), _arg(dy, n, types.get(cfg.y_dtype), here, "dy"), _arg(dx, n, tx, here, "dx"),
            _arg(dz, n, ts, here, "dz"), _arg(dw, width, f32, here, "dw"), ws, ws_bytes)
    _check(lib.rsq_gated_norm_backward(ctypes.byref(cfg), *args, _stream(stream)))


def rsq_residual_norm(cfg: rsq_norm_config, x, residual, scale, w, h, y, stream=None) -> None:
    """x and residual may be row-strided, as the configuration says (norm_config reads their strides)."""
    types, here, rows, width = _types(), _current_device(), cfg.rows, cfg.width
    n, ts, f32 = rows * width, types.get(cfg.side_dtype), types[RSQ_F32]
    args = (_arg_rows(x, rows, width, cfg.x_stride, types.get(cfg.x_dtype), here, "x"),
            _arg_rows(residual, rows, width, cfg.side_stride, ts, here, "residual"), _arg(scale, width, f32, here, "scale"),
            _arg(w, width, f32, here, "w"), _arg(h, n, ts, here, "h"), _arg(y, n, types.get(cfg.y_dtype), here, "y"))
    _check(lib.rsq_residual_norm(ctypes.byref(cfg), *args, _stream(stream)))


def rsq_residual_norm_backward(cfg: rsq_norm_config, x, h, scale, w, dy, dh, dx, dresidual, dscale, dw,
                               workspace=None, stream=None) -> None:
    types, here, rows, width = _types(), _current_device(), cfg.rows, cfg.width
    n, tx, ts, f32 = rows * width, types.get(cfg.x_dtype), types.get(cfg.side_dtype), types[RSQ_F32]
    ws, ws_bytes = _workspace(workspace)
    args = (_arg_rows(x, rows, width, cfg.x_stride, tx, here, "x"), _arg(h, n, ts, here, "h"), _arg(scale, width, f32, here, "scale"),
            _arg(w, width, f32, here, "w"), _arg(dy, n, types.get(cfg.y_dtype), here, "dy"), _arg(dh, n, ts, here, "dh"),
            _arg(dx, n, tx, here, "dx"), _arg(dresidual, n, ts, here, "dresidual"), _arg(dscale, width, f32, here, "dscale"),
            _arg(dw, width, f32, here, "dw"), ws, ws_bytes)
    _check(lib.rsq_residual_norm_backward(ctypes.byref(cfg), *args, _stream(stream)))


def rsq_version() -> str:
    return lib.rsq_version().decode()


# ---------------------------------------------------------------------------
# Convenience containers (torch tensors for device memory)
# ---------------------------------------------------------------------------
class State:
    """A stored state: codes uint8 [B][row_bytes] and scales float32 [B][H][dv] (device)."""

    def __init__(self, codes, scales):
        self.codes = codes
        self.scales = scales


class Window:
    """A pure-write window (device): a uint8 [B][H][W][dk], a_scale float [B][H][W],
    b uint8 [B][H][dv/16][W][16], b_scale float [B][H][W]."""

    def __init__(self, a, a_scale, b, b_scale):
        self.a, self.a_scale, self.b, self.b_scale = a, a_scale, b, b_scale


def gdn_inputs(q, k, v, alpha, beta) -> rsq_gdn_inputs:
    return rsq_gdn_inputs(_dptr(q), _dptr(k), _dptr(v), _dptr(alpha), _dptr(beta))


def diag_inputs(q, k, v, alpha, beta=None) -> rsq_diag_inputs:
    """GLA / KDA inputs: alpha is the decay per key channel ([B][H][dk] float32)."""
    return rsq_diag_inputs(_dptr(q), _dptr(k), _dptr(v), _dptr(alpha), _dptr(beta))


def mamba2_inputs(x, Bm, Cm, dt, A, D, decay=None) -> rsq_mamba2_inputs:
    return rsq_mamba2_inputs(_dptr(x), _dptr(Bm), _dptr(Cm), _dptr(dt), _dptr(A), _dptr(D), _dptr(decay))


def _row_stride(t, row: int, what: str) -> int:
    """Stride of a tensor's rows of `row` elements, 0 for one row.  Rows that share memory are
    refused: those of a broadcast tensor have stride 0, which is "packed" to the kernels."""
    if t.shape[0] < 2:
        return 0
    s = int(t.stride(0))
    if s < row:
        raise ValueError("%s: rows of %d elements lie %d apart (a broadcast tensor has to be copied out)" % (what, row, s))
    return s


def _token_rows(t, what: str) -> tuple[int | None, int]:
    """Address and token stride of a [tokens, ...] argument whose token rows are packed
    but may lie apart (a slice of a projection's output)."""
    if t is None or isinstance(t, int):
        return t, 0
    inner = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] > 1 and t.stride(d) != inner:
            raise ValueError("%s: the row of one token has to be contiguous" % what)
        inner *= t.shape[d]
    p = _dptr(t) if t.dim() < 2 or t.is_contiguous() else _dptr(t[:1].view(-1)) if t.shape[0] else _dptr(t[:1])
    return p, _row_stride(t, inner, what) if t.dim() > 1 else 0


def scan_inputs(x, Bm, Cm, dt=None, A=None, D=None, decay=None) -> rsq_scan_inputs:
    """x [tokens, heads, dv], Bm, Cm [tokens, ngroups, dk]: their tokens may lie apart.  The
    result keeps the tensors that it points at."""
    (xp, xs), (bp, bs), (cp, cs) = _token_rows(x, "x"), _token_rows(Bm, "Bm"), _token_rows(Cm, "Cm")
    types = _types()
    bf16, f32 = types[RSQ_BF16], types[RSQ_F32]
    for name, t, want in (("x", x, bf16), ("Bm", Bm, bf16), ("Cm", Cm, bf16), ("dt", dt, f32), ("A", A, f32), ("D", D, f32),
                          ("decay", decay, f32)):
        if t is not None and not isinstance(t, int) and t.dtype is not want:
            raise ValueError("%s: expected %s, got %s" % (name, want, t.dtype))
    ins = rsq_scan_inputs(xp, bp, cp, _dptr(dt), _dptr(A), _dptr(D), _dptr(decay), xs, bs, cs)
    ins.tensors = (x, Bm, Cm, dt, A, D, decay)
    return ins


def scan_grads(dx=None, dBm=None, dCm=None, ddt=None, dlog_decay=None, dA=None, dD=None,
               dstate_in=None) -> rsq_scan_grads:
    """Null for a gradient that is not wanted.  The result keeps the tensors that it points at."""
    grads = rsq_scan_grads(_dptr(dx), _dptr(dBm), _dptr(dCm), _dptr(ddt), _dptr(dlog_decay), _dptr(dA),
                           _dptr(dD), _dptr(dstate_in))
    grads.tensors = (dx, dBm, dCm, ddt, dlog_decay, dA, dD, dstate_in)
    return grads


def norm_config(x, side, y, *, group: int = 0, order: int = RSQ_NORM_GATE, eps: float = 1e-5) -> rsq_norm_config:
    """From the tensors of the call: x [rows, width], side (the gate z, or the residual
    stream; None: no gate) of the same shape, y a tensor or a torch dtype."""
    rows, width = x.shape
    if side is not None and tuple(side.shape) != (rows, width):
        raise ValueError("x has shape %s, the other input %s" % (tuple(x.shape), tuple(side.shape)))

    return rsq_norm_config(rows, width, int(group), int(order), _dtype_of(x),
                           RSQ_F32 if side is None else _dtype_of(side), _dtype_of(y), float(eps), _row_stride(x, width, "x"),
                           0 if side is None else _row_stride(side, width, "z or residual"))


class Scan:
    """The scan of one layer over sequences of given total length (rsq_scan)."""

    def __init__(self, sequences: int, tokens: int, heads: int, dk: int, dv: int, *, ngroups: int = 1,
                 ragged: bool = False, family: int = RSQ_MAMBA2, in_dtype: int = RSQ_BF16):
        self.cfg = rsq_scan_config(int(family), int(in_dtype), int(sequences), int(heads), int(dk), int(dv),
                                   int(ngroups), int(ragged), int(tokens))
        self.workspace_bytes = rsq_scan_workspace(self.cfg, False)
        self.backward_workspace_bytes = rsq_scan_workspace(self.cfg, True)

    def alloc_workspace(self, backward: bool = False, device="cuda"):
        """One call's scratch (forward, or backward); calls that may overlap need one each."""
        import torch
        n = self.backward_workspace_bytes if backward else self.workspace_bytes
        return torch.empty(n, dtype=torch.uint8, device=device) if n else None

    def forward(self, inputs, out, *, state_in=None, state_out=None, cu_seqlens=None, workspace=None, stream=None):
        rsq_scan(self.cfg, inputs, out, cu_seqlens=cu_seqlens, state_in=state_in, state_out=state_out,
                 workspace=workspace, stream=stream)

    def backward(self, inputs, dout, grads, *, state_in=None, dstate_out=None, cu_seqlens=None, workspace=None,
                 stream=None):
        rsq_scan_backward(self.cfg, inputs, dout, grads, cu_seqlens=cu_seqlens, state_in=state_in,
                          dstate_out=dstate_out, workspace=workspace, stream=stream)


class Context:
    """Owns one rsq_ctx (one layer configuration)."""

    def __init__(self, family: int, batch: int, heads: int, dk: int, dv: int, *, head_bits=None,
                 rounding: int = RSQ_SR8, in_dtype: int = RSQ_BF16, seed: int = 0, ngroups: int = 1,
                 window: int = 0, key_axis: int = 0, allocator=None):
        """``allocator``: optional (alloc(nbytes) -> device address or None,
        release(address)) pair for the context's own device word."""
        self.family, self.batch, self.heads, self.dk, self.dv = family, batch, heads, dk, dv
        self.head_bits = None if head_bits is None else np.asarray(head_bits, np.int8)
        self.rounding, self.in_dtype, self.seed, self.ngroups = rounding, in_dtype, seed, ngroups
        self.window, self.key_axis = window, key_axis
        self._hooks = (None, None)
        if allocator is not None:
            a, r = allocator
            self._hooks = (rsq_alloc_fn(lambda n, _u: a(int(n))), rsq_release_fn(lambda p, _u: r(int(p))))
        self.ctx = rsq_create(family, batch, heads, dk, dv, head_bits=head_bits, rounding=rounding,
                              in_dtype=in_dtype, seed=seed, ngroups=ngroups, window=window,
                              key_axis=key_axis, alloc=self._hooks[0], release=self._hooks[1])
        self.code_bytes, self.scale_bytes = rsq_state_bytes(self.ctx)

    def close(self):
        if getattr(self, "ctx", None):
            rsq_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_state(self, device="cuda") -> State:
        import torch
        codes = torch.empty((self.batch, self.code_bytes // self.batch), dtype=torch.uint8, device=device)
        scales = torch.empty((self.batch, self.heads, self.dk if self.key_axis else self.dv),
                             dtype=torch.float32, device=device)
        return State(codes, scales)

    def decode_step(self, state_in: State, state_out: State, inputs, out, step: int, stream=None):
        rsq_decode_step(self.ctx, state_in, state_out, inputs, out, step, stream)

    def alloc_window(self, device="cuda") -> Window:
        """An empty (all-zero) pure-write window."""
        import torch
        B, H, W = self.batch, self.heads, self.window
        return Window(torch.zeros((B, H, W, self.dk), dtype=torch.uint8, device=device),
                      torch.zeros((B, H, W), dtype=torch.float32, device=device),
                      torch.zeros((B, H, self.dv // 16, W, 16), dtype=torch.uint8, device=device),
                      torch.zeros((B, H, W), dtype=torch.float32, device=device))

    def decode_step_window(self, state_in: State, state_out: State, win_in: Window, win_out: Window,
                           inputs, out, step: int, stream=None):
        rsq_decode_step_window(self.ctx, state_in, state_out, win_in, win_out, inputs, out, step, stream)

    def decode_step_copy_scale(self, state_in: State, state_out: State, inputs, copy_absmax, out,
                               step: int, stream=None):
        rsq_decode_step_copy_scale(self.ctx, state_in, state_out, inputs, copy_absmax, out, step, stream)

    def column_absmax(self, state: State, absmax, stream=None):
        rsq_column_absmax(self.ctx, state, absmax, stream)

    def quantize(self, S, state_out: State, step: int = 0, stream=None):
        rsq_quantize(self.ctx, S, state_out, step, stream)

    def dequantize(self, state_in: State, S_out, stream=None):
        rsq_dequantize(self.ctx, state_in, S_out, stream)

    def check_flags(self, stream=None) -> int:
        return rsq_check_flags(self.ctx, stream)


def pack_host_inputs(ctx: "Context", inputs: dict, out=None):
    """Pack one step's host input arrays (numpy; bf16 as uint16 bits) into the
    library's host layout (rsq_host_input_layout), in page-locked memory.
    Marshalling only: each array is copied byte for byte to its offset."""
    import torch
    names = (("x", "Bm", "Cm", "dt", "A", "D") if ctx.family == RSQ_MAMBA2
             else ("q", "k", "v", "alpha", "beta"))
    off, size, total = rsq_host_input_layout(ctx.ctx)
    if out is None:
        out = torch.empty(total, dtype=torch.uint8, pin_memory=True)
    buf = out.numpy()
    for f, name in enumerate(names):
        if size[f] == 0:
            continue
        a = np.ascontiguousarray(inputs[name]).reshape(-1).view(np.uint8)
        if a.size != size[f]:
            raise ValueError("input %s has %d bytes, the layout expects %d" % (name, a.size, size[f]))
        buf[off[f]:off[f] + size[f]] = a
    return out


class Pipe:
    """An end-to-end pipeline over host buffers for one Context (rsq_pipe)."""

    def __init__(self, ctx: "Context"):
        self.context = ctx  # the pipe borrows the context: keep it alive
        self.pipe = rsq_pipe_create(ctx.ctx)
        self.copy_in, self.compute, self.copy_out = rsq_pipe_streams(self.pipe)

    def step(self, state_in: State, state_out: State, host_inputs, host_out, step: int, win_in=None,
             win_out=None):
        rsq_pipe_step(self.pipe, state_in, state_out, host_inputs, host_out, step, win_in, win_out)

    def sync(self):
        rsq_pipe_sync(self.pipe)

    def close(self):
        if getattr(self, "pipe", None):
            rsq_pipe_destroy(self.pipe)
            self.pipe = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
