"""h3q -- fused NVFP4 activation producers for GB300 (sm_103a).

A thin Python binding of the C ABI in ``include/h3q.h`` (``libh3q.so``, built
in-tree by :func:`nvfp4_activation_quantize_gb300.build.build`).  The functions
carry the C names and only marshal torch CUDA tensors into the C calls; every
step of the computation runs in the library's CUDA kernels.  There is no CPU
fallback: if the library is missing or no GPU is present the calls raise.

Outputs that are not passed in are allocated here with ``torch.empty`` in the
shapes of the ABI (codes ``[rows, cols/2]`` uint8, scales
``[pad128(rows), cols/16]`` uint8 in the 128x4 swizzled layout).  With a ``stream``
other than the current one, that stream first waits for what the current one has queued
(whose memory such an output may be made of) and the output is recorded on it.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

__all__ = [
    "H3Q_OK", "H3Q_ERR_INVALID_ARGUMENT", "H3Q_ERR_CUDA", "H3QError", "library", "library_path",
    "padded_rows", "scale_bytes", "h3q_quantize_nvfp4", "h3q_rmsnorm_adaln_nvfp4",
    "h3q_swiglu_nvfp4", "h3q_dequantize_nvfp4", "h3q_last_error", "h3q_abi_version",
    "h3q_amax_bf16", "h3q_rmsnorm_adaln_amax", "h3q_rmsnorm_adaln_nvfp4_from_rstd", "h3q_swiglu_amax",
    "h3q_global_scale_from_amax",
    "h3q_quantize_nvfp4_dynamic", "h3q_residual_rmsnorm_adaln_nvfp4", "h3q_swiglu_packed_nvfp4",
    "h3q_qkv_epilogue", "h3q_rmsnorm_adaln_nvfp4_host", "host_workspace_bytes",
    "h3q_gemm_swiglu_nvfp4", "h3q_kernel_error_flag",
    "kv_cache_nvfp4", "h3q_kv_cache_write_nvfp4", "h3q_kv_cache_read_nvfp4",
    "h3q_attention_cache_nvfp4", "attention_cache_workspace_bytes", "h3q_attention_varlen",
    "h3q_qkv_epilogue_axes", "h3q_postnorm_residual_adaln_nvfp4",
    "block_rows", "select_blocks_workspace_bytes", "h3q_select_blocks", "h3q_attention_blocks",
]

H3Q_OK = 0
H3Q_ERR_INVALID_ARGUMENT = 1
H3Q_ERR_CUDA = 2

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIGNATURES = {
    "h3q_quantize_nvfp4": [_P, _I64, _I64, _I64, _P, _P, _P, _P],
    "h3q_rmsnorm_adaln_nvfp4": [_P, _I64, _P, _P, _I64, _P, _I64, ctypes.c_float, _I64, _I64,
                                _P, _P, _P, _P, _P],
    "h3q_swiglu_nvfp4": [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P],
    "h3q_dequantize_nvfp4": [_P, _P, _I64, _I64, _P, _P, _P],
    "h3q_amax_bf16": [_P, _I64, _I64, _I64, _P, _P],
    "h3q_rmsnorm_adaln_amax": [_P, _I64, _P, _P, _I64, _P, _I64, ctypes.c_float, _I64, _I64, _P, _P, _P],
    "h3q_rmsnorm_adaln_nvfp4_from_rstd": [_P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P],
    "h3q_swiglu_amax": [_P, _I64, _P, _I64, _I64, _I64, _P, _P],
    "h3q_global_scale_from_amax": [_P, _P, _P],
    "h3q_quantize_nvfp4_dynamic": [_P, _I64, _I64, _I64, _P, _P, _P, _P],
    "h3q_swiglu_packed_nvfp4": [_P, _I64, _P, _I64, _I64, _P, _P, _P, _P],
    "h3q_residual_rmsnorm_adaln_nvfp4": [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _I64,
                                         ctypes.c_float, _I64, _I64, _P, _P, _P, _P, _P],
    "h3q_rmsnorm_adaln_nvfp4_host": [_P, _I64, _I64, _P, _P, _I64, _P, _I64, ctypes.c_float, _P, _P, _P, _P,
                                     _I64, _I64, _P],
    "h3q_qkv_epilogue": [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, ctypes.c_int, _I64, _I64,
                         _I64, ctypes.c_float, _P, _P, _P, _P],
    "h3q_gemm_swiglu_nvfp4": [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P],
    "h3q_kernel_error_flag": [_P],
    "h3q_kv_cache_write_nvfp4": [_P, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64,
                                 _I64, _I64, _I64, _P],
    "h3q_kv_cache_read_nvfp4": [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _P, _I64, _I64, _P,
                                _P, _P],
    "h3q_attention_varlen": [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.c_int,
                             ctypes.c_float, _P, _P, _P],
    "h3q_attention_cache_nvfp4": [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64,
                                  _I64, _I64, _P, _P, ctypes.c_float, _P, _P, _P, _I64, _P],
    "h3q_qkv_epilogue_axes": [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, ctypes.c_int,
                              ctypes.c_int, ctypes.c_int, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _P, _P, _P],
    "h3q_postnorm_residual_adaln_nvfp4": [_P, _I64, _P, _I64, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _P, _I64,
                                          ctypes.c_float, _I64, _I64, _P, _P, _P, _P, _P],
    "h3q_select_blocks": [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.c_int,
                          _I64, _P, _P, _P, _I64, _P],
    "h3q_attention_blocks": [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P,
                             _I64, ctypes.c_int, ctypes.c_float, _P, _P, _P],
}

_lock = threading.Lock()
_lib = None


class H3QError(RuntimeError):
    """A nonzero status from the library, with its message."""

    def __init__(self, fn: str, code: int, message: str):
        super().__init__(f"{fn} returned {code}: {message}")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def library():
    """The loaded ``libh3q.so``; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with nvfp4_activation_quantize_gb300.build.build() "
                    "(there is no fallback implementation)")
            lib = ctypes.CDLL(path)
            for name, args in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            lib.h3q_last_error.argtypes = []
            lib.h3q_last_error.restype = ctypes.c_char_p
            lib.h3q_abi_version.argtypes = []
            lib.h3q_abi_version.restype = ctypes.c_int
            _lib = lib
    return _lib


def h3q_last_error() -> str:
    return library().h3q_last_error().decode()


def h3q_abi_version() -> int:
    return library().h3q_abi_version()


def padded_rows(rows: int) -> int:
    return (rows + 127) // 128 * 128


def scale_bytes(rows: int, cols: int) -> int:
    return padded_rows(rows) * (cols // 16)


def host_workspace_bytes(chunk_rows: int, cols: int, rows: int, with_frames: bool) -> int:
    """Device workspace bytes of h3q_rmsnorm_adaln_nvfp4_host (h3q_host_workspace_bytes in
    include/h3q.h): three staging slots, then the frames when they come from rows_per_frame."""
    a = lambda n: (n + 255) // 256 * 256  # noqa: E731
    slot = a(chunk_rows * cols * 2) + a(chunk_rows * cols // 2) + a(chunk_rows * cols // 16)
    return 3 * slot + (a(rows * 4) if with_frames else 0)


def _check(fn: str, rc: int) -> None:
    if rc != H3Q_OK:
        raise H3QError(fn, rc, h3q_last_error())


def _cuda_tensor(name, t, dtype, device=None):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _rows_view(name, t, dtype, device=None):
    """A 2-D view with unit column stride; returns (tensor, rows, cols, ld)."""
    _cuda_tensor(name, t, dtype, device)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    return t, t.shape[0], t.shape[1], ld


def _contiguous(name, t, dtype, shape, device):
    _cuda_tensor(name, t, dtype, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _outputs(device, rows, cols, codes, scales, stream):
    import torch

    fresh = []
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        fresh.append(codes)
    if scales is None:
        scales = torch.empty((padded_rows(rows), cols // 16), dtype=torch.uint8, device=device)
        fresh.append(scales)
    _lend(stream, device, fresh)
    _contiguous("codes", codes, torch.uint8, (rows, cols // 2), device)
    _contiguous("scales", scales, torch.uint8, (padded_rows(rows), cols // 16), device)
    return codes, scales


def _gsf(global_scale, device):
    import torch

    _cuda_tensor("global_scale", global_scale, torch.float32, device)
    if global_scale.numel() != 1:
        raise ValueError("global_scale must hold one fp32 value")
    return global_scale


def _stream(stream, device) -> int:
    import torch

    if stream is None:
        # (the handle alone: the stream object takes twenty times as long)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and device.index is not None:
            return raw(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _lend(stream, device, fresh) -> None:
    """Tensors that the binding has just allocated, which torch does on the current stream, made ready for a
    kernel on the stream argument: it waits for the current stream's work (which may still use the memory, or
    fill it), and the memory is not given away before the kernel has ended."""
    if stream is None or not fresh:
        return
    import torch

    handle = _stream(stream, device)
    if handle == _stream(None, device):
        return
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):   # a number, or another library's object (1: the legacy default)
        stream = (torch.cuda.default_stream(device) if handle <= 1
                  else torch.cuda.ExternalStream(handle, device=device))

    def capturing(s):
        with torch.cuda.stream(s):
            return torch.cuda.is_current_stream_capturing()

    if capturing(stream) == capturing(current):   # (a graph cannot wait for work outside it, nor such work for it)
        stream.wait_stream(current)
    for t in fresh:
        t.record_stream(stream)


def h3q_quantize_nvfp4(x, global_scale, codes=None, scales=None, stream=None):
    """Standalone NVFP4 quantize of bf16 x [rows, cols]; returns (codes, scales)."""
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    dev = x.device
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_quantize_nvfp4(x.data_ptr(), ld, rows, cols, gsf.data_ptr(),
                                          codes.data_ptr(), scales.data_ptr(), _stream(stream, dev))
    _check("h3q_quantize_nvfp4", rc)
    return codes, scales


def h3q_rmsnorm_adaln_nvfp4(x, gamma, mod_table, global_scale, *, row_frame=None,
                            rows_per_frame=None, eps=1e-6, codes=None, scales=None, row_rstd=None,
                            stream=None):
    """RMSNorm (fp32 statistics) + AdaLN modulation + NVFP4 of bf16 x [rows, cols].

    ``mod_table`` is bf16 [frames, 2, cols] ([t, 0] shift, [t, 1] scale); the frame
    of a row is ``row_frame[row]`` (int32 CUDA tensor) or ``row // rows_per_frame``.
    ``row_rstd`` (fp32 [rows], optional) receives each row's rstd.
    Returns (codes, scales).
    """
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    dev = x.device
    _contiguous("gamma", gamma, torch.bfloat16, (cols,), dev)
    _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
    if mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous():
        raise ValueError("mod_table must be contiguous [frames, 2, cols]")
    frames = mod_table.shape[0]
    rf_ptr = None
    if row_frame is not None:
        _contiguous("row_frame", row_frame, torch.int32, (rows,), dev)
        rf_ptr = row_frame.data_ptr()
        rows_per_frame = 0
    elif rows_per_frame is None:
        raise ValueError("give row_frame or rows_per_frame")
    rstd_ptr = None
    if row_rstd is not None:
        _contiguous("row_rstd", row_rstd, torch.float32, (rows,), dev)
        rstd_ptr = row_rstd.data_ptr()
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_rmsnorm_adaln_nvfp4(
            x.data_ptr(), ld, gamma.data_ptr(), mod_table.data_ptr(), frames, rf_ptr,
            int(rows_per_frame), float(eps), rows, cols, gsf.data_ptr(), codes.data_ptr(),
            scales.data_ptr(), rstd_ptr, _stream(stream, dev))
    _check("h3q_rmsnorm_adaln_nvfp4", rc)
    return codes, scales


def h3q_swiglu_nvfp4(gate, up, global_scale, codes=None, scales=None, stream=None):
    """NVFP4 of bf16(silu(gate) * up) for bf16 gate, up [rows, cols]; returns (codes, scales)."""
    import torch

    gate, rows, cols, ldg = _rows_view("gate", gate, torch.bfloat16)
    dev = gate.device
    up, rows_u, cols_u, ldu = _rows_view("up", up, torch.bfloat16, dev)
    if (rows_u, cols_u) != (rows, cols):
        raise ValueError("gate and up must have the same shape")
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_swiglu_nvfp4(gate.data_ptr(), ldg, up.data_ptr(), ldu, rows, cols,
                                        gsf.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                        _stream(stream, dev))
    _check("h3q_swiglu_nvfp4", rc)
    return codes, scales


def h3q_dequantize_nvfp4(codes, scales, global_scale, out=None, stream=None):
    """fp32 [rows, cols] = E2M1(code) * E4M3(scale) / gsf (checking path)."""
    import torch

    _cuda_tensor("codes", codes, torch.uint8)
    dev = codes.device
    if codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be contiguous [rows, cols/2]")
    rows, cols = codes.shape[0], codes.shape[1] * 2
    _contiguous("scales", scales, torch.uint8, (padded_rows(rows), cols // 16), dev)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=dev)
        _lend(stream, dev, [out])
    _contiguous("out", out, torch.float32, (rows, cols), dev)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_dequantize_nvfp4(codes.data_ptr(), scales.data_ptr(), rows, cols,
                                            gsf.data_ptr(), out.data_ptr(), _stream(stream, dev))
    _check("h3q_dequantize_nvfp4", rc)
    return out


# --------------------------------------------------------------------------- #
# dynamic and calibrated global scales                                          #
# --------------------------------------------------------------------------- #

def _amax_buffer(amax, device, stream):
    import torch

    if amax is None:
        amax = torch.zeros(1, dtype=torch.float32, device=device)
        _lend(stream, device, [amax])
    _cuda_tensor("amax", amax, torch.float32, device)
    if amax.numel() != 1:
        raise ValueError("amax must hold one fp32 value")
    return amax


def h3q_amax_bf16(x, amax=None, stream=None):
    """Fold max |x| of bf16 x [rows, cols] into the fp32 device scalar ``amax``
    (a new zero scalar when None); returns amax."""
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    amax = _amax_buffer(amax, x.device, stream)
    with torch.cuda.device(x.device):
        rc = library().h3q_amax_bf16(x.data_ptr(), ld, rows, cols, amax.data_ptr(),
                                     _stream(stream, x.device))
    _check("h3q_amax_bf16", rc)
    return amax


def h3q_rmsnorm_adaln_amax(x, gamma, mod_table, *, row_frame=None, rows_per_frame=None, eps=1e-6,
                           amax=None, row_rstd=None, stream=None):
    """Fold max |y| of the RMSNorm + AdaLN output y (the bf16 values the producer
    quantizes, same arguments) into ``amax``; returns amax.  ``row_rstd`` (fp32
    [rows], optional) receives each row's rstd, for h3q_rmsnorm_adaln_nvfp4_from_rstd."""
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    dev = x.device
    _contiguous("gamma", gamma, torch.bfloat16, (cols,), dev)
    _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
    if mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous():
        raise ValueError("mod_table must be contiguous [frames, 2, cols]")
    rf_ptr = None
    if row_frame is not None:
        _contiguous("row_frame", row_frame, torch.int32, (rows,), dev)
        rf_ptr = row_frame.data_ptr()
        rows_per_frame = 0
    elif rows_per_frame is None:
        raise ValueError("give row_frame or rows_per_frame")
    amax = _amax_buffer(amax, dev, stream)
    rstd_ptr = None
    if row_rstd is not None:
        _contiguous("row_rstd", row_rstd, torch.float32, (rows,), dev)
        rstd_ptr = row_rstd.data_ptr()
    with torch.cuda.device(dev):
        rc = library().h3q_rmsnorm_adaln_amax(
            x.data_ptr(), ld, gamma.data_ptr(), mod_table.data_ptr(), mod_table.shape[0], rf_ptr,
            int(rows_per_frame), float(eps), rows, cols, amax.data_ptr(), rstd_ptr, _stream(stream, dev))
    _check("h3q_rmsnorm_adaln_amax", rc)
    return amax


def h3q_rmsnorm_adaln_nvfp4_from_rstd(x, gamma, mod_table, row_rstd, global_scale, *, row_frame=None,
                                      rows_per_frame=None, codes=None, scales=None, stream=None):
    """The RMSNorm + AdaLN producer with each row's rstd given (fp32 [rows], e.g. the
    abs-max pass's ``row_rstd``): the statistics are not formed again.  Returns
    (codes, scales)."""
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    dev = x.device
    _contiguous("gamma", gamma, torch.bfloat16, (cols,), dev)
    _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
    if mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous():
        raise ValueError("mod_table must be contiguous [frames, 2, cols]")
    _contiguous("row_rstd", row_rstd, torch.float32, (rows,), dev)
    rf_ptr = None
    if row_frame is not None:
        _contiguous("row_frame", row_frame, torch.int32, (rows,), dev)
        rf_ptr = row_frame.data_ptr()
        rows_per_frame = 0
    elif rows_per_frame is None:
        raise ValueError("give row_frame or rows_per_frame")
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_rmsnorm_adaln_nvfp4_from_rstd(
            x.data_ptr(), ld, gamma.data_ptr(), mod_table.data_ptr(), mod_table.shape[0], rf_ptr,
            int(rows_per_frame), row_rstd.data_ptr(), rows, cols, gsf.data_ptr(), codes.data_ptr(),
            scales.data_ptr(), _stream(stream, dev))
    _check("h3q_rmsnorm_adaln_nvfp4_from_rstd", rc)
    return codes, scales


def h3q_swiglu_amax(gate, up, amax=None, stream=None):
    """Fold max |bf16(silu(gate) * up)| into ``amax``; returns amax."""
    import torch

    gate, rows, cols, ldg = _rows_view("gate", gate, torch.bfloat16)
    dev = gate.device
    up, rows_u, cols_u, ldu = _rows_view("up", up, torch.bfloat16, dev)
    if (rows_u, cols_u) != (rows, cols):
        raise ValueError("gate and up must have the same shape")
    amax = _amax_buffer(amax, dev, stream)
    with torch.cuda.device(dev):
        rc = library().h3q_swiglu_amax(gate.data_ptr(), ldg, up.data_ptr(), ldu, rows, cols,
                                       amax.data_ptr(), _stream(stream, dev))
    _check("h3q_swiglu_amax", rc)
    return amax


def h3q_global_scale_from_amax(amax, global_scale=None, stream=None):
    """The global scale fl(2688 / amax) computed on the device from the fp32 scalar
    ``amax`` (0 gives 1; +inf is clamped); returns the fp32 scalar written."""
    import torch

    _cuda_tensor("amax", amax, torch.float32)
    dev = amax.device
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=dev)
        _lend(stream, dev, [global_scale])
    _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_global_scale_from_amax(amax.data_ptr(), global_scale.data_ptr(),
                                                  _stream(stream, dev))
    _check("h3q_global_scale_from_amax", rc)
    return global_scale


def h3q_quantize_nvfp4_dynamic(x, global_scale=None, codes=None, scales=None, stream=None):
    """NVFP4 of bf16 x [rows, cols] under its own per-call abs-max scale, with the
    abs-max pass's scratch inside the library (no caller scratch, no allocation
    there).  Returns (codes, scales, global_scale); global_scale is the fp32 device
    scalar the call wrote.  Calls overlapping on one device race on that scratch."""
    import torch

    x, rows, cols, ld = _rows_view("x", x, torch.bfloat16)
    dev = x.device
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=dev)
        _lend(stream, dev, [global_scale])
    _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_quantize_nvfp4_dynamic(x.data_ptr(), ld, rows, cols,
                                                  global_scale.data_ptr(), codes.data_ptr(),
                                                  scales.data_ptr(), _stream(stream, dev))
    _check("h3q_quantize_nvfp4_dynamic", rc)
    return codes, scales, global_scale


def h3q_residual_rmsnorm_adaln_nvfp4(h, o, gate_table, gamma, mod_table, global_scale, *, bias=None,
                                     row_frame=None, rows_per_frame=None, eps=1e-6, codes=None,
                                     scales=None, row_rstd=None, stream=None):
    """Residual fold + RMSNorm + AdaLN -> NVFP4: h (fp32 [rows, cols], updated in place)
    += bf16(o + bias) * gate_table[frame], then the AdaLN producer on the folded h.
    ``gate_table`` bf16 [frames, cols]; ``mod_table`` bf16 [frames, 2, cols].
    Returns (codes, scales)."""
    import torch

    _cuda_tensor("h", h, torch.float32)
    dev = h.device
    if h.dim() != 2 or (h.shape[1] > 1 and h.stride(1) != 1):
        raise ValueError("h must be 2-D with contiguous rows")
    rows, cols = h.shape
    ld_h = h.stride(0) if rows > 1 else cols
    o, rows_o, cols_o, ld_o = _rows_view("o", o, torch.bfloat16, dev)
    if (rows_o, cols_o) != (rows, cols):
        raise ValueError("o must have the shape of h")
    bias_ptr = None
    if bias is not None:
        _contiguous("bias", bias, torch.bfloat16, (cols,), dev)
        bias_ptr = bias.data_ptr()
    _cuda_tensor("gate_table", gate_table, torch.bfloat16, dev)
    if gate_table.dim() != 2 or gate_table.shape[1] != cols or not gate_table.is_contiguous():
        raise ValueError("gate_table must be contiguous [frames, cols]")
    _contiguous("gamma", gamma, torch.bfloat16, (cols,), dev)
    _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
    if (mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous()
            or mod_table.shape[0] != gate_table.shape[0]):
        raise ValueError("mod_table must be contiguous [frames, 2, cols], frames as gate_table")
    rf_ptr = None
    if row_frame is not None:
        _contiguous("row_frame", row_frame, torch.int32, (rows,), dev)
        rf_ptr = row_frame.data_ptr()
        rows_per_frame = 0
    elif rows_per_frame is None:
        raise ValueError("give row_frame or rows_per_frame")
    rstd_ptr = None
    if row_rstd is not None:
        _contiguous("row_rstd", row_rstd, torch.float32, (rows,), dev)
        rstd_ptr = row_rstd.data_ptr()
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_residual_rmsnorm_adaln_nvfp4(
            h.data_ptr(), ld_h, o.data_ptr(), ld_o, bias_ptr, gate_table.data_ptr(), gamma.data_ptr(),
            mod_table.data_ptr(), mod_table.shape[0], rf_ptr, int(rows_per_frame), float(eps), rows,
            cols, gsf.data_ptr(), codes.data_ptr(), scales.data_ptr(), rstd_ptr, _stream(stream, dev))
    _check("h3q_residual_rmsnorm_adaln_nvfp4", rc)
    return codes, scales


def h3q_swiglu_packed_nvfp4(o, global_scale, bias=None, codes=None, scales=None, stream=None):
    """SwiGLU of the value-first packed projection o [rows, 2F] (value, then gate)
    with its bias [2F] (or None) added and rounded to bf16 first; returns (codes, scales)
    of the [rows, F] output."""
    import torch

    o, rows, two_f, ld = _rows_view("o", o, torch.bfloat16)
    dev = o.device
    if two_f % 2:
        raise ValueError("o must have an even number of columns")
    f = two_f // 2
    bias_ptr = None
    if bias is not None:
        _contiguous("bias", bias, torch.bfloat16, (two_f,), dev)
        bias_ptr = bias.data_ptr()
    codes, scales = _outputs(dev, rows, f, codes, scales, stream)
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_swiglu_packed_nvfp4(o.data_ptr(), ld, bias_ptr, rows, f, gsf.data_ptr(),
                                               codes.data_ptr(), scales.data_ptr(), _stream(stream, dev))
    _check("h3q_swiglu_packed_nvfp4", rc)
    return codes, scales


def h3q_qkv_epilogue(q, k, v, biases, cos, sin, heads, eps, outs=None, interleaved=False, stream=None):
    """QKV epilogue of projected q, k, v [rows, heads * HD] bf16 (bias not yet added):
    returns (q_out, k_out, v_out), each bf16 [rows, heads, HD], with q and k biased,
    RMS-normed per head and rotated (RoPE on each head's first ROT values, cos and
    sin bf16 [rows, ROT], None for ROT = 0: rotate-half pairs (i, i + ROT/2), or
    pairs (2j, 2j + 1) with ``interleaved``) and v biased."""
    import torch

    q, rows, d, ld_q = _rows_view("q", q, torch.bfloat16)
    dev = q.device
    k, rows_k, d_k, ld_k = _rows_view("k", k, torch.bfloat16, dev)
    v, rows_v, d_v, ld_v = _rows_view("v", v, torch.bfloat16, dev)
    if (rows_k, d_k) != (rows, d) or (rows_v, d_v) != (rows, d):
        raise ValueError("q, k and v must have the same shape")
    if heads < 1 or d % heads:
        raise ValueError("the columns of q must split into heads")
    hd = d // heads
    b = [_contiguous(n, t, torch.bfloat16, (d,), dev) for n, t in zip(("bias_q", "bias_k", "bias_v"), biases)]
    rot, cos_ptr, sin_ptr = 0, None, None
    if cos is not None or sin is not None:
        rot = cos.shape[-1] if cos.dim() == 2 else -1
        _contiguous("cos", cos, torch.bfloat16, (rows, rot), dev)
        _contiguous("sin", sin, torch.bfloat16, (rows, rot), dev)
        cos_ptr, sin_ptr = cos.data_ptr(), sin.data_ptr()
    if outs is None:
        outs = [torch.empty((rows, heads, hd), dtype=torch.bfloat16, device=dev) for _ in range(3)]
        _lend(stream, dev, outs)
    outs = [_contiguous(n, t, torch.bfloat16, (rows, heads, hd), dev)
            for n, t in zip(("q_out", "k_out", "v_out"), outs)]
    with torch.cuda.device(dev):
        rc = library().h3q_qkv_epilogue(q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v,
                                        b[0].data_ptr(), b[1].data_ptr(), b[2].data_ptr(), cos_ptr,
                                        sin_ptr, rot, int(bool(interleaved)), rows, heads, hd, float(eps),
                                        outs[0].data_ptr(),
                                        outs[1].data_ptr(), outs[2].data_ptr(), _stream(stream, dev))
    _check("h3q_qkv_epilogue", rc)
    return outs[0], outs[1], outs[2]


def h3q_rmsnorm_adaln_nvfp4_host(x_host, gamma, mod_table, global_scale, codes_host, scales_host, workspace, *,
                                 row_frame=None, rows_per_frame=None, eps=1e-6, chunk_rows=8192, stream=None):
    """RMSNorm + AdaLN -> NVFP4 on host buffers: x_host (contiguous bf16 [rows, cols] in
    host memory, pinned for the copies to overlap) into host codes [rows, cols/2] and
    scales [pad128(rows), cols/16] (uint8, contiguous), the copies inside the library
    call, pipelined over `chunk_rows`-row chunks.  gamma, mod_table, global_scale and
    row_frame are CUDA tensors; `workspace` is a CUDA uint8 tensor of at least
    host_workspace_bytes(chunk_rows, cols, rows, row_frame is None) bytes.  The host
    outputs may be read once `stream` (default: the current stream) is synchronised."""
    import torch

    if not isinstance(x_host, torch.Tensor) or x_host.is_cuda or x_host.dtype != torch.bfloat16:
        raise ValueError("x_host must be a host bf16 tensor")
    if x_host.dim() != 2 or not x_host.is_contiguous():
        raise ValueError("x_host must be contiguous [rows, cols]")
    rows, cols = x_host.shape
    _cuda_tensor("workspace", workspace, torch.uint8)
    dev = workspace.device
    for name, t, shape in (("codes_host", codes_host, (rows, cols // 2)),
                           ("scales_host", scales_host, (padded_rows(rows), cols // 16))):
        if (not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.uint8 or tuple(t.shape) != shape
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous host uint8 tensor {shape}")
    _contiguous("gamma", gamma, torch.bfloat16, (cols,), dev)
    _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
    if mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous():
        raise ValueError("mod_table must be contiguous [frames, 2, cols]")
    rf_ptr = None
    if row_frame is not None:
        _contiguous("row_frame", row_frame, torch.int32, (rows,), dev)
        rf_ptr = row_frame.data_ptr()
        rows_per_frame = 0
    elif rows_per_frame is None:
        raise ValueError("give row_frame or rows_per_frame")
    gsf = _gsf(global_scale, dev)
    with torch.cuda.device(dev):
        rc = library().h3q_rmsnorm_adaln_nvfp4_host(
            x_host.data_ptr(), rows, cols, gamma.data_ptr(), mod_table.data_ptr(), mod_table.shape[0], rf_ptr,
            int(rows_per_frame), float(eps), gsf.data_ptr(), codes_host.data_ptr(), scales_host.data_ptr(),
            workspace.data_ptr(), workspace.numel(), int(chunk_rows), _stream(stream, dev))
    _check("h3q_rmsnorm_adaln_nvfp4_host", rc)
    return codes_host, scales_host


def h3q_gemm_swiglu_nvfp4(a_codes, a_scales, b_codes, b_scales, alpha, global_scale, codes=None, scales=None,
                          y=None, acc=None, stream=None):
    """The FFN-up projection as a block-scaled NVFP4 GEMM with the SwiGLU + NVFP4 epilogue.

    ``a_codes`` uint8 [m, k/2] and ``a_scales`` uint8 [pad128(m), k/16] (128x4 layout) are
    the NVFP4 activation; ``b_codes`` [n, k/2] and ``b_scales`` [n, k/16] the NVFP4 weight,
    row 2j the value and row 2j+1 the gate of output j.  ``alpha`` and ``global_scale`` are
    device fp32 scalars.  Outputs: codes [m, n/4], scales [pad128(m), n/32]; optional ``y``
    (bf16 [m, n/2]) and ``acc`` (fp32 [m, n], the accumulator before alpha).
    Returns (codes, scales).
    """
    import torch

    _cuda_tensor("a_codes", a_codes, torch.uint8)
    dev = a_codes.device
    if a_codes.dim() != 2 or not a_codes.is_contiguous():
        raise ValueError("a_codes must be contiguous [m, k/2]")
    m, k = a_codes.shape[0], 2 * a_codes.shape[1]
    _cuda_tensor("b_codes", b_codes, torch.uint8, dev)
    if b_codes.dim() != 2 or b_codes.shape[1] != k // 2 or not b_codes.is_contiguous():
        raise ValueError("b_codes must be contiguous [n, k/2]")
    n = b_codes.shape[0]
    f = n // 2
    for name, t, rows in (("a_scales", a_scales, padded_rows(m)), ("b_scales", b_scales, padded_rows(n))):
        _cuda_tensor(name, t, torch.uint8, dev)
        if not t.is_contiguous() or t.numel() != rows * (k // 16):
            raise ValueError(f"{name} must be contiguous with {rows} x {k // 16} bytes")
    _gsf(alpha, dev)
    gsf = _gsf(global_scale, dev)
    codes, scales = _outputs(dev, m, f, codes, scales, stream)
    y_ptr = acc_ptr = None
    if y is not None:
        _contiguous("y", y, torch.bfloat16, (m, f), dev)
        y_ptr = y.data_ptr()
    if acc is not None:
        _contiguous("acc", acc, torch.float32, (m, n), dev)
        acc_ptr = acc.data_ptr()
    with torch.cuda.device(dev):
        rc = library().h3q_gemm_swiglu_nvfp4(
            a_codes.data_ptr(), a_scales.data_ptr(), m, k, b_codes.data_ptr(), b_scales.data_ptr(), n,
            alpha.data_ptr(), gsf.data_ptr(), codes.data_ptr(), scales.data_ptr(), y_ptr, acc_ptr,
            _stream(stream, dev))
    _check("h3q_gemm_swiglu_nvfp4", rc)
    return codes, scales


def h3q_kernel_error_flag() -> int:
    """Reads and clears the flag a kernel sets when one of its bounded waits ran out
    (synchronises the device); 0 when none did."""
    flag = ctypes.c_int(0)
    _check("h3q_kernel_error_flag", library().h3q_kernel_error_flag(ctypes.byref(flag)))
    return flag.value


# --------------------------------------------------------------------------- #
# the paged NVFP4 cache                                                        #
# --------------------------------------------------------------------------- #

def kv_cache_nvfp4(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda"):
    """An empty cache: (k_codes, k_scales, v_codes, v_scales), uint8 [num_pages, kv_heads,
    page_size, head_dim / 2] and [..., head_dim / 16], zeroed."""
    import torch

    return tuple(torch.zeros((num_pages, kv_heads, page_size, head_dim // per), dtype=torch.uint8, device=device)
                 for per in (2, 16, 2, 16))


# The calls of a decoding step run for a few microseconds on the GPU, so they go a short way
# through a C module (csrc/binding.c): it checks the tensors and calls the library, or, where
# anything is not as the call needs it, returns None and leaves it to the code below, whose
# checks say what is wrong.  Where the module could not be built all calls go that way.

_torch = None
_native = None


class _NoShortWay:
    write = read = cached = varlen = axes = postnorm = select = blocks = staticmethod(lambda *args: None)


def _load_torch():
    global _torch, _native
    import importlib.util

    import torch

    lib = library()
    path = _build.BINDING_PATH
    if not os.path.exists(path):
        _native, _torch = _NoShortWay, torch
        return torch
    spec = importlib.util.spec_from_file_location("h3q_binding", path)
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    native.setup(torch.Tensor, torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32,
                 getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
                 raw_stream or (lambda index: torch.cuda.current_stream(index).cuda_stream),
                 *(ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in
                   ("h3q_kv_cache_write_nvfp4", "h3q_kv_cache_read_nvfp4", "h3q_attention_cache_nvfp4",
                    "h3q_attention_varlen")))
    native.setup_blocks(*(ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in
                          ("h3q_qkv_epilogue_axes", "h3q_postnorm_residual_adaln_nvfp4", "h3q_select_blocks",
                           "h3q_attention_blocks")))
    _native = native
    _torch = torch
    return torch


def _handle(stream):
    """The stream argument as the C module takes it: None for the current one, or its handle."""
    return None if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _is(t, dtype, shape, device) -> bool:
    return (isinstance(t, _torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape
            and t.is_contiguous())


def _dense(name, t, dtype, shape, device) -> int:
    """The address of a contiguous CUDA tensor of this type and shape."""
    if not _is(t, dtype, shape, device):
        _contiguous(name, t, dtype, shape, device)
    return t.data_ptr()


def _scale_ptr(t, device) -> int:
    if not (isinstance(t, _torch.Tensor) and t.dtype is _torch.float32 and t.device == device and t.numel() == 1):
        _gsf(t, device)
    return t.data_ptr()


def _invoke(fn, device, stream, args):
    """fn(*args, stream) of the library on the device, which is the current one or becomes it for the call."""
    torch = _torch
    call = getattr(_lib or library(), fn)
    if torch.cuda.current_device() == device.index:
        rc = call(*args, _stream(stream, device))
    else:
        with torch.cuda.device(device):
            rc = call(*args, _stream(stream, device))
    if rc != H3Q_OK:
        raise H3QError(fn, rc, h3q_last_error())


def _cache(cache):
    """Checks the four cache tensors; returns (their addresses, (pages, page_size, kv_heads, head_dim),
    device)."""
    torch = _torch
    if len(cache) != 4:
        raise ValueError("cache must be (k_codes, k_scales, v_codes, v_scales)")
    kc, ks, vc, vs = cache
    _cuda_tensor("k_codes", kc, torch.uint8)
    if kc.dim() != 4:
        raise ValueError("k_codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
    codes = kc.shape
    pages, heads, page, half = codes
    scales = (pages, heads, page, half // 8)
    dev = kc.device
    return ((_dense("k_codes", kc, torch.uint8, codes, dev), _dense("k_scales", ks, torch.uint8, scales, dev),
             _dense("v_codes", vc, torch.uint8, codes, dev), _dense("v_scales", vs, torch.uint8, scales, dev)),
            (pages, page, heads, 2 * half), dev)


def _head_rows(name, t, device=None):
    """bf16 [rows, heads, dim] whose rows are contiguous (any row stride); returns
    (address, shape, row stride)."""
    torch = _torch
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.is_cuda
            and (device is None or t.device == device)):
        _cuda_tensor(name, t, torch.bfloat16, device)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous rows")
    rows, heads, dim = shape
    ld, sh, sd = t.stride()
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim):
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous rows")
    return t.data_ptr(), shape, ld if rows > 1 else heads * dim


def _row_lists(cu_rows, kv_len, block_table, device):
    """Checks the lists of packed rows; returns (cu_rows, kv_len, block_table addresses, batch, max_pages)."""
    i32 = _torch.int32
    if not (isinstance(kv_len, _torch.Tensor) and kv_len.dim() == 1):
        _cuda_tensor("kv_len", kv_len, i32, device)
        raise ValueError("kv_len must be contiguous [batch]")
    batch = kv_len.shape[0]
    if not (isinstance(block_table, _torch.Tensor) and block_table.dim() == 2 and block_table.shape[0] == batch):
        _cuda_tensor("block_table", block_table, i32, device)
        raise ValueError("block_table must be contiguous [batch, max_pages]")
    max_pages = block_table.shape[1]
    return (_dense("cu_rows", cu_rows, i32, (batch + 1,), device), _dense("kv_len", kv_len, i32, (batch,), device),
            _dense("block_table", block_table, i32, (batch, max_pages), device), batch, max_pages)


def h3q_kv_cache_write_nvfp4(k, v, cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale,
                             stream=None):
    """Quantize new key and value rows (bf16 [rows, kv_heads, head_dim], contiguous rows of any
    stride) into the paged NVFP4 ``cache`` (see kv_cache_nvfp4).  Rows cu_rows[b] .. cu_rows[b+1]-1
    are the last positions of sequence b, which has kv_len[b] positions with them; position p is row
    p % page_size of page block_table[b, p // page_size].  All lists are int32 CUDA tensors.  Returns
    the cache."""
    if _torch is None:
        _load_torch()
    rc = _native.write(k, v, cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale,
                       getattr(k, "device", None), _handle(stream))
    if rc is not None:
        if rc != H3Q_OK:
            raise H3QError("h3q_kv_cache_write_nvfp4", rc, h3q_last_error())
        return cache
    ptrs, shape, dev = _cache(cache)
    kp, k_shape, ld_k = _head_rows("k", k, dev)
    vp, v_shape, ld_v = _head_rows("v", v, dev)
    if k_shape[1:] != shape[2:] or v_shape != k_shape:
        raise ValueError("k and v must be [rows, kv_heads, head_dim] of the cache's heads")
    cu, lens, table, batch, max_pages = _row_lists(cu_rows, kv_len, block_table, dev)
    _invoke("h3q_kv_cache_write_nvfp4", dev, stream,
            (kp, ld_k, vp, ld_v, k_shape[0], cu, lens, table, batch, max_pages, _scale_ptr(k_global_scale, dev),
             _scale_ptr(v_global_scale, dev), *ptrs, *shape))
    return cache


def h3q_kv_cache_read_nvfp4(cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale, *, rows=None,
                            outs=None, stream=None):
    """The bf16 values that the cache holds for the packed rows that the lists name (as in
    h3q_kv_cache_write_nvfp4; a whole prefix where cu_rows[b+1] - cu_rows[b] = kv_len[b]).  Give
    ``rows`` (the packed rows) or ``outs`` = (k_out, v_out), bf16 [rows, kv_heads, head_dim].
    Returns (k_out, v_out)."""
    torch = _torch or _load_torch()
    if outs is None:
        if rows is None:
            raise ValueError("give rows or outs")
        if len(cache) != 4 or len(getattr(cache[0], "shape", ())) != 4:
            _cache(cache)
        codes = cache[0].shape
        shape, dev = (rows, codes[1], 2 * codes[3]), cache[0].device
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        _lend(stream, dev, (k_out, v_out))
    else:
        k_out, v_out = outs
    rc = _native.read(cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale, k_out, v_out,
                      getattr(k_out, "device", None), _handle(stream))
    if rc is not None:
        if rc != H3Q_OK:
            raise H3QError("h3q_kv_cache_read_nvfp4", rc, h3q_last_error())
        return k_out, v_out
    ptrs, shape, dev = _cache(cache)
    cu, lens, table, batch, max_pages = _row_lists(cu_rows, kv_len, block_table, dev)
    rows = k_out.shape[0]
    out_shape = (rows, *shape[2:])
    _invoke("h3q_kv_cache_read_nvfp4", dev, stream,
            (*ptrs, *shape, _scale_ptr(k_global_scale, dev), _scale_ptr(v_global_scale, dev), rows, cu, lens, table,
             batch, max_pages, _dense("k_out", k_out, torch.bfloat16, out_shape, dev),
             _dense("v_out", v_out, torch.bfloat16, out_shape, dev)))
    return k_out, v_out


def attention_cache_workspace_bytes(max_rows: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Device workspace bytes of h3q_attention_cache_nvfp4 (h3q_attention_cache_workspace_bytes in
    include/h3q.h)."""
    shared = max_rows * (heads // kv_heads)
    tile = 8 if shared <= 8 else 16 if shared <= 16 or head_dim == 256 else 32
    return 608 * (64 + 2 * tile * (head_dim + 2) * 4)


def _softmax_scale(scale, dim) -> float:
    """The scale, head_dim ** -0.5 when not given (any for a head_dim that the call refuses)."""
    return float(scale) if scale is not None else dim ** -0.5 if dim else 1.0


def _workspace(workspace, nbytes, device, fresh):
    """The caller's workspace, or one that joins the fresh tensors."""
    torch = _torch or _load_torch()
    if workspace is not None:
        _cuda_tensor("workspace", workspace, torch.uint8, device)
        if not workspace.is_contiguous() or workspace.numel() < nbytes:
            raise ValueError(f"workspace must be contiguous with at least {nbytes} bytes")
        return workspace
    fresh.append(torch.empty(nbytes, dtype=torch.uint8, device=device))
    return fresh[-1]


def h3q_attention_cache_nvfp4(q, cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale, *, max_rows=None,
                              tree_mask=None, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens over the paged NVFP4 cache that holds their context and, at its
    end, themselves (written before with the same lists).

    ``q`` is bf16 [rows, heads, head_dim] (contiguous rows of any stride), heads a multiple of the
    cache's.  Every sequence has at most ``max_rows`` (1 .. 64) new tokens; more of one are not computed.
    It need not be given for one token a sequence, that is, for no more rows than sequences.  ``tree_mask`` (int64
    [rows]): bit j says that the token sees token j of its sequence; without it a token sees itself
    and those before.  ``scale`` defaults to head_dim ** -0.5.  ``lse`` (fp32 [heads, rows], optional)
    receives the log of the sums of exponentials.  ``workspace`` (uint8, at least
    attention_cache_workspace_bytes) is allocated when not given.  Returns out, bf16 [rows, heads,
    head_dim]; rows of no sequence are left as they were."""
    torch = _torch or _load_torch()
    if len(getattr(q, "shape", ())) != 3:
        _head_rows("q", q)
    q_shape = q.shape
    rows, heads, dim = q_shape
    dev = q.device
    if max_rows is None:
        if isinstance(kv_len, torch.Tensor) and kv_len.dim() == 1 and rows > kv_len.shape[0]:
            raise ValueError(f"q has {rows} rows for {kv_len.shape[0]} sequences: give max_rows, the most new tokens "
                             "that one has")
        max_rows = 1
    max_rows = int(max_rows)
    scale = _softmax_scale(scale, dim)
    fresh = []
    if out is None:
        out = torch.empty(q_shape, dtype=torch.bfloat16, device=dev)
        fresh.append(out)
    if len(cache) != 4 or len(getattr(cache[0], "shape", ())) != 4:
        _cache(cache)
    kv_heads = cache[0].shape[1]
    # (a number of heads that the call refuses needs no workspace to be refused)
    nbytes = attention_cache_workspace_bytes(max_rows, heads, kv_heads, dim) if kv_heads and heads >= kv_heads else 256
    workspace = _workspace(workspace, nbytes, dev, fresh)
    _lend(stream, dev, fresh)
    rc = _native.cached(q, cache, cu_rows, kv_len, block_table, k_global_scale, v_global_scale, max_rows, tree_mask,
                        scale, out, lse, workspace, dev, _handle(stream))
    if rc is not None:
        if rc != H3Q_OK:
            raise H3QError("h3q_attention_cache_nvfp4", rc, h3q_last_error())
        return out
    ptrs, shape, dev = _cache(cache)
    qp, q_shape, ld = _head_rows("q", q, dev)
    if dim != shape[3]:
        raise ValueError(f"q has head_dim {dim}, the cache {shape[3]}")
    cu, lens, table, batch, max_pages = _row_lists(cu_rows, kv_len, block_table, dev)
    mask_ptr = _dense("tree_mask", tree_mask, torch.int64, (rows,), dev) if tree_mask is not None else None
    lse_ptr = _dense("lse", lse, torch.float32, (heads, rows), dev) if lse is not None else None
    out_ptr = _dense("out", out, torch.bfloat16, q_shape, dev)
    _invoke("h3q_attention_cache_nvfp4", dev, stream,
            (qp, ld, rows, heads, max_rows, cu, lens, table, batch, max_pages, mask_ptr, *ptrs, *shape,
             _scale_ptr(k_global_scale, dev), _scale_ptr(v_global_scale, dev), scale, out_ptr, lse_ptr,
             workspace.data_ptr(), workspace.numel()))
    return out


def h3q_attention_varlen(q, k, v, cu_q, cu_k, *, causal=True, scale=None, out=None, lse=None, stream=None):
    """Softmax attention over packed sequences: q bf16 [rows_q, heads, head_dim], k and v bf16
    [rows_k, kv_heads, head_dim] (contiguous rows of any stride; heads a multiple of kv_heads).
    Sequence b has queries cu_q[b] .. cu_q[b+1]-1 and keys cu_k[b] .. cu_k[b+1]-1 (int32 CUDA tensors);
    with ``causal`` its last query sees its last key and every query one fewer than the next.
    ``scale`` defaults to head_dim ** -0.5.  ``lse`` (fp32 [heads, rows_q], optional) receives the log
    of the sums of exponentials.  Returns out, bf16 [rows_q, heads, head_dim]; rows of no sequence are
    left as they were."""
    torch = _torch or _load_torch()
    if len(getattr(q, "shape", ())) != 3:
        _head_rows("q", q)
    q_shape, dev = q.shape, q.device
    scale = _softmax_scale(scale, q_shape[2])
    if out is None:
        out = torch.empty(q_shape, dtype=torch.bfloat16, device=dev)
        _lend(stream, dev, [out])
    causal = bool(causal)
    rc = _native.varlen(q, k, v, cu_q, cu_k, causal, scale, out, lse, dev, _handle(stream))
    if rc is not None:
        if rc != H3Q_OK:
            raise H3QError("h3q_attention_varlen", rc, h3q_last_error())
        return out
    qp, q_shape, ld_q = _head_rows("q", q)
    kp, k_shape, ld_k = _head_rows("k", k, dev)
    vp, v_shape, ld_v = _head_rows("v", v, dev)
    rows_q, heads, dim = q_shape
    rows_k, kv_heads, dim_k = k_shape
    if dim_k != dim or v_shape != k_shape:
        raise ValueError("k and v must have the same shape, and q's head_dim")
    if not (isinstance(cu_q, torch.Tensor) and cu_q.dim() == 1 and cu_q.shape[0] >= 1):
        _cuda_tensor("cu_q", cu_q, torch.int32, dev)
        raise ValueError("cu_q must be contiguous [batch + 1]")
    lists = cu_q.shape
    cu_q_ptr = _dense("cu_q", cu_q, torch.int32, lists, dev)
    cu_k_ptr = _dense("cu_k", cu_k, torch.int32, lists, dev)
    out_ptr = _dense("out", out, torch.bfloat16, q_shape, dev)
    lse_ptr = _dense("lse", lse, torch.float32, (heads, rows_q), dev) if lse is not None else None
    _invoke("h3q_attention_varlen", dev, stream,
            (qp, ld_q, kp, ld_k, vp, ld_v, cu_q_ptr, cu_k_ptr, lists[0] - 1, rows_q, rows_k, heads, kv_heads, dim,
             int(causal), scale, out_ptr, lse_ptr))
    return out


def _per_axis(name, value, axes):
    """A number for all axes, or one for each, as a C array of doubles."""
    values = [float(x) for x in value] if isinstance(value, (list, tuple)) else [float(value)] * axes
    if len(values) != axes:
        raise ValueError(f"{name} must be a number, or one for each axis")
    return (ctypes.c_double * axes)(*values)


def h3q_qkv_epilogue_axes(q, k, v, positions, axis_dims, heads, *, kv_heads=None, theta=10000.0, scale=1.0, sections=False,
                          biases=None, weights=None, norm=True, eps=1e-6, interleaved=False, outs=None, stream=None):
    """QKV epilogue with rotary positions of several axes: projected q [rows, heads * HD] and k, v
    [rows, kv_heads * HD] bf16 (contiguous rows of any stride; ``kv_heads`` defaults to ``heads``) ->
    (q_out, k_out, v_out), bf16 [rows, heads or kv_heads, HD].  q and k are biased, RMS-normed
    per head (``norm``) and turned by the angles of ``positions`` (int32 [rows, axes], e.g. time, height,
    width), v is biased.  ``axis_dims`` are the values of a head that turn with each axis, in order; pair i of
    an axis of d values turns by scale * theta ** (-2 i / d) a step (``theta`` and ``scale``: a number, or one
    per axis), or with ``sections`` pair j of all by scale * theta ** (-2 j / sum(axis_dims)).  Pairs are
    (j, j + sum / 2), or (2j, 2j + 1) with ``interleaved``.  ``biases`` (of q, k and v) and ``weights`` (of
    q's and k's norm, [HD]) are tuples of bf16 tensors, any of them None."""
    torch = _torch or _load_torch()
    if kv_heads is None:
        kv_heads = heads
    shape = getattr(q, "shape", ())
    if len(shape) == 2 and heads > 0 and kv_heads > 0:
        dev, fresh = q.device, outs
        if fresh is None:
            rows, size, empty, bf16 = shape[0], shape[1] // heads, torch.empty, torch.bfloat16
            fresh = (empty((rows, heads, size), dtype=bf16, device=dev), empty((rows, kv_heads, size), dtype=bf16, device=dev),
                     empty((rows, kv_heads, size), dtype=bf16, device=dev))
            if stream is not None:
                _lend(stream, dev, fresh)
        rc = _native.axes(q, k, v, positions, axis_dims, heads, kv_heads, theta, scale, sections, biases, weights, norm,
                          eps, interleaved, fresh, dev, None if stream is None else _handle(stream))
        if rc == H3Q_OK:
            return fresh if outs is None else tuple(fresh)
        if rc is not None:
            raise H3QError("h3q_qkv_epilogue_axes", rc, h3q_last_error())
    q, rows, d, ld_q = _rows_view("q", q, torch.bfloat16)
    dev = q.device
    k, rows_k, d_k, ld_k = _rows_view("k", k, torch.bfloat16, dev)
    v, rows_v, d_v, ld_v = _rows_view("v", v, torch.bfloat16, dev)
    if heads < 1 or kv_heads < 1 or d % heads:
        raise ValueError("the columns of q must split into heads")
    hd = d // heads
    if (rows_k, d_k) != (rows, kv_heads * hd) or (rows_v, d_v) != (rows, kv_heads * hd):
        raise ValueError("k and v must have q's rows and kv_heads heads of q's size")
    axes = len(axis_dims)
    positions_ptr = _dense("positions", positions, torch.int32, (rows, axes), dev)
    b = [None if t is None else _dense(n, t, torch.bfloat16, (c,), dev)
         for n, t, c in zip(("bias_q", "bias_k", "bias_v"), biases or (None,) * 3, (d, d_k, d_k))]
    w = [None if t is None else _dense(n, t, torch.bfloat16, (hd,), dev)
         for n, t in zip(("weight_q", "weight_k"), weights or (None,) * 2)]
    if outs is None:
        outs = [torch.empty((rows, h, hd), dtype=torch.bfloat16, device=dev) for h in (heads, kv_heads, kv_heads)]
        _lend(stream, dev, outs)
    o = [_dense(n, t, torch.bfloat16, (rows, h, hd), dev)
         for n, t, h in zip(("q_out", "k_out", "v_out"), outs, (heads, kv_heads, kv_heads))]
    _invoke("h3q_qkv_epilogue_axes", dev, stream,
            (q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, *b, *w, positions_ptr, axes,
             (_I64 * axes)(*axis_dims), _per_axis("theta", theta, axes), _per_axis("scale", scale, axes),
             int(bool(sections)), int(bool(interleaved)), int(bool(norm)), rows, heads, kv_heads, hd, float(eps), *o))
    return outs[0], outs[1], outs[2]


def h3q_postnorm_residual_adaln_nvfp4(h, o, gamma_post, gamma, global_scale, *, bias=None, gate_table=None,
                                      mod_table=None, residual_scale=1.0, row_frame=None, rows_per_frame=None, eps=1e-6,
                                      codes=None, scales=None, row_rstd=None, stream=None):
    """The norm after a block, its gate and scaled residual, the norm before the next block -> NVFP4:
    h (fp32 [rows, cols], updated in place) = residual_scale * h + gate_table[frame] * RMSNorm(bf16(o + bias)) *
    gamma_post, then RMSNorm(h) * gamma with the modulation of ``mod_table`` (bf16 [frames, 2, cols]: [t, 0] shift,
    [t, 1] scale).  ``gate_table`` (bf16 [frames, cols]), ``mod_table`` and ``bias`` may be None; with a
    table the frame of a row is ``row_frame[row]`` (int32 CUDA tensor) or ``row // rows_per_frame``.
    ``row_rstd`` (fp32 [rows], optional) receives the rstd of the new h.  Returns (codes, scales)."""
    torch = _torch or _load_torch()
    shape = getattr(h, "shape", ())
    if len(shape) == 2:
        dev, u8, to_codes, to_scales = h.device, torch.uint8, codes, scales
        rows, cols = shape
        if to_codes is None:
            to_codes = torch.empty((rows, cols // 2), dtype=u8, device=dev)
        if to_scales is None:
            to_scales = torch.empty(((rows + 127) // 128 * 128, cols // 16), dtype=u8, device=dev)
        if stream is not None:
            _lend(stream, dev, [t for t, given in ((to_codes, codes), (to_scales, scales)) if given is None])
        rc = _native.postnorm(h, o, gamma_post, gamma, global_scale, bias, gate_table, mod_table, residual_scale,
                              row_frame, rows_per_frame, eps, to_codes, to_scales, row_rstd, dev,
                              None if stream is None else _handle(stream))
        if rc == H3Q_OK:
            return to_codes, to_scales
        if rc is not None:
            raise H3QError("h3q_postnorm_residual_adaln_nvfp4", rc, h3q_last_error())
    _cuda_tensor("h", h, torch.float32)
    dev = h.device
    if h.dim() != 2 or (h.shape[1] > 1 and h.stride(1) != 1):
        raise ValueError("h must be 2-D with contiguous rows")
    rows, cols = h.shape
    ld_h = h.stride(0) if rows > 1 else cols
    o, rows_o, cols_o, ld_o = _rows_view("o", o, torch.bfloat16, dev)
    if (rows_o, cols_o) != (rows, cols):
        raise ValueError("o must have the shape of h")
    vector = (cols,)
    bias_ptr = _dense("bias", bias, torch.bfloat16, vector, dev) if bias is not None else None
    post_ptr = _dense("gamma_post", gamma_post, torch.bfloat16, vector, dev)
    gamma_ptr = _dense("gamma", gamma, torch.bfloat16, vector, dev)
    frames, gate_ptr, table_ptr, rf_ptr = 0, None, None, None
    if gate_table is not None:
        _cuda_tensor("gate_table", gate_table, torch.bfloat16, dev)
        if gate_table.dim() != 2 or gate_table.shape[1] != cols or not gate_table.is_contiguous():
            raise ValueError("gate_table must be contiguous [frames, cols]")
        frames, gate_ptr = gate_table.shape[0], gate_table.data_ptr()
    if mod_table is not None:
        _cuda_tensor("mod_table", mod_table, torch.bfloat16, dev)
        if (mod_table.dim() != 3 or mod_table.shape[1:] != (2, cols) or not mod_table.is_contiguous()
                or (gate_table is not None and mod_table.shape[0] != frames)):
            raise ValueError("mod_table must be contiguous [frames, 2, cols], frames as gate_table")
        frames, table_ptr = mod_table.shape[0], mod_table.data_ptr()
    if gate_ptr is not None or table_ptr is not None:
        if row_frame is not None:
            rf_ptr = _dense("row_frame", row_frame, torch.int32, (rows,), dev)
            rows_per_frame = 0
        elif rows_per_frame is None:
            raise ValueError("give row_frame or rows_per_frame")
    rstd_ptr = _dense("row_rstd", row_rstd, torch.float32, (rows,), dev) if row_rstd is not None else None
    codes, scales = _outputs(dev, rows, cols, codes, scales, stream)
    _invoke("h3q_postnorm_residual_adaln_nvfp4", dev, stream,
            (h.data_ptr(), ld_h, o.data_ptr(), ld_o, bias_ptr, post_ptr, gate_ptr, float(residual_scale), gamma_ptr,
             table_ptr, frames, rf_ptr, int(rows_per_frame or 0), float(eps), rows, cols, _scale_ptr(global_scale, dev),
             codes.data_ptr(), scales.data_ptr(), rstd_ptr))
    return codes, scales


def block_rows(rows: int, batch: int, block: int) -> int:
    """Rows of the lists of blocks (h3q_block_rows in include/h3q.h): query block i of sequence b has row
    cu[b] // block + b + i."""
    return rows // block + batch


def select_blocks_workspace_bytes(rows_q, rows_k, batch, kv_heads, head_dim, block_q, block_k) -> int:
    """Device workspace bytes of h3q_select_blocks (h3q_select_blocks_workspace_bytes in include/h3q.h)."""
    keys, lists = block_rows(rows_k, batch, block_k), block_rows(rows_q, batch, block_q)
    nbytes = (lists + keys) * kv_heads * (head_dim + 1) * 8 + (keys * kv_heads + 7) // 8 * 8 * head_dim * 4 + 256
    if rows_k // block_k > 16000:   # rows of scores
        nbytes += min(lists * kv_heads, 1024) * ((rows_k // block_k + 32) // 32 * 32) * 4
    return nbytes


def _block_sequences(q, k, cu_q, cu_k):
    """Checks what the calls over blocks share; returns (q, ld_q, k, ld_k, cu_q, cu_k, batch, rows_q, rows_k, heads,
    kv_heads, dim, device)."""
    torch = _torch
    qp, (rows_q, heads, dim), ld_q = _head_rows("q", q)
    dev = q.device
    kp, (rows_k, kv_heads, dim_k), ld_k = _head_rows("k", k, dev)
    if dim_k != dim:
        raise ValueError("k must have q's head_dim")
    if not (isinstance(cu_q, torch.Tensor) and cu_q.dim() == 1 and cu_q.shape[0] >= 1):
        _cuda_tensor("cu_q", cu_q, torch.int32, dev)
        raise ValueError("cu_q must be contiguous [batch + 1]")
    lists = cu_q.shape
    return (qp, ld_q, kp, ld_k, _dense("cu_q", cu_q, torch.int32, lists, dev),
            _dense("cu_k", cu_k, torch.int32, lists, dev), lists[0] - 1, rows_q, rows_k, heads, kv_heads, dim, dev)


def h3q_select_blocks(q, k, cu_q, cu_k, top, *, block_q=128, block_k=128, causal=False, first=0, blocks=None, scores=None,
                      workspace=None, stream=None):
    """The key blocks that each query block of packed sequences attends to: int32 [kv_heads,
    block_rows(rows_q, batch, block_q), top], ascending, then -1 -- the ``top`` blocks with the highest scores
    mean(queries of the block and group) . mean(keys of the block), ties to the lowest numbers; always the
    ``first`` blocks and, with ``causal``, those of the query block's own positions.  q bf16
    [rows_q, heads, head_dim], k bf16 [rows_k, kv_heads, head_dim] and cu_q, cu_k as h3q_attention_varlen
    takes them.  ``scores`` (fp32 of the lists' shape, optional) receives the entries' scores.  Where
    ``workspace`` (uint8, select_blocks_workspace_bytes) is not given it is allocated.  Returns the lists."""
    torch = _torch or _load_torch()
    if block_q < 1 or block_k < 1:
        raise ValueError("block_q and block_k must be 64, 128 or 256")
    if not 1 <= top <= 4096:
        raise ValueError("top must be in [1, 4096]")
    if (len(getattr(q, "shape", ())) != 3 or len(getattr(k, "shape", ())) != 3 or len(getattr(cu_q, "shape", ())) != 1
            or cu_q.shape[0] < 1):
        _block_sequences(q, k, cu_q, cu_k)
    (rows_q, _, dim), (rows_k, kv_heads, _), batch, dev = q.shape, k.shape, cu_q.shape[0] - 1, q.device
    shape = (kv_heads, block_rows(rows_q, batch, block_q), int(top))
    fresh = []
    if blocks is None:
        blocks = torch.empty(shape, dtype=torch.int32, device=dev)
        fresh.append(blocks)
    nbytes = select_blocks_workspace_bytes(rows_q, rows_k, batch, kv_heads, dim, block_q, block_k)
    workspace = _workspace(workspace, nbytes, dev, fresh)
    _lend(stream, dev, fresh)
    rc = _native.select(q, k, cu_q, cu_k, top, block_q, block_k, causal, first, blocks, scores, workspace, dev,
                        _handle(stream))
    if rc is not None:
        if rc != H3Q_OK:
            raise H3QError("h3q_select_blocks", rc, h3q_last_error())
        return blocks
    qp, ld_q, kp, ld_k, cu_q_ptr, cu_k_ptr, batch, rows_q, rows_k, heads, kv_heads, dim, dev = _block_sequences(
        q, k, cu_q, cu_k)
    blocks_ptr = _dense("blocks", blocks, torch.int32, shape, dev)
    scores_ptr = _dense("scores", scores, torch.float32, shape, dev) if scores is not None else None
    _invoke("h3q_select_blocks", dev, stream,
            (qp, ld_q, kp, ld_k, cu_q_ptr, cu_k_ptr, batch, rows_q, rows_k, heads, kv_heads, dim, block_q, block_k,
             shape[2], int(bool(causal)), int(first), blocks_ptr, scores_ptr, workspace.data_ptr(),
             workspace.numel()))
    return blocks


def h3q_attention_blocks(q, k, v, cu_q, cu_k, blocks, *, block_q=128, block_k=128, causal=False, scale=None, out=None,
                         lse=None, stream=None):
    """Softmax attention as h3q_attention_varlen's over the key blocks that ``blocks`` (int32 [kv_heads,
    block_rows(rows_q, batch, block_q), top], as h3q_select_blocks makes them) lists for each query block: entries
    that are no block of the sequence, or not above those before them, are passed over.  head_dim 64 or 128.
    ``lse`` (fp32 [heads, rows_q], optional) receives the log of the sums of exponentials.  Returns out, bf16
    [rows_q, heads, head_dim]; rows of no sequence are left as they were."""
    torch = _torch or _load_torch()
    shape = getattr(q, "shape", ())
    if len(shape) == 3:
        dev, fresh = q.device, out
        if fresh is None:
            fresh = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            _lend(stream, dev, [fresh])
        rc = _native.blocks(q, k, v, cu_q, cu_k, blocks, block_q, block_k, causal, _softmax_scale(scale, shape[2]), fresh,
                            lse, dev, _handle(stream))
        if rc is not None:
            if rc != H3Q_OK:
                raise H3QError("h3q_attention_blocks", rc, h3q_last_error())
            return fresh
    qp, ld_q, kp, ld_k, cu_q_ptr, cu_k_ptr, batch, rows_q, rows_k, heads, kv_heads, dim, dev = _block_sequences(
        q, k, cu_q, cu_k)
    vp, v_shape, ld_v = _head_rows("v", v, dev)
    if v_shape != k.shape:
        raise ValueError("k and v must have the same shape")
    if block_q < 1 or block_k < 1:
        raise ValueError("block_q and block_k must be 64, 128 or 256")
    _cuda_tensor("blocks", blocks, torch.int32, dev)
    rows = block_rows(rows_q, batch, block_q)
    if blocks.dim() != 3 or tuple(blocks.shape[:2]) != (kv_heads, rows) or not blocks.is_contiguous():
        raise ValueError(f"blocks must be contiguous [{kv_heads}, {rows}, top], got {tuple(blocks.shape)}")
    if out is None:
        out = torch.empty((rows_q, heads, dim), dtype=torch.bfloat16, device=dev)
        _lend(stream, dev, [out])
    out_ptr = _dense("out", out, torch.bfloat16, (rows_q, heads, dim), dev)
    lse_ptr = _dense("lse", lse, torch.float32, (heads, rows_q), dev) if lse is not None else None
    _invoke("h3q_attention_blocks", dev, stream,
            (qp, ld_q, kp, ld_k, vp, ld_v, cu_q_ptr, cu_k_ptr, batch, rows_q, rows_k, heads, kv_heads, dim, block_q,
             block_k, blocks.data_ptr(), blocks.shape[2], int(bool(causal)), _softmax_scale(scale, dim), out_ptr,
             lse_ptr))
    return out
