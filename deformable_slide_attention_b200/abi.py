"""ctypes binding over ``libdsa3d.so`` (declared in ``include/dsa3d.h``).

The ``dsa3d_*`` functions here carry the C names and take plain integers for pointers and the
stream; they only marshal arguments.  :func:`forward` and :func:`backward` are conveniences for
torch CUDA tensors: they validate shapes, allocate the outputs (and the backward workspace) with
torch's caching allocator and call the C entry points on the current stream.

There is no fallback: if the library is missing, or no CUDA device is present, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import operator
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdsa3d.so"
_lib = None
_lock = threading.Lock()

DSA3D_F32 = 0
DSA3D_BF16 = 1
DSA3D_SILU = 0
DSA3D_GELU = 1
_ACTIVATIONS = {"silu": DSA3D_SILU, "gelu": DSA3D_GELU}

_STATUS = {0: "DSA3D_OK", 1: "DSA3D_ERR_INVALID_ARGUMENT", 2: "DSA3D_ERR_UNSUPPORTED",
           3: "DSA3D_ERR_WORKSPACE_TOO_SMALL", 4: "DSA3D_ERR_CUDA", 5: "DSA3D_ERR_DEVICE_CHECK"}


class Dsa3dError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)} ({dsa3d_status_string(status)})")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m "
                               "deformable_slide_attention_b200.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        I, Z, P = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        dims = [I] * 8
        lib.dsa3d_abi_version.restype = I
        lib.dsa3d_abi_version.argtypes = []
        lib.dsa3d_status_string.restype = ctypes.c_char_p
        lib.dsa3d_status_string.argtypes = [I]
        lib.dsa3d_forward.restype = I
        lib.dsa3d_forward.argtypes = [P, P, P, P, P, P, P, Z, *dims, I, P]
        lib.dsa3d_forward_workspace_bytes.restype = Z
        lib.dsa3d_forward_workspace_bytes.argtypes = [*dims, I]
        lib.dsa3d_backward_workspace_bytes.restype = Z
        lib.dsa3d_backward_workspace_bytes.argtypes = [*dims, I]
        lib.dsa3d_backward.restype = I
        lib.dsa3d_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, Z, *dims, I, P]
        lib.dsa3d_backward_noalloc.restype = I
        lib.dsa3d_backward_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, P, *dims, I, P]
        lib.dsa3d_forward_taps.restype = I
        lib.dsa3d_forward_taps.argtypes = [P, P, P, P, P, P, *dims, I, P]
        lib.dsa3d_backward_taps_workspace_bytes.restype = Z
        lib.dsa3d_backward_taps_workspace_bytes.argtypes = [*dims, I]
        lib.dsa3d_backward_taps.restype = I
        lib.dsa3d_backward_taps.argtypes = [P, P, P, P, P, P, P, P, P, P, P, Z, *dims, I, P]
        cdims = [I] * 7  # F, Hp, Wp, C, kt, kh, kw
        lib.dsa3d_dwconv3d.restype = I
        lib.dsa3d_dwconv3d.argtypes = [P, P, P, P, P, *cdims, I, P]
        lib.dsa3d_dwconv3d_backward.restype = I
        lib.dsa3d_dwconv3d_backward.argtypes = [P, P, P, P, P, P, *cdims, I, P]
        lib.dsa3d_offset_head_workspace_bytes.restype = Z
        lib.dsa3d_offset_head_workspace_bytes.argtypes = [I, I, I, I]
        lib.dsa3d_offset_head.restype = I
        lib.dsa3d_offset_head.argtypes = [P, P, P, P, P, P, P, Z, I, I, I, I, I, I, I, I, I, I, P]
        lib.dsa3d_offset_head_backward_workspace_bytes.restype = Z
        lib.dsa3d_offset_head_backward_workspace_bytes.argtypes = [I, I, I, I]
        lib.dsa3d_offset_head_backward.restype = I
        lib.dsa3d_offset_head_backward.argtypes = [P] * 11 + [Z] + [I] * 10 + [P]
        L, FL, D = ctypes.c_longlong, ctypes.c_float, ctypes.c_double
        lib.dsa3d_layer_norm.restype = I
        lib.dsa3d_layer_norm.argtypes = [P] * 7 + [L, I, FL, I, P]
        lib.dsa3d_layer_norm_backward_workspace_bytes.restype = Z
        lib.dsa3d_layer_norm_backward_workspace_bytes.argtypes = [L, I, I]
        lib.dsa3d_layer_norm_backward.restype = I
        lib.dsa3d_layer_norm_backward.argtypes = [P] * 9 + [Z, L, I, I, P]
        for f in (lib.dsa3d_rotary3d, lib.dsa3d_rotary3d_backward):
            f.restype = I
            f.argtypes = [P] * 4 + [L] * 6 + [I] * 5 + [I * 3, D * 3, D * 3, D, I, I, P]
        lib.dsa3d_gated_ffn_workspace_bytes.restype = Z
        lib.dsa3d_gated_ffn_workspace_bytes.argtypes = [L, I, I, I]
        lib.dsa3d_gated_ffn.restype = I
        lib.dsa3d_gated_ffn.argtypes = [P] * 7 + [Z, L, I, I, I, I, P]
        lib.dsa3d_gated_ffn_backward_workspace_bytes.restype = Z
        lib.dsa3d_gated_ffn_backward_workspace_bytes.argtypes = [L, I, I, I]
        lib.dsa3d_gated_ffn_backward.restype = I
        lib.dsa3d_gated_ffn_backward.argtypes = [P] * 10 + [Z, L, I, I, I, I, P]
        lib.dsa3d_check_device.restype = I
        lib.dsa3d_check_device.argtypes = [P]
        lib.dsa3d_timing_enable.restype = I
        lib.dsa3d_timing_enable.argtypes = [I]
        lib.dsa3d_timing_read.restype = I
        lib.dsa3d_timing_read.argtypes = [ctypes.POINTER(KernelTime), I]
        lib.dsa3d_timing_reset.restype = None
        lib.dsa3d_timing_reset.argtypes = []
        _lib = lib
        return lib


_INT3, _DBL3 = ctypes.c_int * 3, ctypes.c_double * 3


@functools.lru_cache(maxsize=256)
def _three(kind, values):
    """A C array of three numbers; the library only reads it."""
    return kind(*values)


def _axes(axes, start, step):
    return (_three(_INT3, tuple(map(operator.index, axes))), _three(_DBL3, tuple(map(float, start))),
            _three(_DBL3, tuple(map(float, step))))


class KernelTime(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("launches", ctypes.c_longlong),
                ("total_ms", ctypes.c_double)]


# --- the C entry points, one to one -----------------------------------------------------------
def dsa3d_abi_version() -> int:
    return _load().dsa3d_abi_version()


def dsa3d_status_string(status: int) -> str:
    try:
        return _load().dsa3d_status_string(int(status)).decode()
    except RuntimeError:
        return _STATUS.get(status, "unknown status")


def dsa3d_forward(q, k, v, offsets, out, lse, workspace, workspace_bytes, F, Hp, Wp, heads, dh,
                  kt, kh, kw, dtype, stream) -> int:
    return _load().dsa3d_forward(q, k, v, offsets, out, lse, workspace, workspace_bytes, F, Hp, Wp,
                                 heads, dh, kt, kh, kw, dtype, stream)


def dsa3d_forward_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype) -> int:
    return _load().dsa3d_forward_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype)


def dsa3d_backward_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype) -> int:
    return _load().dsa3d_backward_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype)


def dsa3d_backward(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets, workspace, workspace_bytes,
                   F, Hp, Wp, heads, dh, kt, kh, kw, dtype, stream) -> int:
    return _load().dsa3d_backward(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets, workspace,
                                  workspace_bytes, F, Hp, Wp, heads, dh, kt, kh, kw, dtype, stream)


def dsa3d_backward_noalloc(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets, F, Hp, Wp, heads,
                           dh, kt, kh, kw, dtype, stream) -> int:
    """The backward for callers that cannot allocate: its scratch is a fixed device array inside
    the library (see include/dsa3d.h)."""
    return _load().dsa3d_backward_noalloc(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets,
                                          F, Hp, Wp, heads, dh, kt, kh, kw, dtype, stream)


def dsa3d_forward_taps(q, k, v, offsets, out, lse, F, Hp, Wp, heads, dh, kt, kh, kw, dtype,
                       stream) -> int:
    """Forward with per-tap offsets ([heads][N][K][3])."""
    return _load().dsa3d_forward_taps(q, k, v, offsets, out, lse, F, Hp, Wp, heads, dh, kt, kh, kw,
                                      dtype, stream)


def dsa3d_backward_taps_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype) -> int:
    return _load().dsa3d_backward_taps_workspace_bytes(F, Hp, Wp, heads, dh, kt, kh, kw, dtype)


def dsa3d_backward_taps(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets, workspace,
                        workspace_bytes, F, Hp, Wp, heads, dh, kt, kh, kw, dtype, stream) -> int:
    """Backward with per-tap offsets; doffsets is [heads][N][K][3]."""
    return _load().dsa3d_backward_taps(q, k, v, offsets, lse, dout, dq, dk, dv, doffsets, workspace,
                                       workspace_bytes, F, Hp, Wp, heads, dh, kt, kh, kw, dtype,
                                       stream)


def dsa3d_dwconv3d(x, weight, bias, add, y, F, Hp, Wp, C, kt, kh, kw, dtype, stream) -> int:
    """The DWConv3D term of Eq. 1 (depthwise 3-D convolution, optional fused add)."""
    return _load().dsa3d_dwconv3d(x, weight, bias, add, y, F, Hp, Wp, C, kt, kh, kw, dtype, stream)


def dsa3d_dwconv3d_backward(x, weight, dy, dx, dweight, dbias, F, Hp, Wp, C, kt, kh, kw, dtype,
                            stream) -> int:
    return _load().dsa3d_dwconv3d_backward(x, weight, dy, dx, dweight, dbias, F, Hp, Wp, C, kt, kh,
                                           kw, dtype, stream)


def dsa3d_offset_head_workspace_bytes(F, Hp, Wp, C) -> int:
    return _load().dsa3d_offset_head_workspace_bytes(F, Hp, Wp, C)


def dsa3d_offset_head(x, dw_weight, dw_bias, pw_weight, pw_bias, offsets, workspace,
                      workspace_bytes, F, Hp, Wp, C, heads, taps, kt, kh, kw, dtype, stream) -> int:
    """The offset network's forward: depthwise conv then the pointwise layer, into offsets."""
    return _load().dsa3d_offset_head(x, dw_weight, dw_bias, pw_weight, pw_bias, offsets, workspace,
                                     workspace_bytes, F, Hp, Wp, C, heads, taps, kt, kh, kw, dtype,
                                     stream)


def dsa3d_offset_head_backward_workspace_bytes(F, Hp, Wp, C) -> int:
    return _load().dsa3d_offset_head_backward_workspace_bytes(F, Hp, Wp, C)


def dsa3d_offset_head_backward(x, dw_weight, dw_bias, pw_weight, doffsets, dx, d_dw_weight,
                               d_dw_bias, d_pw_weight, d_pw_bias, workspace, workspace_bytes, F,
                               Hp, Wp, C, heads, taps, kt, kh, kw, dtype, stream) -> int:
    return _load().dsa3d_offset_head_backward(x, dw_weight, dw_bias, pw_weight, doffsets, dx,
                                              d_dw_weight, d_dw_bias, d_pw_weight, d_pw_bias,
                                              workspace, workspace_bytes, F, Hp, Wp, C, heads, taps,
                                              kt, kh, kw, dtype, stream)


def dsa3d_layer_norm(x, add, weight, bias, y, h, stats, rows, C, eps, dtype, stream) -> int:
    """Layer norm over the channels, with an optional fused residual sum (h = x + add)."""
    return _load().dsa3d_layer_norm(x, add, weight, bias, y, h, stats, rows, C, eps, dtype, stream)


def dsa3d_layer_norm_backward_workspace_bytes(rows, C, dtype) -> int:
    return _load().dsa3d_layer_norm_backward_workspace_bytes(rows, C, dtype)


def dsa3d_layer_norm_backward(h, weight, stats, dy, add, dx, dweight, dbias, workspace, workspace_bytes,
                              rows, C, dtype, stream) -> int:
    return _load().dsa3d_layer_norm_backward(h, weight, stats, dy, add, dx, dweight, dbias, workspace,
                                             workspace_bytes, rows, C, dtype, stream)


def dsa3d_rotary3d(q, k, q_out, k_out, ldq, ldk, ldqo, ldko, first, rows, F, Hp, Wp, heads, dh, axes,
                   start, step, base, interleaved, dtype, stream) -> int:
    """Rotary positions of the token grid for q and k; axes, start and step are sequences of three."""
    return _load().dsa3d_rotary3d(q, k, q_out, k_out, ldq, ldk, ldqo, ldko, first, rows, F, Hp, Wp, heads,
                                  dh, *_axes(axes, start, step), base, interleaved, dtype, stream)


def dsa3d_rotary3d_backward(dq_out, dk_out, dq, dk, lddqo, lddko, lddq, lddk, first, rows, F, Hp, Wp, heads,
                            dh, axes, start, step, base, interleaved, dtype, stream) -> int:
    return _load().dsa3d_rotary3d_backward(dq_out, dk_out, dq, dk, lddqo, lddko, lddq, lddk, first, rows, F,
                                           Hp, Wp, heads, dh, *_axes(axes, start, step), base, interleaved, dtype,
                                           stream)


def dsa3d_gated_ffn_workspace_bytes(rows, C, hidden, dtype) -> int:
    return _load().dsa3d_gated_ffn_workspace_bytes(rows, C, hidden, dtype)


def dsa3d_gated_ffn(x, gate_weight, up_weight, down_weight, add, y, workspace, workspace_bytes, rows, C,
                    hidden, activation, dtype, stream) -> int:
    """y = (act(x Wg) * (x Wu)) Wd (+ add)."""
    return _load().dsa3d_gated_ffn(x, gate_weight, up_weight, down_weight, add, y, workspace, workspace_bytes,
                                   rows, C, hidden, activation, dtype, stream)


def dsa3d_gated_ffn_backward_workspace_bytes(rows, C, hidden, dtype) -> int:
    return _load().dsa3d_gated_ffn_backward_workspace_bytes(rows, C, hidden, dtype)


def dsa3d_gated_ffn_backward(x, gate_weight, up_weight, down_weight, dy, dx, dgate_weight, dup_weight,
                             ddown_weight, workspace, workspace_bytes, rows, C, hidden, activation, dtype,
                             stream) -> int:
    return _load().dsa3d_gated_ffn_backward(x, gate_weight, up_weight, down_weight, dy, dx, dgate_weight,
                                            dup_weight, ddown_weight, workspace, workspace_bytes, rows, C,
                                            hidden, activation, dtype, stream)


def dsa3d_check_device(stream) -> int:
    return _load().dsa3d_check_device(stream)


def dsa3d_timing_enable(enable: bool) -> int:
    return _load().dsa3d_timing_enable(1 if enable else 0)


def dsa3d_timing_read() -> dict:
    """{kernel name: (launches, total ms)} accumulated since the last reset."""
    buf = (KernelTime * 64)()
    n = _load().dsa3d_timing_read(buf, 64)
    return {buf[i].kernel.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(min(n, 64))}


def dsa3d_timing_reset() -> None:
    _load().dsa3d_timing_reset()


# --- torch conveniences -----------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return DSA3D_F32
    if t.dtype == torch.bfloat16:
        return DSA3D_BF16
    raise TypeError(f"3D-DSA takes float32 or bfloat16 tensors, got {t.dtype}")


def _stream_handle(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status, what):
    if status != 0:
        raise Dsa3dError(status, what)


def _need(t, name, shape, dtype):
    """t must be a contiguous tensor of exactly this shape and dtype: the C ABI takes plain
    pointers and reads sizes from the extents, so a mismatched tensor would be read past its end."""
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(ref, *ts):
    """Every tensor given must be a CUDA tensor on ref's device."""
    for t in (ref, *ts):
        if t is not None and (not t.is_cuda or t.device != ref.device):
            raise ValueError("tensors must be CUDA tensors on one device")


def _workspace(ws):
    if ws is not None:
        torch = _torch()
        if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.dim() != 1:
            raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    return ws


def _shapes(q, offsets, dims, taps=None):
    """N, heads, dh; offsets must be [heads][N][3], or [heads][N][taps][3] when taps is given."""
    F, Hp, Wp = dims
    N = F * Hp * Wp
    if q.dim() != 3 or q.shape[0] != N:
        raise ValueError(f"q must be [N={N}][heads][dh], got {tuple(q.shape)}")
    heads, dh = q.shape[1], q.shape[2]
    want = (heads, N, 3) if taps is None else (heads, N, taps, 3)
    if tuple(offsets.shape) != want:
        raise ValueError(f"offsets must be {want}, got {tuple(offsets.shape)}")
    return N, heads, dh


def forward(q, k, v, offsets, dims, window, out=None, lse=None, stream=None, want_lse=True,
            workspace="auto"):
    """3D-DSA forward on CUDA tensors.  Returns (out [N][heads][dh], lse [heads][N] or None).

    workspace: "auto" allocates what dsa3d_forward_workspace_bytes asks for (the sorted
    tensor-core path where the shape has one); None runs the general CUDA-core kernel; a uint8
    CUDA tensor is used as given.
    """
    torch = _torch()
    N, heads, dh = _shapes(q, offsets, dims)
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.shape, q.dtype)
    _need(offsets, "offsets", offsets.shape, torch.float32)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.shape, q.dtype)
    if lse is None and want_lse:
        lse = torch.empty((heads, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (heads, N), torch.float32)
    if isinstance(workspace, str):
        need = dsa3d_forward_workspace_bytes(*dims, heads, dh, *window, code)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _on_device(q, k, v, offsets, out, lse, _workspace(workspace))
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(dsa3d_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets.data_ptr(), out.data_ptr(),
                         lse.data_ptr() if lse is not None else None, ws_ptr, ws_bytes, *dims, heads,
                         dh, *window, code, _stream_handle(stream)), "dsa3d_forward")
    return out, lse


def backward(q, k, v, offsets, lse, dout, dims, window, workspace=None, stream=None, grads=None):
    """3D-DSA backward on CUDA tensors.  Returns (dq, dk, dv, doffsets)."""
    torch = _torch()
    N, heads, dh = _shapes(q, offsets, dims)
    code = _dtype_code(q)
    _check_backward_tensors(q, k, v, offsets, lse, dout, heads, N)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(offsets))
    dq, dk, dv, doff = grads
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, q.shape, q.dtype)
    _need(doff, "doffsets", offsets.shape, torch.float32)
    need = dsa3d_backward_workspace_bytes(*dims, heads, dh, *window, code)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _on_device(q, k, v, offsets, lse, dout, dq, dk, dv, doff, _workspace(workspace))
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(dsa3d_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets.data_ptr(),
                          lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                          doff.data_ptr(), ws_ptr, ws_bytes, *dims, heads, dh, *window, code,
                          _stream_handle(stream)), "dsa3d_backward")
    return dq, dk, dv, doff


def _check_backward_tensors(q, k, v, offsets, lse, dout, heads, N):
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", dout)):
        _need(t, name, q.shape, q.dtype)
    _need(offsets, "offsets", offsets.shape, torch.float32)
    _need(lse, "lse", (heads, N), torch.float32)


def _taps(window):
    kt, kh, kw = window
    return kt * kh * kw


def forward_taps(q, k, v, offsets, dims, window, out=None, lse=None, stream=None, want_lse=True):
    """3D-DSA forward with per-tap offsets ([heads][N][kt*kh*kw][3]) on CUDA tensors.
    Returns (out [N][heads][dh], lse [heads][N] or None)."""
    torch = _torch()
    N, heads, dh = _shapes(q, offsets, dims, _taps(window))
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.shape, q.dtype)
    _need(offsets, "offsets", offsets.shape, torch.float32)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.shape, q.dtype)
    if lse is None and want_lse:
        lse = torch.empty((heads, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (heads, N), torch.float32)
    _on_device(q, k, v, offsets, out, lse)
    _check(dsa3d_forward_taps(q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets.data_ptr(),
                              out.data_ptr(), lse.data_ptr() if lse is not None else None, *dims,
                              heads, dh, *window, code, _stream_handle(stream)), "dsa3d_forward_taps")
    return out, lse


def backward_taps(q, k, v, offsets, lse, dout, dims, window, workspace=None, stream=None, grads=None):
    """3D-DSA backward with per-tap offsets.  Returns (dq, dk, dv, doffsets [heads][N][K][3])."""
    torch = _torch()
    N, heads, dh = _shapes(q, offsets, dims, _taps(window))
    code = _dtype_code(q)
    _check_backward_tensors(q, k, v, offsets, lse, dout, heads, N)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(offsets))
    dq, dk, dv, doff = grads
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, q.shape, q.dtype)
    _need(doff, "doffsets", offsets.shape, torch.float32)
    need = dsa3d_backward_taps_workspace_bytes(*dims, heads, dh, *window, code)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _on_device(q, k, v, offsets, lse, dout, dq, dk, dv, doff, _workspace(workspace))
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(dsa3d_backward_taps(q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets.data_ptr(),
                               lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                               dv.data_ptr(), doff.data_ptr(), ws_ptr, ws_bytes, *dims, heads, dh,
                               *window, code, _stream_handle(stream)), "dsa3d_backward_taps")
    return dq, dk, dv, doff


def _conv_shapes(x, weight, dims):
    """(C, kt, kh, kw) of a convolution call; x must be [N][C] with N = F*Hp*Wp and weight
    [C][kt][kh][kw] fp32, both contiguous."""
    torch = _torch()
    N = dims[0] * dims[1] * dims[2]
    if x.dim() != 2 or x.shape[0] != N:
        raise ValueError(f"x must be [N={N}][C], got {tuple(x.shape)}")
    _need(x, "x", x.shape, x.dtype)
    C = x.shape[1]
    if weight.dim() != 4 or weight.shape[0] != C:
        raise ValueError(f"weight must be [C={C}][kt][kh][kw], got {tuple(weight.shape)}")
    _need(weight, "weight", weight.shape, torch.float32)
    return (C, *weight.shape[1:])


def dwconv3d(x, weight, bias, dims, add=None, out=None, stream=None):
    """Depthwise 3-D convolution of x [N][C] with weight [C][kt][kh][kw] (fp32) and bias [C]
    (fp32 or None), plus add [N][C] if given (the attention output viewed as [N][C]; out may be
    add itself).  Returns out [N][C]."""
    torch = _torch()
    code = _dtype_code(x)
    C, kt, kh, kw = _conv_shapes(x, weight, dims)
    if bias is not None:
        _need(bias, "bias", (C,), torch.float32)
    if add is not None:
        _need(add, "add", x.shape, x.dtype)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.shape, x.dtype)
    _on_device(x, weight, bias, add, out)
    _check(dsa3d_dwconv3d(x.data_ptr(), weight.data_ptr(), bias.data_ptr() if bias is not None else None,
                          add.data_ptr() if add is not None else None, out.data_ptr(), *dims, C, kt,
                          kh, kw, code, _stream_handle(stream)), "dsa3d_dwconv3d")
    return out


def dwconv3d_backward(x, weight, dy, dims, stream=None):
    """Gradients of sum(dwconv3d(x, weight, bias) * dy): (dx [N][C], dweight, dbias [C] fp32)."""
    torch = _torch()
    code = _dtype_code(x)
    C, kt, kh, kw = _conv_shapes(x, weight, dims)
    _need(dy, "dy", x.shape, x.dtype)
    _on_device(x, weight, dy)
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight, dtype=torch.float32)
    db = torch.empty(x.shape[1], dtype=torch.float32, device=x.device)
    _check(dsa3d_dwconv3d_backward(x.data_ptr(), weight.data_ptr(), dy.data_ptr(), dx.data_ptr(),
                                   dw.data_ptr(), db.data_ptr(), *dims, C, kt, kh, kw, code,
                                   _stream_handle(stream)), "dsa3d_dwconv3d_backward")
    return dx, dw, db


def offset_head(x, dw_weight, dw_bias, pw_weight, pw_bias, dims, heads, per_tap=False, stream=None):
    """The offset network's forward on CUDA tensors: offsets [heads][N][3] (or [heads][N][K][3]
    with per_tap) from x [N][C], dw_weight [C][kt][kh][kw], dw_bias [C] or None, pw_weight
    [C][heads * (K) * 3] and pw_bias (fp32)."""
    torch = _torch()
    code = _dtype_code(x)
    C, kt, kh, kw = _conv_shapes(x, dw_weight, dims)
    taps = kt * kh * kw if per_tap else 1
    width = heads * taps * 3
    if dw_bias is not None:
        _need(dw_bias, "dw_bias", (C,), torch.float32)
    _need(pw_weight, "pw_weight", (C, width), torch.float32)
    _need(pw_bias, "pw_bias", (width,), torch.float32)
    N = x.shape[0]
    offsets = torch.empty((heads, N, taps, 3) if per_tap else (heads, N, 3), dtype=torch.float32,
                          device=x.device)
    ws = torch.empty(dsa3d_offset_head_workspace_bytes(*dims, C), dtype=torch.uint8, device=x.device)
    _on_device(x, dw_weight, dw_bias, pw_weight, pw_bias)
    _check(dsa3d_offset_head(x.data_ptr(), dw_weight.data_ptr(),
                             dw_bias.data_ptr() if dw_bias is not None else None,
                             pw_weight.data_ptr(), pw_bias.data_ptr(), offsets.data_ptr(),
                             ws.data_ptr(), ws.numel(), *dims, C, heads, taps, kt, kh, kw, code,
                             _stream_handle(stream)), "dsa3d_offset_head")
    return offsets


def offset_head_backward(x, dw_weight, dw_bias, pw_weight, doffsets, dims, heads, per_tap=False,
                         stream=None):
    """Gradients of sum(offsets * doffsets) for offsets = offset_head(...): (dx [N][C] in x's
    dtype, d dw_weight, d dw_bias, d pw_weight, d pw_bias, all fp32 but dx)."""
    torch = _torch()
    code = _dtype_code(x)
    C, kt, kh, kw = _conv_shapes(x, dw_weight, dims)
    taps = kt * kh * kw if per_tap else 1
    width = heads * taps * 3
    N = x.shape[0]
    if dw_bias is not None:
        _need(dw_bias, "dw_bias", (C,), torch.float32)
    _need(pw_weight, "pw_weight", (C, width), torch.float32)
    _need(doffsets, "doffsets", (heads, N, taps, 3) if per_tap else (heads, N, 3), torch.float32)
    _on_device(x, dw_weight, dw_bias, pw_weight, doffsets)
    dx = torch.empty_like(x)
    grads = (torch.empty_like(dw_weight), torch.empty(C, dtype=torch.float32, device=x.device),
             torch.empty_like(pw_weight), torch.empty(width, dtype=torch.float32, device=x.device))
    ws = torch.empty(dsa3d_offset_head_backward_workspace_bytes(*dims, C), dtype=torch.uint8,
                     device=x.device)
    _check(dsa3d_offset_head_backward(x.data_ptr(), dw_weight.data_ptr(),
                                      dw_bias.data_ptr() if dw_bias is not None else None,
                                      pw_weight.data_ptr(), doffsets.data_ptr(), dx.data_ptr(),
                                      *(t.data_ptr() for t in grads), ws.data_ptr(), ws.numel(), *dims,
                                      C, heads, taps, kt, kh, kw, code, _stream_handle(stream)),
           "dsa3d_offset_head_backward")
    return (dx, *grads)


# --- the transformer block around the operator -----------------------------------------------------
_NO_CONTEXT = contextlib.nullcontext()


def _on_stream(ref, stream, inputs):
    """Context of a call's allocations and launches: ref's device, and the given stream where there is
    one (the outputs and workspaces then belong to that stream).  Inputs that another stream owns are
    recorded on it, so that freeing them right after the call is safe."""
    torch = _torch()
    if stream is None:
        return _NO_CONTEXT if torch.cuda.current_device() == ref.device.index else torch.cuda.device(ref.device)
    if stream.device != ref.device:
        raise ValueError("stream and tensors must be on one device")
    with torch.cuda.device(ref.device):
        if stream != torch.cuda.current_stream():
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)
    return torch.cuda.stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _current_stream_handle(ref):
    """Handle of the current stream of ref's device (which _on_stream has made the current one), without
    building a Stream object: small calls are bound by the host."""
    return _torch()._C._cuda_getCurrentRawStream(ref.device.index)


def _rows2d(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows][C], got {tuple(t.shape)}")
    _need(t, name, t.shape, t.dtype)
    return t.shape


def layer_norm(x, weight=None, bias=None, eps=1e-5, add=None, out=None, want_stats=True, stream=None):
    """Layer norm of x [rows][C] over the channels, or of h = x + add [rows][C] (a residual sum, kept in
    x's dtype); weight and bias [C] fp32 or None.  Returns (y, h, stats): h is x itself without add,
    stats [2][rows] fp32 (means, reciprocal standard deviations; None unless want_stats) is what
    layer_norm_backward takes."""
    torch = _torch()
    code = _dtype_code(x)
    rows, C = _rows2d(x, "x")
    if add is not None:
        _need(add, "add", x.shape, x.dtype)
    if weight is not None:
        _need(weight, "weight", (C,), torch.float32)
    if bias is not None:
        _need(bias, "bias", (C,), torch.float32)
    if out is not None:
        _need(out, "out", x.shape, x.dtype)
    _on_device(x, add, weight, bias, out)
    with _on_stream(x, stream, (x, add, weight, bias, out)):
        y = torch.empty_like(x) if out is None else out
        h = None if add is None else torch.empty_like(x)
        stats = x.new_empty((2, rows), dtype=torch.float32) if want_stats else None
        _check(dsa3d_layer_norm(x.data_ptr(), _ptr(add), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(h),
                                _ptr(stats), rows, C, eps, code, _current_stream_handle(x)), "dsa3d_layer_norm")
    return y, (x if h is None else h), stats


def layer_norm_backward(h, weight, stats, dy, add=None, stream=None):
    """Gradients of sum(layer_norm(h, weight, bias)[0] * dy): (dx [rows][C], dweight, dbias [C] fp32).
    h and stats as the forward returned them; add [rows][C] is added to dx (the residual branch's
    gradient).  Without a weight the two weight gradients are None."""
    torch = _torch()
    code = _dtype_code(h)
    rows, C = _rows2d(h, "h")
    _need(dy, "dy", h.shape, h.dtype)
    _need(stats, "stats", (2, rows), torch.float32)
    if add is not None:
        _need(add, "add", h.shape, h.dtype)
    if weight is not None:
        _need(weight, "weight", (C,), torch.float32)
    _on_device(h, weight, stats, dy, add)
    with _on_stream(h, stream, (h, weight, stats, dy, add)):
        dx = torch.empty_like(h)
        dw = db = ws = None
        ws_bytes = 0
        if weight is not None:
            dw, db = torch.empty_like(weight), torch.empty_like(weight)
            ws_bytes = dsa3d_layer_norm_backward_workspace_bytes(rows, C, code)
            ws = weight.new_empty(ws_bytes // 4)
        _check(dsa3d_layer_norm_backward(h.data_ptr(), _ptr(weight), stats.data_ptr(), dy.data_ptr(), _ptr(add),
                                         dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws), ws_bytes, rows, C, code,
                                         _current_stream_handle(h)), "dsa3d_layer_norm_backward")
    return dx, dw, db


def _token_stride(t, name, shape, dtype):
    """t must be [rows][heads][dh] with contiguous heads; returns its token stride in elements."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    rows, heads, dh = shape
    s0, s1, s2 = t.stride()
    if (dh > 1 and s2 != 1) or (heads > 1 and s1 != dh):
        raise ValueError(f"{name} must have contiguous [heads][dh] rows")
    if rows > 1 and s0 < heads * dh:
        raise ValueError(f"{name}'s tokens overlap")
    return s0 if rows > 1 else heads * dh


def _rotary(call, what, q, k, dims, axes, first, start, step, base, interleaved, out, stream):
    torch = _torch()
    code = _dtype_code(q)
    if q.dim() != 3:
        raise ValueError(f"q must be [rows][heads][dh], got {tuple(q.shape)}")
    if len(axes) != 3 or len(dims) != 3 or len(start) != 3 or len(step) != 3:
        raise ValueError("dims, axes, start and step have three entries: frames, rows, columns")
    rows, heads, dh = q.shape
    ldq = _token_stride(q, "q", q.shape, q.dtype)
    ldk = ldq if k is None else _token_stride(k, "k", q.shape, q.dtype)
    qo, ko = (None, None) if out is None else out
    if out is not None:
        if (k is None) != (ko is None) or qo is None:
            raise ValueError("out must hold one tensor for each of q and k")
        ldqo = _token_stride(qo, "out[0]", q.shape, q.dtype)
        ldko = ldqo if ko is None else _token_stride(ko, "out[1]", q.shape, q.dtype)
    else:
        ldqo = ldko = heads * dh
    _on_device(q, k, qo, ko)
    with _on_stream(q, stream, (q, k, qo, ko)):
        if out is None:
            qo = q.new_empty(q.shape)
            ko = None if k is None else k.new_empty(q.shape)
        _check(call(q.data_ptr(), _ptr(k), qo.data_ptr(), _ptr(ko), ldq, ldk, ldqo, ldko, first, rows, *dims,
                    heads, dh, axes, start, step, base, 1 if interleaved else 0, code, _current_stream_handle(q)),
               what)
    return qo, ko


def rotary3d(q, k, dims, axes, first=0, start=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0), base=10000.0,
             interleaved=True, out=None, stream=None):
    """Rotary positions for q and k [rows][heads][dh] (k may be None), the tokens first .. first + rows - 1
    of the grid dims = (F, Hp, Wp).  axes: head dims of the frame, row and column axis (even); pairs are
    (2i, 2i+1), or (i, i + sum(axes)/2) with interleaved=False.  Positions are start + step * index.
    Tokens may be strided (views of a packed projection); out = (q_out, k_out) may be q and k themselves.
    Returns (q_out, k_out)."""
    return _rotary(dsa3d_rotary3d, "dsa3d_rotary3d", q, k, dims, axes, first, start, step, base, interleaved,
                   out, stream)


def rotary3d_backward(dq, dk, dims, axes, first=0, start=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0), base=10000.0,
                      interleaved=True, out=None, stream=None):
    """Gradients of rotary3d's q and k from those of its outputs (the inverse rotation); the other
    arguments are rotary3d's.  Returns (gradient of q, gradient of k)."""
    return _rotary(dsa3d_rotary3d_backward, "dsa3d_rotary3d_backward", dq, dk, dims, axes, first, start, step,
                   base, interleaved, out, stream)


def _ffn_shapes(x, gate_weight, up_weight, down_weight, activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    rows, C = _rows2d(x, "x")
    if gate_weight.dim() != 2 or gate_weight.shape[0] != C:
        raise ValueError(f"gate_weight must be [C={C}][hidden], got {tuple(gate_weight.shape)}")
    hidden = gate_weight.shape[1]
    _need(gate_weight, "gate_weight", (C, hidden), x.dtype)
    _need(up_weight, "up_weight", (C, hidden), x.dtype)
    _need(down_weight, "down_weight", (hidden, C), x.dtype)
    return rows, C, hidden


def _ffn_workspace(workspace, need, device):
    if isinstance(workspace, str):
        return _torch().empty(need, dtype=_torch().uint8, device=device)
    return workspace


def gated_ffn(x, gate_weight, up_weight, down_weight, activation="silu", add=None, out=None, workspace="auto",
              stream=None):
    """Gated feed-forward block y = (act(x Wg) * (x Wu)) Wd (+ add) for x [rows][C], gate_weight and
    up_weight [C][hidden], down_weight [hidden][C], all of x's dtype; activation "silu" or "gelu" (erf).
    add [rows][C] is the residual branch; out may be add itself.  workspace: "auto" allocates what
    dsa3d_gated_ffn_workspace_bytes asks for; a smaller uint8 tensor makes the call go through the
    tokens in more chunks.  Returns y."""
    torch = _torch()
    code = _dtype_code(x)
    rows, C, hidden = _ffn_shapes(x, gate_weight, up_weight, down_weight, activation)
    if add is not None:
        _need(add, "add", x.shape, x.dtype)
    if out is not None:
        _need(out, "out", x.shape, x.dtype)
    given = None if isinstance(workspace, str) else _workspace(workspace)
    _on_device(x, gate_weight, up_weight, down_weight, add, out, given)
    with _on_stream(x, stream, (x, gate_weight, up_weight, down_weight, add, out, given)):
        y = torch.empty_like(x) if out is None else out
        ws = _ffn_workspace(workspace, dsa3d_gated_ffn_workspace_bytes(rows, C, hidden, code), x.device)
        _check(dsa3d_gated_ffn(x.data_ptr(), gate_weight.data_ptr(), up_weight.data_ptr(), down_weight.data_ptr(),
                               _ptr(add), y.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(), rows, C, hidden,
                               _ACTIVATIONS[activation], code, _current_stream_handle(x)), "dsa3d_gated_ffn")
    return y


def gated_ffn_backward(x, gate_weight, up_weight, down_weight, dy, activation="silu", workspace="auto",
                       stream=None):
    """Gradients of sum(gated_ffn(x, ...) * dy): (dx, dgate_weight, dup_weight, ddown_weight), all of x's
    dtype, from x and dy alone (x Wg and x Wu are formed again)."""
    torch = _torch()
    code = _dtype_code(x)
    rows, C, hidden = _ffn_shapes(x, gate_weight, up_weight, down_weight, activation)
    _need(dy, "dy", x.shape, x.dtype)
    given = None if isinstance(workspace, str) else _workspace(workspace)
    _on_device(x, gate_weight, up_weight, down_weight, dy, given)
    with _on_stream(x, stream, (x, gate_weight, up_weight, down_weight, dy, given)):
        grads = (torch.empty_like(x), torch.empty_like(gate_weight), torch.empty_like(up_weight),
                 torch.empty_like(down_weight))
        ws = _ffn_workspace(workspace, dsa3d_gated_ffn_backward_workspace_bytes(rows, C, hidden, code), x.device)
        _check(dsa3d_gated_ffn_backward(x.data_ptr(), gate_weight.data_ptr(), up_weight.data_ptr(),
                                        down_weight.data_ptr(), dy.data_ptr(), *(t.data_ptr() for t in grads),
                                        _ptr(ws), 0 if ws is None else ws.numel(), rows, C, hidden,
                                        _ACTIVATIONS[activation], code, _current_stream_handle(x)),
               "dsa3d_gated_ffn_backward")
    return grads
