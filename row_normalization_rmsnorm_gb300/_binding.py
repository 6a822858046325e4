"""ctypes binding of libgb300norm.so (the C ABI in include/gb300norm.h).

Argument marshalling only: every function below takes torch tensors on one
CUDA device, passes their data pointers, row strides, shapes and dtype codes
to the C entry point of the same name (with that device current) and raises
NormError on a non-zero status.  Nothing is computed here and there is no
CPU path: a CPU tensor, or a missing library, is an error.

The C ABI sees only pointers, so the extent of every buffer is checked here
before the call: each 2-D tensor must be (M, N) in the activation dtype with
contiguous rows, w / b / dW / dB must hold N elements, rstd / mean at least
M FP32 values, a checkpoint must be (M, norm_ckpt_row_bytes(N)) uint8, and
every tensor must sit on x's device.  Shape and dtype errors raise ValueError
(before any device check), a CPU tensor TypeError.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgb300norm.so")

NORM_F32, NORM_F16, NORM_BF16 = 0, 1, 2
DTYPE_CODE = {torch.float32: NORM_F32, torch.float16: NORM_F16, torch.bfloat16: NORM_BF16}
CODE_DTYPE = {v: k for k, v in DTYPE_CODE.items()}

# status codes (include/gb300norm.h)
NORM_OK = 0
NORM_ERR_NULL = 1
NORM_ERR_SHAPE = 2
NORM_ERR_STRIDE = 3
NORM_ERR_DTYPE = 4
NORM_ERR_WORKSPACE = 5
NORM_ERR_ALIGN = 6
NORM_ERR_VALUE = 7
NORM_ERR_ALIAS = 8
NORM_ERR_CUDA = 9
NORM_ERR_ARG = 10
NORM_ERR_TOO_LARGE = 11

# saved rows of a backward: in full, or 8-bit checkpoints
NORM_SAVED_FULL, NORM_SAVED_E4M3, NORM_SAVED_INT8 = 0, 1, 2

# Every entry point the header declares, with its ctypes signature.
_P, _I64, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "norm_status_str": ([_I], ctypes.c_char_p),
    "norm_version": ([], _I),
    "norm_bwd_workspace_bytes": ([_I64, _I64, _I, _I, ctypes.POINTER(_SZ)], _I),
    "norm_rms_fwd": ([_P, _I64, _P, _P, _I64, _P, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_rms_bwd": ([_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I, _P, _SZ, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_ln_fwd": ([_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_ln_bwd": ([_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _I, _P, _SZ, _I64, _I64, _F, _F, _I, _I,
                     _P], _I),
    "norm_fused_add_rms_fwd": ([_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _I64, _F, _F, _I, _I, _P],
                               _I),
    "norm_fused_add_rms_bwd": ([_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I, _P, _SZ, _I64, _I64, _F,
                                _F, _I, _I, _P], _I),
    "norm_device_status": ([_I, ctypes.POINTER(_I)], _I),
    "norm_debug_set_path": ([_I], _I),
    "norm_debug_tune": ([_I, _I], _I),
    "norm_last_cuda_error": ([], _I),
    "norm_noalloc_scratch_bytes": ([], _SZ),
    "norm_rms_bwd_noalloc": ([_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_cuda_error_string": ([_I], ctypes.c_char_p),
    "norm_sum_ranks": ([_P, _I64, _I64, _P, _I, _P], _I),
    "norm_debug_launches": ([_I], _I64),
    "norm_ckpt_row_bytes": ([_I64, ctypes.POINTER(_SZ)], _I),
    "norm_ckpt_encode": ([_P, _I64, _P, _I64, _I, _I64, _I64, _I, _P], _I),
    "norm_ckpt_decode": ([_P, _I64, _I, _P, _I64, _I64, _I64, _I, _P], _I),
    "norm_rms_fwd_ckpt": ([_P, _I64, _P, _P, _I64, _P, _P, _I64, _I, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_rms_bwd_ckpt": ([_P, _I64, _P, _I64, _I, _P, _P, _P, _I64, _P, _I, _P, _SZ, _I64, _I64, _F, _I, _I, _P],
                          _I),
    "norm_ln_fwd_ckpt": ([_P, _I64, _P, _P, _P, _I64, _P, _P, _P, _I64, _I, _I64, _I64, _F, _F, _I, _I, _P], _I),
    "norm_ln_bwd_ckpt": ([_P, _I64, _P, _I64, _I, _P, _P, _P, _I64, _P, _P, _I, _P, _SZ, _I64, _I64, _F, _I, _I,
                          _P], _I),
    "norm_fused_add_rms_fwd_ckpt": ([_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _P, _I64, _I, _I64, _I64, _F,
                                     _F, _I, _I, _P], _I),
    "norm_fused_add_rms_bwd_ckpt": ([_P, _I64, _P, _I64, _P, _I64, _I, _P, _P, _P, _I64, _P, _I, _P, _SZ, _I64, _I64,
                                     _F, _I, _I, _P], _I),
    "norm_block_bwd_workspace_bytes": ([_I64, _I64, _I64, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "norm_block_rms_fwd": ([_P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64,
                            _I, _I64, _I64, _F, _F, _F, _F, _I, _I, _I, _P], _I),
    "norm_block_rms_bwd": ([_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64,
                            _P, _I64, _P, _I64, _P, _P, _I, _P, _SZ, _I64, _I64, _F, _F, _F, _I, _I, _I, _P], _I),
}


class NormError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn}: status {status} ({status_str(status)})"
        if status == NORM_ERR_CUDA:
            code = lib.norm_last_cuda_error()
            msg += f"; CUDA error {code}: {lib.norm_cuda_error_string(code).decode()}"
        super().__init__(msg)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(nvcc, sm_103a). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in SIGNATURES.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


lib = _load()


def status_str(status: int) -> str:
    return lib.norm_status_str(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != NORM_OK:
        raise NormError(fn, rc)


# The current stream's raw handle without building a torch.cuda.Stream object
# on every call (that alone cost more than the rest of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, like=None):
    """Raw cudaStream_t (an int) for the C ABI: `stream`, else the current
    stream of `like`'s device (else of the current device)."""
    if stream is None:
        if _raw_stream is not None:
            dev = like.get_device() if like is not None else torch.cuda.current_device()
            return _raw_stream(dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _mat(t, name, M, N, dtype, required=True):
    """Check a 2-D row tensor: shape (M, N), the activation dtype, rows
    contiguous.  Runs before any device check, so a shape error is reported
    as such whatever the tensor's device."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    _tensor(t, name)
    if t.dim() != 2 or tuple(t.shape) != (M, N):
        raise ValueError(f"{name} must have shape ({M}, {N}), got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if M > 0 and N > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")


def _vec(t, name, n, dtypes, at_least=False, required=True):
    """Check a 1-D contiguous vector of n elements (at least n when
    `at_least`) whose dtype is one of `dtypes`."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    _tensor(t, name)
    if t.dim() != 1:
        raise ValueError(f"{name} must be 1-D, got shape {tuple(t.shape)}")
    if (t.numel() < n) if at_least else (t.numel() != n):
        raise ValueError(f"{name} must have {'at least ' if at_least else ''}{n} elements, got {t.numel()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.numel() > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _act_dtype(x, name="x"):
    _tensor(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D [M, N], got shape {tuple(x.shape)}")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"{name} dtype {x.dtype} is not supported")
    return x.dtype


def _weight(w, N):
    _tensor(w, "w")
    _vec(w, "w", N, tuple(DTYPE_CODE))
    return w.dtype


def _grad_dtype(w_dtype, *grads):
    """dtype code of the dW / dB outputs: FP32 or the weight's dtype, the
    same for every gradient given."""
    given = [(n, t) for n, t in grads if t is not None]
    if not given:
        return NORM_F32
    dt = given[0][1].dtype
    if dt not in (torch.float32, w_dtype):
        raise ValueError(f"{given[0][0]} must be float32 or the weight dtype {w_dtype}, got {dt}")
    for n, t in given[1:]:
        if t.dtype != dt:
            raise ValueError(f"{n} must have the same dtype as {given[0][0]} ({dt}), got {t.dtype}")
    return DTYPE_CODE[dt]


def _device(x, *others):
    """Index of the CUDA device every tensor lives on (x's), or an error."""
    if not x.is_cuda:
        raise TypeError("x must be a CUDA tensor (this library has no CPU path)")
    dev = x.get_device()
    for name, t in others:
        if t is None:
            continue
        _tensor(t, name)
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor (this library has no CPU path)")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, x on cuda:{dev}")
    return dev


def _on(dev, fn):
    """Run fn with `dev` as the current device: the C ABI takes its device
    (launch shapes, status word) from the current device."""
    if dev == torch.cuda.current_device():
        return fn()
    with torch.cuda.device(dev):
        return fn()


def _rs(t):
    return t.stride(0) if (t is not None and t.dim() == 2) else 0


def _ptr(t):
    return None if t is None else (t.data_ptr() or None)


def _ws(workspace):
    if workspace is None:
        return None, 0
    _tensor(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def norm_bwd_workspace_bytes(M: int, N: int, has_dw: bool, has_db: bool = False) -> int:
    out = ctypes.c_size_t(0)
    _check("norm_bwd_workspace_bytes", lib.norm_bwd_workspace_bytes(M, N, int(has_dw), int(has_db),
                                                                    ctypes.byref(out)))
    return out.value


def norm_device_status(reset: bool = False) -> int:
    v = ctypes.c_int(0)
    _check("norm_device_status", lib.norm_device_status(int(reset), ctypes.byref(v)))
    return v.value


def norm_debug_set_path(mode: int):
    _check("norm_debug_set_path", lib.norm_debug_set_path(int(mode)))


def norm_debug_tune(key: int, value: int):
    _check("norm_debug_tune", lib.norm_debug_tune(int(key), int(value)))


def norm_debug_launches(reset: bool = False) -> int:
    """Kernels this library has launched since load or the last reset."""
    return int(lib.norm_debug_launches(int(reset)))


_F32 = (torch.float32,)


def norm_sum_ranks(parts, out, stream=None):
    """out = the rows of parts (FP32, [world, N], one per rank) added in rank
    order in FP32 and converted once to out's dtype (FP32, FP16 or BF16, N
    elements)."""
    _tensor(parts, "parts")
    if parts.dim() != 2 or parts.shape[0] < 1 or parts.shape[1] < 1:
        raise ValueError(f"parts must be 2-D [world, N] with world, N >= 1, got shape {tuple(parts.shape)}")
    if parts.dtype != torch.float32:
        raise ValueError(f"parts must be float32, got {parts.dtype}")
    if not parts.is_contiguous():
        raise ValueError("parts must be contiguous")
    world, N = parts.shape
    _vec(out, "out", N, tuple(DTYPE_CODE))
    dev = _device(parts, ("out", out))
    _on(dev, lambda: _check("norm_sum_ranks", lib.norm_sum_ranks(
        _ptr(parts), world, N, _ptr(out), DTYPE_CODE[out.dtype], _stream(stream, parts))))


def norm_rms_fwd(x, w, y, rstd=None, offset=0.0, eps=1e-6, stream=None):
    """y = RMSNorm(x) with scale (w + offset); rstd (FP32, [M]) optional."""
    dt = _act_dtype(x)
    M, N = x.shape
    wdt = _weight(w, N)
    _mat(y, "y", M, N, dt)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    dev = _device(x, ("w", w), ("y", y), ("rstd", rstd))
    _on(dev, lambda: _check("norm_rms_fwd", lib.norm_rms_fwd(
        _ptr(x), _rs(x), _ptr(w), _ptr(y), _rs(y), _ptr(rstd), M, N, float(offset), float(eps),
        DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def _rms_bwd_checks(dy, x, w, rstd, dx, dw):
    dt = _act_dtype(x)
    M, N = x.shape
    wdt = _weight(w, N)
    _mat(dy, "dy", M, N, dt)
    _mat(dx, "dx", M, N, dt)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    _vec(dw, "dw", N, (torch.float32, wdt), required=False)
    dwt = _grad_dtype(wdt, ("dw", dw))
    dev = _device(x, ("dy", dy), ("w", w), ("rstd", rstd), ("dx", dx), ("dw", dw))
    return dt, wdt, dwt, dev


def norm_rms_bwd(dy, x, w, rstd, dx, dw=None, workspace=None, offset=0.0, eps=1e-6, stream=None):
    """dx (and dw unless None = frozen) of RMSNorm; rstd None = recompute."""
    dt, wdt, dwt, dev = _rms_bwd_checks(dy, x, w, rstd, dx, dw)
    M, N = x.shape
    _device(x, ("workspace", workspace))
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_rms_bwd", lib.norm_rms_bwd(
        _ptr(dy), _rs(dy), _ptr(x), _rs(x), _ptr(w), _ptr(rstd), _ptr(dx), _rs(dx), _ptr(dw), dwt, wsp, wsb,
        M, N, float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_rms_bwd_noalloc(dy, x, w, rstd, dx, dw=None, offset=0.0, eps=1e-6, stream=None):
    """norm_rms_bwd without a workspace: the dW partial sums use the
    library's fixed scratch (for callers that cannot allocate)."""
    dt, wdt, dwt, dev = _rms_bwd_checks(dy, x, w, rstd, dx, dw)
    M, N = x.shape
    _on(dev, lambda: _check("norm_rms_bwd_noalloc", lib.norm_rms_bwd_noalloc(
        _ptr(dy), _rs(dy), _ptr(x), _rs(x), _ptr(w), _ptr(rstd), _ptr(dx), _rs(dx), _ptr(dw), dwt, M, N,
        float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_ln_fwd(x, w, b, y, mean=None, rstd=None, offset=0.0, eps=1e-6, stream=None):
    """y = LayerNorm(x) with scale (w + offset) and bias b (None = no bias)."""
    dt = _act_dtype(x)
    M, N = x.shape
    wdt = _weight(w, N)
    _vec(b, "b", N, (wdt,), required=False)
    _mat(y, "y", M, N, dt)
    _vec(mean, "mean", M, _F32, at_least=True, required=False)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    dev = _device(x, ("w", w), ("b", b), ("y", y), ("mean", mean), ("rstd", rstd))
    _on(dev, lambda: _check("norm_ln_fwd", lib.norm_ln_fwd(
        _ptr(x), _rs(x), _ptr(w), _ptr(b), _ptr(y), _rs(y), _ptr(mean), _ptr(rstd), M, N, float(offset),
        float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_ln_bwd(dy, x, w, mean, rstd, dx, dw=None, db=None, workspace=None, offset=0.0, eps=1e-6,
                stream=None):
    """dx, and dw / db unless None (frozen), of LayerNorm."""
    dt = _act_dtype(x)
    M, N = x.shape
    wdt = _weight(w, N)
    _mat(dy, "dy", M, N, dt)
    _mat(dx, "dx", M, N, dt)
    _vec(mean, "mean", M, _F32, at_least=True, required=False)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    _vec(dw, "dw", N, (torch.float32, wdt), required=False)
    _vec(db, "db", N, (torch.float32, wdt), required=False)
    dwt = _grad_dtype(wdt, ("dw", dw), ("db", db))
    dev = _device(x, ("dy", dy), ("w", w), ("mean", mean), ("rstd", rstd), ("dx", dx), ("dw", dw), ("db", db),
                  ("workspace", workspace))
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_ln_bwd", lib.norm_ln_bwd(
        _ptr(dy), _rs(dy), _ptr(x), _rs(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx), _rs(dx), _ptr(dw),
        _ptr(db), dwt, wsp, wsb, M, N, float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt],
        _stream(stream, x))))


def norm_fused_add_rms_fwd(x, residual, w, y, h_out, rstd=None, offset=0.0, eps=1e-6, stream=None):
    """h_out = x + residual (rounded), y = RMSNorm(h) with scale (w + offset)."""
    dt = _act_dtype(x)
    M, N = x.shape
    wdt = _weight(w, N)
    _mat(residual, "residual", M, N, dt)
    _mat(y, "y", M, N, dt)
    _mat(h_out, "h_out", M, N, dt)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    dev = _device(x, ("residual", residual), ("w", w), ("y", y), ("h_out", h_out), ("rstd", rstd))
    _on(dev, lambda: _check("norm_fused_add_rms_fwd", lib.norm_fused_add_rms_fwd(
        _ptr(x), _rs(x), _ptr(residual), _rs(residual), _ptr(w), _ptr(y), _rs(y), _ptr(h_out), _rs(h_out),
        _ptr(rstd), M, N, float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_fused_add_rms_bwd(dy, dh_out, h, w, rstd, dx, dw=None, workspace=None, offset=0.0, eps=1e-6,
                           stream=None):
    """dx (= d residual) and dw unless None, of FusedAddRMSNorm at saved h."""
    dt = _act_dtype(h, "h")
    M, N = h.shape
    wdt = _weight(w, N)
    _mat(dy, "dy", M, N, dt)
    _mat(dh_out, "dh_out", M, N, dt, required=False)
    _mat(dx, "dx", M, N, dt)
    _vec(rstd, "rstd", M, _F32, at_least=True, required=False)
    _vec(dw, "dw", N, (torch.float32, wdt), required=False)
    dwt = _grad_dtype(wdt, ("dw", dw))
    dev = _device(h, ("dy", dy), ("dh_out", dh_out), ("w", w), ("rstd", rstd), ("dx", dx), ("dw", dw),
                  ("workspace", workspace))
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_fused_add_rms_bwd", lib.norm_fused_add_rms_bwd(
        _ptr(dy), _rs(dy), _ptr(dh_out), _rs(dh_out), _ptr(h), _rs(h), _ptr(w), _ptr(rstd), _ptr(dx), _rs(dx),
        _ptr(dw), dwt, wsp, wsb, M, N, float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt],
        _stream(stream, h))))


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints
# ---------------------------------------------------------------------------
def norm_ckpt_row_bytes(N: int) -> int:
    """Bytes of the checkpoint of one row of N values."""
    out = ctypes.c_size_t(0)
    _check("norm_ckpt_row_bytes", lib.norm_ckpt_row_bytes(N, ctypes.byref(out)))
    return out.value


# Quick acceptance of a call's tensors, for the calls below: a small call costs
# more here than on the GPU, and the usual one has every tensor on one CUDA
# device, of the right shape and dtype, rows contiguous.  Anything else (None
# back) goes through the checks that say what is wrong, or accept what is unusual
# (no rows, one column, longer statistics).
def _quick_rows(dev, shape, dtype, *tensors):
    """Row strides of 2-D tensors (0 for None), or None."""
    out = []
    for t in tensors:
        if t is None:
            out.append(0)
            continue
        if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
            return None
        s = t.stride()
        if s[1] != 1 or s[0] < shape[1]:
            return None
        out.append(s[0])
    return out


def _quick_vecs(dev, n, dtype, *tensors):
    """Whether 1-D tensors (or None) hold n elements of dtype each."""
    for t in tensors:
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev
                              or t.shape != (n,) or t.stride() != (1,)):
            return False
    return True


def _on_dev(t, dev):
    """Whether t is None or a tensor on that device."""
    return t is None or (isinstance(t, torch.Tensor) and t.get_device() == dev)


def _quick(x):
    """(device, M, N) of a 2-D CUDA tensor with rows, or None."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2 or x.dtype not in DTYPE_CODE:
        return None
    M, N = x.shape
    return (x.get_device(), M, N) if M > 0 and N > 1 else None   # (with no rows or one column, strides mean little)


def _quick_gate(dev, gate, rows_per_gate, M, N, dtype, w_dtype):
    """_gate for a usual gate, or None."""
    if gate is None:
        return 0, 0, 0, DTYPE_CODE[dtype]
    if not isinstance(gate, torch.Tensor) or gate.get_device() != dev:
        return None
    return _gate(gate, rows_per_gate, M, N, dtype, w_dtype)


def _ckpt_bytes(N):
    return (N + 15) // 16 * 16 + ((N + 31) // 32 + 15) // 16 * 16


def _ckpt(t, name, M, N, required=True):
    """Check a checkpoint buffer: (M, norm_ckpt_row_bytes(N)) bytes with
    contiguous rows."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    _mat(t, name, M, _ckpt_bytes(N), torch.uint8)


def _quick_norm(x, w, rows, stats, ckpt, workspace, cols=()):
    """(device, M, N, dtype, weight dtype, row strides of `rows`, ckpt's stride)
    of a usual call of a checkpointed norm, or None.  cols: per-column vectors
    (or None) of w's dtype or FP32."""
    q = _quick(x)
    if q is None or not isinstance(w, torch.Tensor) or ckpt is None or stats[-1] is None:
        return None
    dev, M, N = q
    dt, wdt = x.dtype, w.dtype
    st = _quick_rows(dev, x.shape, dt, *rows)
    if (st is None or wdt not in DTYPE_CODE or not _quick_vecs(dev, N, wdt, w)
            or not _quick_vecs(dev, M, torch.float32, *stats)):
        return None
    for t in cols:
        if t is not None and (not isinstance(t, torch.Tensor) or not _quick_vecs(dev, N, t.dtype, t)
                              or (t.dtype is not wdt and t.dtype is not torch.float32)):
            return None
    if any(t is None for t in rows[:1] + rows[-1:]) or not _on_dev(workspace, dev):
        return None
    sq = _quick_rows(dev, (M, _ckpt_bytes(N)), torch.uint8, ckpt)
    return None if sq is None else (dev, M, N, dt, wdt, st, sq[0])


def norm_ckpt_encode(x, ckpt, format, stream=None):
    """ckpt (uint8, [M, norm_ckpt_row_bytes(N)]) = the rows of x as 8-bit codes
    of `format` with one power-of-two scale per 32 columns."""
    dt = _act_dtype(x)
    M, N = x.shape
    _ckpt(ckpt, "ckpt", M, N)
    dev = _device(x, ("ckpt", ckpt))
    _on(dev, lambda: _check("norm_ckpt_encode", lib.norm_ckpt_encode(
        _ptr(x), _rs(x), _ptr(ckpt), _rs(ckpt), int(format), M, N, DTYPE_CODE[dt], _stream(stream, x))))


def norm_ckpt_decode(ckpt, format, x, stream=None):
    """x = the values the checkpoint's codes stand for, rounded to x's dtype."""
    dt = _act_dtype(x)
    M, N = x.shape
    _ckpt(ckpt, "ckpt", M, N)
    dev = _device(x, ("ckpt", ckpt))
    _on(dev, lambda: _check("norm_ckpt_decode", lib.norm_ckpt_decode(
        _ptr(ckpt), _rs(ckpt), int(format), _ptr(x), _rs(x), M, N, DTYPE_CODE[dt], _stream(stream, x))))


def norm_rms_fwd_ckpt(x, w, y, rstd, ckpt, format, offset=0.0, eps=1e-6, stream=None):
    """norm_rms_fwd that also keeps x as an 8-bit checkpoint."""
    q = _quick_norm(x, w, (x, y), (rstd,), ckpt, None)
    if q is None:
        dt = _act_dtype(x)
        M, N = x.shape
        wdt = _weight(w, N)
        _mat(y, "y", M, N, dt)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _ckpt(ckpt, "ckpt", M, N)
        dev = _device(x, ("w", w), ("y", y), ("rstd", rstd), ("ckpt", ckpt))
        q = dev, M, N, dt, wdt, (_rs(x), _rs(y)), _rs(ckpt)
    dev, M, N, dt, wdt, (sx, sy), sq = q
    _on(dev, lambda: _check("norm_rms_fwd_ckpt", lib.norm_rms_fwd_ckpt(
        _ptr(x), sx, _ptr(w), _ptr(y), sy, _ptr(rstd), _ptr(ckpt), sq, int(format), M, N, float(offset),
        float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_rms_bwd_ckpt(dy, ckpt, format, w, rstd, dx, dw=None, workspace=None, offset=0.0, stream=None):
    """dx (and dw unless None = frozen) of RMSNorm at the checkpointed rows."""
    q = _quick_norm(dy, w, (dy, dx), (rstd,), ckpt, workspace, (dw,))
    if q is None:
        dt = _act_dtype(dy, "dy")
        M, N = dy.shape
        wdt = _weight(w, N)
        _ckpt(ckpt, "ckpt", M, N)
        _mat(dx, "dx", M, N, dt)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _vec(dw, "dw", N, (torch.float32, wdt), required=False)
        _grad_dtype(wdt, ("dw", dw))
        dev = _device(dy, ("ckpt", ckpt), ("w", w), ("rstd", rstd), ("dx", dx), ("dw", dw), ("workspace", workspace))
        q = dev, M, N, dt, wdt, (_rs(dy), _rs(dx)), _rs(ckpt)
    dev, M, N, dt, wdt, (sdy, sdx), sq = q
    dwt = NORM_F32 if dw is None else DTYPE_CODE[dw.dtype]
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_rms_bwd_ckpt", lib.norm_rms_bwd_ckpt(
        _ptr(dy), sdy, _ptr(ckpt), sq, int(format), _ptr(w), _ptr(rstd), _ptr(dx), sdx, _ptr(dw), dwt,
        wsp, wsb, M, N, float(offset), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, dy))))


def norm_ln_fwd_ckpt(x, w, b, y, mean, rstd, ckpt, format, offset=0.0, eps=1e-6, stream=None):
    """norm_ln_fwd that also keeps x - mean as an 8-bit checkpoint (mean may be
    None)."""
    q = _quick_norm(x, w, (x, y), (mean, rstd), ckpt, None, (b,))
    if q is None or (b is not None and b.dtype is not w.dtype):
        dt = _act_dtype(x)
        M, N = x.shape
        wdt = _weight(w, N)
        _vec(b, "b", N, (wdt,), required=False)
        _mat(y, "y", M, N, dt)
        _vec(mean, "mean", M, _F32, at_least=True, required=False)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _ckpt(ckpt, "ckpt", M, N)
        dev = _device(x, ("w", w), ("b", b), ("y", y), ("mean", mean), ("rstd", rstd), ("ckpt", ckpt))
        q = dev, M, N, dt, wdt, (_rs(x), _rs(y)), _rs(ckpt)
    dev, M, N, dt, wdt, (sx, sy), sq = q
    _on(dev, lambda: _check("norm_ln_fwd_ckpt", lib.norm_ln_fwd_ckpt(
        _ptr(x), sx, _ptr(w), _ptr(b), _ptr(y), sy, _ptr(mean), _ptr(rstd), _ptr(ckpt), sq, int(format), M, N,
        float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_ln_bwd_ckpt(dy, ckpt, format, w, rstd, dx, dw=None, db=None, workspace=None, offset=0.0, stream=None):
    """dx, and dw / db unless None (frozen), of LayerNorm at the checkpointed
    x - mean."""
    q = _quick_norm(dy, w, (dy, dx), (rstd,), ckpt, workspace, (dw, db))
    if q is None or (dw is not None and db is not None and dw.dtype is not db.dtype):
        dt = _act_dtype(dy, "dy")
        M, N = dy.shape
        wdt = _weight(w, N)
        _ckpt(ckpt, "ckpt", M, N)
        _mat(dx, "dx", M, N, dt)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _vec(dw, "dw", N, (torch.float32, wdt), required=False)
        _vec(db, "db", N, (torch.float32, wdt), required=False)
        _grad_dtype(wdt, ("dw", dw), ("db", db))
        dev = _device(dy, ("ckpt", ckpt), ("w", w), ("rstd", rstd), ("dx", dx), ("dw", dw), ("db", db),
                      ("workspace", workspace))
        q = dev, M, N, dt, wdt, (_rs(dy), _rs(dx)), _rs(ckpt)
    dev, M, N, dt, wdt, (sdy, sdx), sq = q
    one = dw if dw is not None else db
    dwt = NORM_F32 if one is None else DTYPE_CODE[one.dtype]
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_ln_bwd_ckpt", lib.norm_ln_bwd_ckpt(
        _ptr(dy), sdy, _ptr(ckpt), sq, int(format), _ptr(w), _ptr(rstd), _ptr(dx), sdx, _ptr(dw), _ptr(db), dwt, wsp, wsb,
        M, N, float(offset), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, dy))))


def norm_fused_add_rms_fwd_ckpt(x, residual, w, y, h_out, rstd, ckpt, format, offset=0.0, eps=1e-6, stream=None):
    """norm_fused_add_rms_fwd that also keeps h as an 8-bit checkpoint."""
    q = _quick_norm(x, w, (x, residual, y, h_out), (rstd,), ckpt, None)
    if q is None or residual is None or y is None:
        dt = _act_dtype(x)
        M, N = x.shape
        wdt = _weight(w, N)
        _mat(residual, "residual", M, N, dt)
        _mat(y, "y", M, N, dt)
        _mat(h_out, "h_out", M, N, dt)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _ckpt(ckpt, "ckpt", M, N)
        dev = _device(x, ("residual", residual), ("w", w), ("y", y), ("h_out", h_out), ("rstd", rstd), ("ckpt", ckpt))
        q = dev, M, N, dt, wdt, (_rs(x), _rs(residual), _rs(y), _rs(h_out)), _rs(ckpt)
    dev, M, N, dt, wdt, (sx, sr, sy, sh), sq = q
    _on(dev, lambda: _check("norm_fused_add_rms_fwd_ckpt", lib.norm_fused_add_rms_fwd_ckpt(
        _ptr(x), sx, _ptr(residual), sr, _ptr(w), _ptr(y), sy, _ptr(h_out), sh, _ptr(rstd), _ptr(ckpt), sq, int(format), M,
        N, float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, x))))


def norm_fused_add_rms_bwd_ckpt(dy, dh_out, ckpt, format, w, rstd, dx, dw=None, workspace=None, offset=0.0,
                                stream=None):
    """dx (= d residual) and dw unless None, of FusedAddRMSNorm at the
    checkpointed h."""
    q = _quick_norm(dy, w, (dy, dh_out, dx), (rstd,), ckpt, workspace, (dw,))
    if q is None or dx is None:
        dt = _act_dtype(dy, "dy")
        M, N = dy.shape
        wdt = _weight(w, N)
        _mat(dh_out, "dh_out", M, N, dt, required=False)
        _ckpt(ckpt, "ckpt", M, N)
        _mat(dx, "dx", M, N, dt)
        _vec(rstd, "rstd", M, _F32, at_least=True)
        _vec(dw, "dw", N, (torch.float32, wdt), required=False)
        _grad_dtype(wdt, ("dw", dw))
        dev = _device(dy, ("dh_out", dh_out), ("ckpt", ckpt), ("w", w), ("rstd", rstd), ("dx", dx), ("dw", dw),
                      ("workspace", workspace))
        q = dev, M, N, dt, wdt, (_rs(dy), _rs(dh_out), _rs(dx)), _rs(ckpt)
    dev, M, N, dt, wdt, (sdy, sdh, sdx), sq = q
    dwt = NORM_F32 if dw is None else DTYPE_CODE[dw.dtype]
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_fused_add_rms_bwd_ckpt", lib.norm_fused_add_rms_bwd_ckpt(
        _ptr(dy), sdy, _ptr(dh_out), sdh, _ptr(ckpt), sq, int(format), _ptr(w), _ptr(rstd), _ptr(dx), sdx, _ptr(dw), dwt,
        wsp, wsb, M, N, float(offset), DTYPE_CODE[dt], DTYPE_CODE[wdt], _stream(stream, dy))))


# ---------------------------------------------------------------------------
# The block boundary: norm after a block, gate, scales, residual sum, norm
# before the next block
# ---------------------------------------------------------------------------
def norm_block_bwd_workspace_bytes(M: int, N: int, gate_rows: int, has_dw_post: bool, has_dw_pre: bool,
                                   has_dgate: bool) -> int:
    """Workspace bytes of norm_block_rms_bwd (gate_rows: rows of the gate, 0 =
    no gate)."""
    out = ctypes.c_size_t(0)
    _check("norm_block_bwd_workspace_bytes", lib.norm_block_bwd_workspace_bytes(
        M, N, gate_rows, int(has_dw_post), int(has_dw_pre), int(has_dgate), ctypes.byref(out)))
    return out.value


def _gate(gate, rows_per_gate, M, N, dtype, w_dtype, name="gate"):
    """(rows, row stride, rows per gate row, dtype code) of a gate: None, [N]
    (or [1, N]) for a scale per channel, or [rows, N] with rows_per_gate
    consecutive rows of x for each (None: M / rows)."""
    if gate is None:
        return 0, 0, 0, DTYPE_CODE[dtype]
    _tensor(gate, name)
    if gate.dim() not in (1, 2) or gate.shape[-1] != N:
        raise ValueError(f"{name} must be [N] or [rows, N] with N = {N}, got shape {tuple(gate.shape)}")
    rows = 1 if gate.dim() == 1 else gate.shape[0]
    if N > 1 and gate.stride(-1) != 1:
        raise ValueError(f"{name} rows must be contiguous (stride(-1) == 1)")
    if gate.dtype != dtype and not (rows == 1 and gate.dtype == w_dtype):
        raise ValueError(f"{name} must be {dtype}" + (f" or {w_dtype}" if rows == 1 else "") + f", got {gate.dtype}")
    if rows < 1:
        raise ValueError(f"{name} has no rows")
    if rows_per_gate is None or (rows == 1 and not rows_per_gate):
        if rows > 1 and M % rows:
            raise ValueError(f"{name} has {rows} rows, which do not divide {M}: pass rows_per_gate")
        rows_per_gate = max(1, M // rows)
    rows_per_gate = int(rows_per_gate)
    if rows_per_gate < 1 or (M > 0 and -(-M // rows_per_gate) != rows):
        raise ValueError(f"{name} has {rows} rows; {M} rows at {rows_per_gate} each take "
                         f"{-(-M // max(1, rows_per_gate))}")
    return rows, gate.stride(0) if gate.dim() == 2 else N, rows_per_gate, DTYPE_CODE[gate.dtype]


def _block_weights(w_post, w_pre, N):
    if w_post is None and w_pre is None:
        raise ValueError("one of w_post and w_pre is required")
    for t, name in ((w_post, "w_post"), (w_pre, "w_pre")):
        if t is not None:
            _tensor(t, name)
    wdt = _weight(w_post if w_post is not None else w_pre, N)
    if w_post is not None and w_pre is not None:
        _vec(w_pre, "w_pre", N, (wdt,))
    return wdt


def _quick_block(x, w_post, w_pre, rows, stats, ckpts, gate, rows_per_gate):
    """(device, M, N, dtype, weight dtype, row strides of `rows`, the ckpts' one
    stride, _gate's answer) of a usual call, or None."""
    q = _quick(x)
    w = w_post if w_post is not None else w_pre
    if q is None or not isinstance(w, torch.Tensor):
        return None
    dev, M, N = q
    dt, wdt = x.dtype, w.dtype
    st = _quick_rows(dev, x.shape, dt, *rows)
    if (st is None or wdt not in DTYPE_CODE or not _quick_vecs(dev, N, wdt, w_post, w_pre)
            or not _quick_vecs(dev, M, torch.float32, *stats)):
        return None
    gt = _quick_gate(dev, gate, rows_per_gate, M, N, dt, wdt)
    sq = 0
    for t in ckpts:
        if t is not None:
            s = _quick_rows(dev, (M, _ckpt_bytes(N)), torch.uint8, t)
            if s is None or (sq and s[0] != sq):
                return None
            sq = s[0]
    return None if gt is None else (dev, M, N, dt, wdt, st, sq, gt)


def norm_block_rms_fwd(x, residual, w_post, w_pre, y, h_out, rstd_post=None, rstd_pre=None, gate=None,
                       rows_per_gate=None, x_ckpt=None, h_ckpt=None, ckpt_format=NORM_SAVED_FULL, residual_scale=1.0,
                       block_scale=1.0, offset=0.0, eps=1e-6, stream=None):
    """h_out = residual_scale * residual + block_scale * gate * RMSNorm(x; w_post)
    and y = RMSNorm(h; w_pre), weights taken as (w + offset).

    w_post None: no norm of x; w_pre (and y) None: no norm of h.  gate: None,
    [N], or [rows, N] with rows_per_gate consecutive rows each.  rstd_* (FP32,
    [M]) and the checkpoints x_ckpt, h_ckpt (of ckpt_format) are for
    norm_block_rms_bwd."""
    q = _quick_block(x, w_post, w_pre, (x, residual, y, h_out), (rstd_post, rstd_pre), (x_ckpt, h_ckpt), gate,
                     rows_per_gate)
    if q is None or residual is None or (y is None) != (w_pre is None) or (y is None and h_out is None):
        dt = _act_dtype(x)
        M, N = x.shape
        wdt = _block_weights(w_post, w_pre, N)
        _mat(residual, "residual", M, N, dt)
        _mat(y, "y", M, N, dt, required=w_pre is not None)
        _mat(h_out, "h_out", M, N, dt, required=y is None)
        _vec(rstd_post, "rstd_post", M, _F32, at_least=True, required=False)
        _vec(rstd_pre, "rstd_pre", M, _F32, at_least=True, required=False)
        gt = _gate(gate, rows_per_gate, M, N, dt, wdt)
        _ckpt(x_ckpt, "x_ckpt", M, N, required=False)
        _ckpt(h_ckpt, "h_ckpt", M, N, required=False)
        if x_ckpt is not None and h_ckpt is not None and M > 1 and x_ckpt.stride(0) != h_ckpt.stride(0):
            raise ValueError("x_ckpt and h_ckpt must have the same row stride")
        dev = _device(x, ("residual", residual), ("w_post", w_post), ("w_pre", w_pre), ("y", y), ("h_out", h_out),
                      ("rstd_post", rstd_post), ("rstd_pre", rstd_pre), ("gate", gate), ("x_ckpt", x_ckpt),
                      ("h_ckpt", h_ckpt))
        q = (dev, M, N, dt, wdt, (_rs(x), _rs(residual), _rs(y), _rs(h_out)),
             _rs(x_ckpt if x_ckpt is not None else h_ckpt), gt)
    dev, M, N, dt, wdt, (sx, sr, sy, sh), sq, (grows, gstride, R, gdt) = q
    _on(dev, lambda: _check("norm_block_rms_fwd", lib.norm_block_rms_fwd(
        _ptr(x), sx, _ptr(residual), sr, _ptr(w_post), _ptr(w_pre), _ptr(gate), gstride, grows, R, _ptr(y), sy,
        _ptr(h_out), sh, _ptr(rstd_post), _ptr(rstd_pre), _ptr(x_ckpt), _ptr(h_ckpt), sq, int(ckpt_format), M, N, float(residual_scale),
        float(block_scale), float(offset), float(eps), DTYPE_CODE[dt], DTYPE_CODE[wdt], gdt, _stream(stream, x))))


def norm_block_rms_bwd(dy, dh_out, x, h, w_post, w_pre, rstd_post, rstd_pre, dx=None, dresidual=None, dw_post=None,
                       dw_pre=None, gate=None, dgate=None, rows_per_gate=None, saved_format=NORM_SAVED_FULL,
                       workspace=None, residual_scale=1.0, block_scale=1.0, offset=0.0, stream=None):
    """Gradients of norm_block_rms_fwd (None = not wanted) at the saved x and h,
    which are rows of the activations' dtype or, with saved_format E4M3 / INT8,
    their checkpoints.  dgate has gate's shape and dtype."""
    first, name = (dy, "dy") if dy is not None else (dh_out, "dh_out")
    full = saved_format == NORM_SAVED_FULL
    q = _quick_block(first, w_post, w_pre, (dy, dh_out, x, h, dx, dresidual) if full else (dy, dh_out, dx, dresidual),
                     (rstd_post, rstd_pre), () if full else (x, h), gate, rows_per_gate)
    if q is not None and (
            (dy is None) != (w_pre is None) or (dh_out is None and w_pre is None)
            or (x is None and (w_post is not None or dgate is not None)) or (h is None and w_pre is not None)
            or (rstd_post is None and w_post is not None) or (rstd_pre is None and w_pre is not None)
            or (dgate is not None and (gate is None or not _on_dev(dgate, q[0]) or dgate.shape != gate.shape
                                       or dgate.dtype is not gate.dtype or dgate.stride(-1) != 1))
            or not _quick_vecs(q[0], q[2], q[4], dw_post, dw_pre)
            or not _on_dev(workspace, q[0])):
        q = None   # wrong or unusual: the checks below say which
    if q is not None:
        dev, M, N, dt, wdt, st, sq, (grows, gstride, R, gdt) = q
        dwt = DTYPE_CODE[wdt]
        if full:
            sdy, sdh, sx, sh, sdx, sdr = st
        else:
            (sdy, sdh, sdx, sdr), sx, sh = st, sq, sq
    else:
        dt = _act_dtype(first, name)
        M, N = first.shape
        wdt = _block_weights(w_post, w_pre, N)
        _mat(dy, "dy", M, N, dt, required=w_pre is not None)
        if w_pre is None and dy is not None:
            raise ValueError("dy is given without w_pre")
        _mat(dh_out, "dh_out", M, N, dt, required=w_pre is None)
        for t, n, req in ((x, "x", w_post is not None or dgate is not None), (h, "h", w_pre is not None)):
            if full:
                _mat(t, n, M, N, dt, required=req)
            else:
                _ckpt(t, n, M, N, required=req)
        _vec(rstd_post, "rstd_post", M, _F32, at_least=True, required=w_post is not None)
        _vec(rstd_pre, "rstd_pre", M, _F32, at_least=True, required=w_pre is not None)
        _mat(dx, "dx", M, N, dt, required=False)
        _mat(dresidual, "dresidual", M, N, dt, required=False)
        _vec(dw_post, "dw_post", N, (torch.float32, wdt), required=False)
        _vec(dw_pre, "dw_pre", N, (torch.float32, wdt), required=False)
        dwt = _grad_dtype(wdt, ("dw_post", dw_post), ("dw_pre", dw_pre))
        grows, gstride, R, gdt = _gate(gate, rows_per_gate, M, N, dt, wdt)
        if dgate is not None:
            if gate is None:
                raise ValueError("dgate is given without a gate")
            _tensor(dgate, "dgate")
            if tuple(dgate.shape) != tuple(gate.shape) or dgate.dtype != gate.dtype:
                raise ValueError(f"dgate must have gate's shape {tuple(gate.shape)} and dtype {gate.dtype}, got "
                                 f"{tuple(dgate.shape)}, {dgate.dtype}")
            if N > 1 and dgate.stride(-1) != 1:
                raise ValueError("dgate rows must be contiguous (stride(-1) == 1)")
        dev = _device(first, ("dh_out", dh_out), ("x", x), ("h", h), ("w_post", w_post), ("w_pre", w_pre),
                      ("rstd_post", rstd_post), ("rstd_pre", rstd_pre), ("gate", gate), ("dx", dx),
                      ("dresidual", dresidual), ("dgate", dgate), ("dw_post", dw_post), ("dw_pre", dw_pre),
                      ("workspace", workspace))
        sdy, sdh, sx, sh, sdx, sdr = _rs(dy), _rs(dh_out), _rs(x), _rs(h), _rs(dx), _rs(dresidual)
    dgstride = 0 if dgate is None else dgate.stride(0) if dgate.dim() == 2 else dgate.shape[-1]
    wsp, wsb = _ws(workspace)
    _on(dev, lambda: _check("norm_block_rms_bwd", lib.norm_block_rms_bwd(
        _ptr(dy), sdy, _ptr(dh_out), sdh, _ptr(x), sx, _ptr(h), sh, int(saved_format), _ptr(w_post), _ptr(w_pre),
        _ptr(rstd_post), _ptr(rstd_pre), _ptr(gate), gstride, grows, R, _ptr(dx), sdx, _ptr(dresidual), sdr,
        _ptr(dgate), dgstride, _ptr(dw_post), _ptr(dw_pre), dwt, wsp, wsb, M, N, float(residual_scale), float(block_scale),
        float(offset), DTYPE_CODE[dt], DTYPE_CODE[wdt], gdt, _stream(stream, first))))
