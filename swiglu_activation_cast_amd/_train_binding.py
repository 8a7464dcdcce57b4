"""ctypes binding of libmxtrain.so (argument marshalling only).

The training operators beside the MXFP8 casts: layer norm, the experts' bf16
products and the orthogonalised weight update.  As in the casts' binding,
every function takes torch tensors that live on the GPU, checks shapes,
dtypes and devices (the C ABI sees bare pointers), allocates outputs and
workspaces with torch where the caller passes none, and calls the C entry
point of the same name on torch's current stream, or on `stream`.  There is no
CPU or PyTorch fallback.

On a `stream` other than the current one, what the call allocates comes from
the current stream's pool: memory whose last use may still be running there,
and which torch hands out again once it is freed here, as it does an input's
that the caller drops.  So the other stream first waits for the current one,
and inputs, outputs and workspace are recorded on it (_other_stream).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
TRAIN_LIB_PATH = os.path.join(_PKG_DIR, "libmxtrain.so")

_i64 = ctypes.c_int64
_p = ctypes.c_void_p
_int = ctypes.c_int
_f32 = ctypes.c_float

_SIGNATURES = {
    "mxtrain_layer_norm_fwd": (_int, [_p, _i64, _p, _p, _int, _i64, _i64, _int, _f32, _p, _i64, _p, _p, _p]),
    "mxtrain_layer_norm_bwd_workspace": (_i64, [_i64, _i64]),
    "mxtrain_layer_norm_bwd": (_int, [_p, _i64, _p, _i64, _p, _p, _p, _int, _i64, _i64, _int, _p, _i64, _p, _p, _p,
                                      _i64, _p]),
    "mxtrain_grouped_gemm": (_int, [_p, _i64, _p, _i64, _i64, _int, _p, _i64, _i64, _i64, _i64, _p, _i64, _int, _p]),
    "mxtrain_grouped_gemm_k": (_int, [_p, _i64, _p, _i64, _p, _i64, _i64, _i64, _i64, _p, _i64, _i64, _int, _p]),
    "mxtrain_newton_schulz_workspace": (_i64, [_i64, _i64, _i64, _int]),
    "mxtrain_newton_schulz": (_int, [_p, _i64, _i64, _int, _i64, _i64, _i64, _int, _p, _f32, _p, _i64, _i64, _int, _p,
                                     _i64, _p]),
    "mxtrain_status_str": (ctypes.c_char_p, [_int]),
}

# element types (MXTRAIN_* in mxtrain.h)
_TYPES = {torch.bfloat16: 0, torch.float32: 1}

_train_lib = None


class MxtrainError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


def train_lib() -> ctypes.CDLL:
    """The loaded libmxtrain.so with argument types set (raises if not built)."""
    global _train_lib
    if _train_lib is not None:
        return _train_lib
    if not os.path.exists(TRAIN_LIB_PATH):
        raise RuntimeError(
            f"{TRAIN_LIB_PATH} is not built; run `python -m swiglu_activation_cast_amd._build` "
            "(or __graft_entry__.build()) first"
        )
    handle = ctypes.CDLL(TRAIN_LIB_PATH)
    for name, (restype, argtypes) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.argtypes = argtypes
        fn.restype = restype
    _train_lib = handle
    return handle


def train_status_str(status: int) -> str:
    return train_lib().mxtrain_status_str(int(status)).decode()


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    return getattr(train_lib(), name)


def _call(name: str, device: torch.device, *args) -> None:
    """The C call with `device` current; raises on a status."""
    fn = _entry(name)
    if device.index == torch.cuda.current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != 0:
        raise MxtrainError(name, status, train_status_str(status))


# The current stream's handle without building a torch Stream object around
# it: 0.1 us of a small call's 10, against 1.9.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: torch.device, stream) -> int:
    if stream is None:
        return _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    return _entry(name)(*sizes)


def _other_stream(device: torch.device, stream, *tensors) -> None:
    """Makes `stream`, where it is not the current one, wait for the current
    one, and keeps the tensors' memory from being reused before it is done."""
    current = torch.cuda.current_stream(device)
    handle = _stream_of(device, stream)
    if handle != current.cuda_stream:
        if hasattr(stream, "wait_stream"):
            other = stream
        elif handle == 0:  # an ExternalStream of handle 0 would be a new stream
            other = torch.cuda.default_stream(device)
        else:
            other = torch.cuda.ExternalStream(handle, device=device)
        other.wait_stream(current)
        for t in tensors:
            if t is not None:
                t.record_stream(other)


def _workspace(nbytes: int, given: Optional[torch.Tensor], device: torch.device) -> Optional[torch.Tensor]:
    """`given`, checked, or a new workspace."""
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        if given.numel() * given.element_size() < nbytes:
            raise ValueError(f"workspace must hold at least {nbytes} bytes")
        return given
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _place(ws: Optional[torch.Tensor]) -> Tuple[Optional[int], int]:
    """A workspace's address and bytes."""
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _gpu(t, name: str, dtypes, dim: int, device=None) -> torch.Tensor:
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda and t.dim() == dim
            and (device is None or t.device == device)):
        return t
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        want = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise TypeError(f"{name} must be a {want} tensor, got {getattr(t, 'dtype', type(t).__name__)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")


def _ld(t: torch.Tensor, name: str) -> int:
    """Row stride of the last two dimensions, whose columns must be adjacent."""
    rows, cols = t.shape[-2:]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.stride(-2) if rows > 1 else max(t.stride(-2), cols)


def _vector(t: Optional[torch.Tensor], name: str, n: int, device, dtypes) -> Optional[int]:
    """Address of n adjacent elements, or None."""
    if t is None:
        return None
    if t.dtype in dtypes and t.device == device and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    _gpu(t, name, dtypes, 1, device)
    raise ValueError(f"{name} must hold {n} adjacent elements")


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _gpu(t, name, (dtype,), len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _f32_out(t: Optional[torch.Tensor], name: str, n: int, device) -> Tuple[torch.Tensor, int]:
    """An fp32 vector of n elements, given or new, and its address."""
    if t is None:
        t = torch.empty(n, dtype=torch.float32, device=device)
        return t, t.data_ptr()
    return t, _vector(t, name, n, device, _F32)


_F32 = (torch.float32,)
_FLOATS = (torch.bfloat16, torch.float32)


def mxtrain_layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                           out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                           rstd: Optional[torch.Tensor] = None, stream=None
                           ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm of the rows of x [M, N] (bf16 or fp32); returns (y, mean, rstd).

    y = (x - mean) * rstd * weight + bias in x's dtype, with the fp32 row
    statistics [M] that the backward pass reads.  weight and bias: [N], bf16
    or fp32 (the same), or None."""
    _gpu(x, "x", _FLOATS, 2)
    M, N = x.shape
    dev = x.device
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    pw, pb = _vector(weight, "weight", N, dev, _FLOATS), _vector(bias, "bias", N, dev, _FLOATS)
    param = weight if weight is not None else bias
    y = _out(out, "out", x.shape, x.dtype, dev)
    mean, pm = _f32_out(mean, "mean", M, dev)
    rstd, pr = _f32_out(rstd, "rstd", M, dev)
    if stream is not None:
        _other_stream(dev, stream, x, weight, bias, y, mean, rstd)
    _call("mxtrain_layer_norm_fwd", dev, x.data_ptr(), _ld(x, "x"), pw, pb,
          0 if param is None else _TYPES[param.dtype], M, N, _TYPES[x.dtype], eps, y.data_ptr(), _ld(y, "out"),
          pm, pr, _stream_of(dev, stream))
    return y, mean, rstd


def mxtrain_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                           weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
                           dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None
                           ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of mxtrain_layer_norm_fwd for upstream dy; returns (dx, dweight, dbias).

    dx has x's dtype; dweight and dbias are fp32 [N] sums over the rows."""
    _gpu(x, "x", _FLOATS, 2)
    M, N = x.shape
    dev = x.device
    _gpu(dy, "dy", (x.dtype,), 2, dev)
    if dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape")
    pw = _vector(weight, "weight", N, dev, _FLOATS)
    pm, pr = _vector(mean, "mean", M, dev, _F32), _vector(rstd, "rstd", M, dev, _F32)
    dx = _out(out, "out", x.shape, x.dtype, dev)
    dw, pdw = _f32_out(dweight, "dweight", N, dev)
    db, pdb = _f32_out(dbias, "dbias", N, dev)
    ws = _workspace(_workspace_bytes("mxtrain_layer_norm_bwd_workspace", M, N), workspace, dev)
    if stream is not None:
        _other_stream(dev, stream, dy, x, mean, rstd, weight, dx, dw, db, ws)
    _call("mxtrain_layer_norm_bwd", dev, dy.data_ptr(), _ld(dy, "dy"), x.data_ptr(), _ld(x, "x"), pm, pr, pw,
          0 if weight is None else _TYPES[weight.dtype], M, N, _TYPES[x.dtype], dx.data_ptr(), _ld(dx, "out"),
          pdw, pdb, *_place(ws), _stream_of(dev, stream))
    return dx, dw, db


def _ends(t: torch.Tensor, device) -> Tuple[int, int]:
    _gpu(t, "group_ends", (torch.int32,), 1, device)
    if t.shape[0] > 1 and t.stride(0) != 1:
        raise ValueError("group_ends must be contiguous")
    return t.data_ptr(), t.shape[0]


def _out_dtype(out: Optional[torch.Tensor], out_dtype: torch.dtype) -> torch.dtype:
    dtype = out.dtype if out is not None else out_dtype
    if dtype not in _TYPES:
        raise TypeError(f"results are bfloat16 or float32, not {dtype}")
    return dtype


def mxtrain_grouped_gemm(a: torch.Tensor, b: torch.Tensor, group_ends: torch.Tensor, *, transpose_b: bool = True,
                         out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """The experts' products in bf16: row i of a [M, K], in group g, times b[g].

    transpose_b True: b [G, N, K], a_g b_g^T (forward); False: b [G, K, N],
    a_g b_g (input gradient).  group_ends: device int32 [G], cumulative row
    ends of any group sizes, read on the GPU only.  Returns [M, N] in `out`'s
    dtype or `out_dtype` (bf16 or fp32); rows past the last end are left as
    they are in `out` (uninitialized when `out` is None)."""
    _gpu(a, "a", (torch.bfloat16,), 2)
    dev = a.device
    _gpu(b, "b", (torch.bfloat16,), 3, dev)
    pe, G = _ends(group_ends, dev)
    M, K = a.shape
    N, kb = (b.shape[1], b.shape[2]) if transpose_b else (b.shape[2], b.shape[1])
    if b.shape[0] != G or kb != K:
        raise ValueError(f"b must be [{G}, N, {K}] (transpose_b) or [{G}, {K}, N], got {tuple(b.shape)}")
    c = _out(out, "out", (M, N), _out_dtype(out, out_dtype), dev)
    ldb = _ld(b, "b")
    if stream is not None:
        _other_stream(dev, stream, a, b, group_ends, c)
    _call("mxtrain_grouped_gemm", dev, a.data_ptr(), _ld(a, "a"), b.data_ptr(), ldb,
          b.stride(0) if G > 1 else 0, int(transpose_b), pe, G, M, N, K, c.data_ptr(), _ld(c, "out"),
          _TYPES[c.dtype], _stream_of(dev, stream))
    return c


def mxtrain_grouped_gemm_k(a: torch.Tensor, b: torch.Tensor, group_ends: torch.Tensor, *,
                           out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """The experts' weight gradients: a_g^T b_g [G, M, N] over each group's
    tokens, a [T, M] and b [T, N] in bf16; an empty group gives zeros."""
    _gpu(a, "a", (torch.bfloat16,), 2)
    dev = a.device
    _gpu(b, "b", (torch.bfloat16,), 2, dev)
    pe, G = _ends(group_ends, dev)
    T, M = a.shape
    N = b.shape[1]
    if b.shape[0] != T:
        raise ValueError("a [T, M] and b [T, N] must have the same tokens")
    c = _out(out, "out", (G, M, N), _out_dtype(out, out_dtype), dev)
    ldc = _ld(c, "out")
    if stream is not None:
        _other_stream(dev, stream, a, b, group_ends, c)
    _call("mxtrain_grouped_gemm_k", dev, a.data_ptr(), _ld(a, "a"), b.data_ptr(), _ld(b, "b"), pe, G, M, N, T,
          c.data_ptr(), ldc, c.stride(0) if G > 1 else max(ldc * M, 1), _TYPES[c.dtype], _stream_of(dev, stream))
    return c


def mxtrain_newton_schulz(g: torch.Tensor, *, steps: int = 5,
                          coeffs: Sequence[float] = (3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                          out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Orthogonalised update of each matrix of g [m, n] or [B, m, n] (bf16 or fp32).

    X = g / (|g| + eps), then `steps` times X <- a X + b (X X^T) X +
    c (X X^T)^2 X with (a, b, c) = coeffs.  Returns g's shape in `out`'s
    dtype, `out_dtype`, or g's; the workspace is
    mxtrain_newton_schulz_workspace(B, m, n, type) bytes, 256-byte aligned."""
    if not isinstance(g, torch.Tensor) or g.dim() not in (2, 3):
        raise ValueError("g must be a matrix [m, n] or a batch [B, m, n]")
    _gpu(g, "g", _FLOATS, g.dim())
    dev = g.device
    if len(coeffs) != 3:
        raise ValueError("coeffs must be three numbers")
    c = _out(out, "out", tuple(g.shape), _out_dtype(out, out_dtype or g.dtype), dev)
    m, n = g.shape[-2:]
    batch = g.shape[0] if g.dim() == 3 else 1
    ld_g, ld_c = _ld(g, "g"), _ld(c, "out")
    several = g.dim() == 3 and batch > 1
    stride_g = g.stride(0) if several else 0
    stride_c = c.stride(0) if several else 0
    nbytes = _workspace_bytes("mxtrain_newton_schulz_workspace", batch, m, n, _TYPES[c.dtype])
    ws = _workspace(nbytes, workspace, dev)
    if stream is not None:
        _other_stream(dev, stream, g, c, ws)
    _call("mxtrain_newton_schulz", dev, g.data_ptr(), ld_g, stride_g, _TYPES[g.dtype], batch, m, n, int(steps),
          (ctypes.c_float * 3)(*coeffs), eps, c.data_ptr(), ld_c, stride_c, _TYPES[c.dtype], *_place(ws),
          _stream_of(dev, stream))
    return c
