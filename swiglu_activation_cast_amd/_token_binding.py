"""ctypes binding of libmxtrain.so's second part, include/mxtrain_tokens.h
(argument marshalling only): tokens sorted by expert and back, embedding
lookup, dropout, and their gradients.

The conventions are those of the training operators' binding: torch tensors on
the GPU, shapes, dtypes and devices checked here, outputs and workspaces
allocated where the caller passes none, the C entry point of the same name on
torch's current stream or on `stream`, no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._train_binding import (_FLOATS, _SIGNATURES, _TYPES, _call, _f32, _gpu, _i64, _int, _other_stream, _out, _p,
                             _place, _stream_of, _workspace, _workspace_bytes)

_u64 = ctypes.c_uint64
_f64 = ctypes.c_double

_SIGNATURES.update({
    "mxtrain_expert_sort_workspace": (_i64, [_i64, _i64]),
    "mxtrain_expert_sort": (_int, [_p, _i64, _int, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _p]),
    "mxtrain_dispatch_fwd": (_int, [_p, _i64, _int, _p, _i64, _i64, _i64, _i64, _p, _i64, _p]),
    "mxtrain_sort_dispatch": (_int, [_p, _i64, _int, _p, _i64, _int, _i64, _i64, _i64, _i64, _i64, _p, _i64, _p, _p,
                                     _p, _p, _i64, _p]),
    "mxtrain_dispatch_bwd": (_int, [_p, _i64, _int, _p, _i64, _i64, _i64, _i64, _p, _i64, _p]),
    "mxtrain_combine_fwd": (_int, [_p, _i64, _int, _p, _p, _int, _p, _i64, _i64, _i64, _i64, _i64, _p, _i64, _p]),
    "mxtrain_combine_bwd": (_int, [_p, _i64, _p, _i64, _int, _p, _p, _int, _i64, _i64, _i64, _i64, _p, _i64, _p, _p]),
    "mxtrain_embedding_fwd": (_int, [_p, _i64, _int, _i64, _i64, _p, _i64, _int, _i64, _i64, _f32, _p, _i64, _int,
                                     _p]),
    "mxtrain_embedding_bwd_workspace": (_i64, [_i64, _i64, _i64, _int, _int]),
    "mxtrain_embedding_bwd": (_int, [_p, _i64, _int, _p, _i64, _int, _i64, _i64, _f32, _i64, _i64, _p, _i64, _int,
                                     _int, _p, _i64, _p]),
    "mxtrain_dropout_fwd": (_int, [_p, _i64, _p, _i64, _int, _i64, _i64, _f64, _u64, _u64, _p, _p, _i64, _p]),
    "mxtrain_dropout_bwd": (_int, [_p, _i64, _int, _i64, _i64, _f64, _u64, _u64, _p, _p, _i64, _p]),
})

# integer types (MXTRAIN_I* in mxtrain_tokens.h)
_INTS = {torch.int32: 0, torch.int64: 1}


def _row_stride(t: torch.Tensor, name: str) -> int:
    """_ld of a matrix, with half of its calls."""
    rows, cols = t.shape
    step, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return step if rows > 1 else max(step, cols)


def _matrix(out: Optional[torch.Tensor], rows: int, cols: int, dtype, device) -> Tuple[torch.Tensor, int]:
    """`out`, checked, or a new matrix, and its row stride.  (Sizes apart, here and
    below: torch reads a tuple 0.35 us slower, a torch.Size 0.9, of a call's 8.)"""
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device), cols
    _out(out, "out", (rows, cols), dtype, device)
    return out, _row_stride(out, "out")


# ------------------------------------------------------- tokens and experts
def _pairs(t, name: str, dtypes, device=None) -> Tuple[int, int]:
    """(T, k) of a tensor [T, k], or [T] for one expert a token."""
    _gpu(t, name, dtypes, 1 if isinstance(t, torch.Tensor) and t.dim() == 1 else 2, device)
    return (t.shape[0], 1) if t.dim() == 1 else (t.shape[0], t.shape[1])


def _id_stride(ids: torch.Tensor) -> int:
    """Elements from one token's ids to the next's."""
    if ids.dim() == 1:
        return ids.stride(0) if ids.shape[0] > 1 else 1
    return _row_stride(ids, "ids")


def _first(first: int) -> int:
    if not -(1 << 63) <= first < 1 << 63:
        raise ValueError(f"first must fit 64 bits, got {first}")
    return first


def _index_out(t: Optional[torch.Tensor], name: str, shape, device) -> torch.Tensor:
    if t is None:
        return torch.empty(*shape, dtype=torch.int32, device=device)
    if t.dtype != torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on the inputs' device")
    return t


def _rank(rank, device) -> Tuple[int, int]:
    T, k = _pairs(rank, "rank", (torch.int32,), device)
    if not rank.is_contiguous():
        raise ValueError("rank must be contiguous")
    return T, k


def _weights(weights, rank: torch.Tensor) -> int:
    _gpu(weights, "weights", _FLOATS, rank.dim(), rank.device)
    if weights.shape != rank.shape or not weights.is_contiguous():
        raise ValueError("weights must be contiguous and have rank's shape")
    return weights.data_ptr()


def mxtrain_expert_sort(ids: torch.Tensor, num_experts: int, *, first: int = 0, rank: Optional[torch.Tensor] = None,
                        ends: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Stable sort of token-expert pairs by expert; returns (rank, ends, order).

    ids: [T, k] (or [T]) experts of each token, int32 or int64; a pair is kept
    where ids - first is in [0, num_experts).  rank, in ids' shape: the pair's
    row among the kept pairs, -1 where dropped.  ends [num_experts]: the
    group_ends of the grouped products.  order [T k]: the pair t k + j in each row,
    -1 past the last.  All int32."""
    T, k = _pairs(ids, "ids", _INTS)
    dev = ids.device
    rank = _index_out(rank, "rank", ids.shape, dev)
    ends = _index_out(ends, "ends", (num_experts,), dev)
    order = _index_out(order, "order", (T * k,), dev)
    ws = _workspace(_workspace_bytes("mxtrain_expert_sort_workspace", T * k, num_experts), workspace, dev)
    if stream is not None:
        _other_stream(dev, stream, ids, rank, ends, order, ws)
    _call("mxtrain_expert_sort", dev, ids.data_ptr(), _id_stride(ids), _INTS[ids.dtype], T, k, _first(first), num_experts,
          rank.data_ptr(), ends.data_ptr(), order.data_ptr(), *_place(ws), _stream_of(dev, stream))
    return rank, ends, order


def mxtrain_dispatch_fwd(x: torch.Tensor, rank: torch.Tensor, *, rows: Optional[int] = None,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The rows of x [T, H] (bf16 or fp32) at the places `rank` [T, k] names: out[rank[t, j]] = x[t].

    out: [rows, H] in x's dtype, rows = T k unless given; rows that no pair
    names are left as they are in `out` (uninitialized when `out` is None)."""
    _gpu(x, "x", _FLOATS, 2)
    dev = x.device
    T, k = _rank(rank, dev)
    if x.shape[0] != T:
        raise ValueError("x and rank must have the same tokens")
    if rows is None:
        rows = T * k if out is None else out.shape[0]
    xs, ld_out = _matrix(out, rows, x.shape[1], x.dtype, dev)
    if stream is not None:
        _other_stream(dev, stream, x, rank, xs)
    _call("mxtrain_dispatch_fwd", dev, x.data_ptr(), _row_stride(x, "x"), _TYPES[x.dtype], rank.data_ptr(), T, k,
          x.shape[1], rows, xs.data_ptr(), ld_out, _stream_of(dev, stream))
    return xs


def mxtrain_sort_dispatch(x: torch.Tensor, ids: torch.Tensor, num_experts: int, *, first: int = 0,
                          out: Optional[torch.Tensor] = None, rank: Optional[torch.Tensor] = None,
                          ends: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """mxtrain_expert_sort and mxtrain_dispatch_fwd in one call; returns (xs, rank, ends, order).

    xs: [T k, H], the rows of x sorted by expert; rows past the last end are left
    as they are in `out` (uninitialized when `out` is None)."""
    _gpu(x, "x", _FLOATS, 2)
    dev = x.device
    T, k = _pairs(ids, "ids", _INTS, dev)
    H = x.shape[1]
    if x.shape[0] != T:
        raise ValueError("x and ids must have the same tokens")
    xs, ld_out = _matrix(out, T * k, H, x.dtype, dev)
    rank = _index_out(rank, "rank", ids.shape, dev)
    ends = _index_out(ends, "ends", (num_experts,), dev)
    order = _index_out(order, "order", (T * k,), dev)
    ws = _workspace(_workspace_bytes("mxtrain_expert_sort_workspace", T * k, num_experts), workspace, dev)
    if stream is not None:
        _other_stream(dev, stream, x, ids, xs, rank, ends, order, ws)
    _call("mxtrain_sort_dispatch", dev, x.data_ptr(), _row_stride(x, "x"), _TYPES[x.dtype], ids.data_ptr(),
          _id_stride(ids), _INTS[ids.dtype], T, k, _first(first), num_experts, H, xs.data_ptr(), ld_out, rank.data_ptr(),
          ends.data_ptr(), order.data_ptr(), *_place(ws), _stream_of(dev, stream))
    return xs, rank, ends, order


def mxtrain_dispatch_bwd(dxs: torch.Tensor, rank: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """Gradient of the dispatch: dx[t] = sum_j dxs[rank[t, j]], [T, H] in dxs' dtype."""
    _gpu(dxs, "dxs", _FLOATS, 2)
    dev = dxs.device
    T, k = _rank(rank, dev)
    R, H = dxs.shape
    dx, ld_out = _matrix(out, T, H, dxs.dtype, dev)
    if stream is not None:
        _other_stream(dev, stream, dxs, rank, dx)
    _call("mxtrain_dispatch_bwd", dev, dxs.data_ptr(), _row_stride(dxs, "dxs"), _TYPES[dxs.dtype], rank.data_ptr(),
          T, k, H, R, dx.data_ptr(), ld_out, _stream_of(dev, stream))
    return dx


def mxtrain_combine_fwd(ys: torch.Tensor, rank: torch.Tensor, weights: torch.Tensor, *,
                        residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """The experts' rows summed back: y[t] = residual[t] + sum_j weights[t, j] ys[rank[t, j]].

    ys [R, H] in bf16 or fp32, rank [T, k] as the sort gave it (dropped pairs
    add nothing), weights of rank's shape in bf16 or fp32, residual [T, H] in ys'
    dtype or None.  Returns [T, H] in ys' dtype."""
    _gpu(ys, "ys", _FLOATS, 2)
    dev = ys.device
    T, k = _rank(rank, dev)
    R, H = ys.shape
    pw = _weights(weights, rank)
    if residual is not None:
        _gpu(residual, "residual", (ys.dtype,), 2, dev)
        if residual.shape != (T, H):
            raise ValueError(f"residual must have shape {(T, H)}, got {tuple(residual.shape)}")
    y, ld_out = _matrix(out, T, H, ys.dtype, dev)
    if stream is not None:
        _other_stream(dev, stream, ys, rank, weights, residual, y)
    _call("mxtrain_combine_fwd", dev, ys.data_ptr(), _row_stride(ys, "ys"), _TYPES[ys.dtype], rank.data_ptr(), pw,
          _TYPES[weights.dtype], None if residual is None else residual.data_ptr(),
          0 if residual is None else _row_stride(residual, "residual"), T, k, H, R, y.data_ptr(), ld_out,
          _stream_of(dev, stream))
    return y


def mxtrain_combine_bwd(dy: torch.Tensor, ys: torch.Tensor, rank: torch.Tensor, weights: torch.Tensor, *,
                        out: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of mxtrain_combine_fwd for upstream dy [T, H]; returns (dys, dweights).

    dys [R, H] in ys' dtype: dys[rank[t, j]] = weights[t, j] dy[t]; rows that no
    pair names are left as they are in `out` (uninitialized when `out` is None).
    dweights, fp32 in rank's shape: <dy[t], ys[rank[t, j]]>, 0 for dropped
    pairs.  residual's gradient is dy."""
    _gpu(ys, "ys", _FLOATS, 2)
    dev = ys.device
    _gpu(dy, "dy", (ys.dtype,), 2, dev)
    T, k = _rank(rank, dev)
    R, H = ys.shape
    if dy.shape != (T, H):
        raise ValueError(f"dy must have shape {(T, H)}, got {tuple(dy.shape)}")
    pw = _weights(weights, rank)
    dys, ld_out = _matrix(out, R, H, ys.dtype, dev)
    if dweights is None:
        dweights = torch.empty(*rank.shape, dtype=torch.float32, device=dev)
    elif (dweights.dtype != torch.float32 or dweights.device != dev or dweights.shape != rank.shape
          or not dweights.is_contiguous()):
        raise ValueError("dweights must be a contiguous float32 tensor of rank's shape on the inputs' device")
    if stream is not None:
        _other_stream(dev, stream, dy, ys, rank, weights, dys, dweights)
    _call("mxtrain_combine_bwd", dev, dy.data_ptr(), _row_stride(dy, "dy"), ys.data_ptr(), _row_stride(ys, "ys"),
          _TYPES[ys.dtype], rank.data_ptr(), pw, _TYPES[weights.dtype], T, k, H, R, dys.data_ptr(), ld_out,
          dweights.data_ptr(), _stream_of(dev, stream))
    return dys, dweights


# ----------------------------------------------------------------- embedding
def _tokens(ids, device) -> Tuple[int, int]:
    """(T, stride) of token ids: any stride in one dimension, adjacent in several."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError(f"ids must be an int32 or int64 tensor, got {type(ids).__name__}")
    _gpu(ids, "ids", _INTS, ids.dim(), device)
    if ids.dim() == 1 and ids.shape[0] > 1:
        return ids.shape[0], ids.stride(0)
    if not ids.is_contiguous():
        raise ValueError("ids of several dimensions must be contiguous")
    return ids.numel(), 1


def _rows_of(t, name: str, dtypes, ids: torch.Tensor, device) -> torch.Tensor:
    """t [*ids, H] as rows [T, H]."""
    _gpu(t, name, dtypes, ids.dim() + 1, device)
    if t.shape[:-1] != ids.shape:
        raise ValueError(f"{name} must have shape {(*ids.shape, 'H')}, got {tuple(t.shape)}")
    if t.dim() == 2:
        return t
    if not t.is_contiguous():
        raise ValueError(f"{name} of more than two dimensions must be contiguous")
    return t.view(ids.numel(), t.shape[-1])


def mxtrain_embedding_fwd(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, first: int = 0,
                          out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Rows of weight [V, H] (bf16 or fp32) times `scale`: [*ids, H] in `out`'s dtype, `out_dtype`, or weight's.

    ids: int32 or int64, any shape (strided where one-dimensional); the row is
    ids - first, zeros where that is not in [0, V)."""
    _gpu(weight, "weight", _FLOATS, 2)
    dev = weight.device
    V, H = weight.shape
    T, step = _tokens(ids, dev)
    dtype = out.dtype if out is not None else out_dtype or weight.dtype
    if dtype not in _TYPES:
        raise TypeError(f"results are bfloat16 or float32, not {dtype}")
    if out is None:
        y, ld_out = torch.empty(*ids.shape, H, dtype=dtype, device=dev), H
    else:
        y = _out(out, "out", (*ids.shape, H), dtype, dev)
        ld_out = _row_stride(_rows_of(y, "out", _FLOATS, ids, dev), "out")
    if stream is not None:
        _other_stream(dev, stream, weight, ids, y)
    _call("mxtrain_embedding_fwd", dev, weight.data_ptr(), _row_stride(weight, "weight"), _TYPES[weight.dtype], V, H,
          ids.data_ptr(), step, _INTS[ids.dtype], T, _first(first), scale, y.data_ptr(), ld_out, _TYPES[dtype],
          _stream_of(dev, stream))
    return y


def mxtrain_embedding_bwd(dy: torch.Tensor, ids: torch.Tensor, num_embeddings: int, *, scale: float = 1.0,
                          first: int = 0, out_dtype: torch.dtype = torch.float32,
                          out: Optional[torch.Tensor] = None, accumulate: bool = False,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of mxtrain_embedding_fwd for upstream dy [*ids, H] (bf16 or fp32).

    dweight [num_embeddings, H] in `out`'s dtype or `out_dtype`: scale times the sum
    of the rows of dy whose id - first is the row's number, zeros where there
    are none.  accumulate=True adds to the rows of `out` that tokens name and
    leaves the others alone."""
    if not isinstance(dy, torch.Tensor) or not isinstance(ids, torch.Tensor):
        raise TypeError("dy and ids must be tensors")
    _gpu(dy, "dy", _FLOATS, ids.dim() + 1)
    dev = dy.device
    T, step = _tokens(ids, dev)
    rows = _rows_of(dy, "dy", _FLOATS, ids, dev)
    H = dy.shape[-1]
    if accumulate and out is None:
        raise ValueError("accumulate needs the `out` to add to")
    dtype = out.dtype if out is not None else out_dtype
    if dtype not in _TYPES:
        raise TypeError(f"results are bfloat16 or float32, not {dtype}")
    dw, ld_out = _matrix(out, num_embeddings, H, dtype, dev)
    ws = _workspace(_workspace_bytes("mxtrain_embedding_bwd_workspace", T, num_embeddings, H, _TYPES[dy.dtype],
                                     _TYPES[dtype]), workspace, dev)
    if stream is not None:
        _other_stream(dev, stream, dy, ids, dw, ws)
    _call("mxtrain_embedding_bwd", dev, rows.data_ptr(), _row_stride(rows, "dy"), _TYPES[dy.dtype], ids.data_ptr(),
          step, _INTS[ids.dtype], T, _first(first), scale, num_embeddings, H, dw.data_ptr(), ld_out, _TYPES[dtype],
          int(accumulate), *_place(ws), _stream_of(dev, stream))
    return dw


# ------------------------------------------------------------------- dropout
def _word(v: int, name: str) -> int:
    if not 0 <= v < 1 << 64:
        raise ValueError(f"{name} must be in [0, 2^64), got {v}")
    return v


def _state(state: Optional[torch.Tensor], device) -> Optional[int]:
    if state is None:
        return None
    _gpu(state, "state", (torch.int64,), 1, device)
    if state.shape[0] != 2 or not state.is_contiguous():
        raise ValueError("state must hold two adjacent int64")
    return state.data_ptr()


def mxtrain_dropout_fwd(x: torch.Tensor, p: float, seed: int, offset: int, *,
                        residual: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """residual + dropout(x) of x [M, N] (bf16 or fp32), in x's dtype.

    An element is dropped with probability t / 65536, t = round(65536 p), and
    multiplied by 65536 / (65536 - t) otherwise.  The mask is a function of p,
    seed, offset, row and column (Philox4x32-10, include/mxtrain_tokens.h): give
    every call an offset of its own.  state: int64 [2] on the device, added to
    (seed, offset), so that a captured graph can draw new masks."""
    _gpu(x, "x", _FLOATS, 2)
    dev = x.device
    M, N = x.shape
    if residual is not None:
        _gpu(residual, "residual", (x.dtype,), 2, dev)
        if residual.shape != x.shape:
            raise ValueError("residual and x must have the same shape")
    y, ld_out = _matrix(out, M, N, x.dtype, dev)
    ps = _state(state, dev)
    if stream is not None:
        _other_stream(dev, stream, x, residual, state, y)
    _call("mxtrain_dropout_fwd", dev, x.data_ptr(), _row_stride(x, "x"),
          None if residual is None else residual.data_ptr(),
          0 if residual is None else _row_stride(residual, "residual"), _TYPES[x.dtype], M, N, p, _word(seed, "seed"),
          _word(offset, "offset"), ps, y.data_ptr(), ld_out, _stream_of(dev, stream))
    return y


def mxtrain_dropout_bwd(dy: torch.Tensor, p: float, seed: int, offset: int, *, state: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of mxtrain_dropout_fwd with the same p, seed, offset and state: the
    same mask on dy [M, N] (residual's gradient is dy)."""
    _gpu(dy, "dy", _FLOATS, 2)
    dev = dy.device
    M, N = dy.shape
    dx, ld_out = _matrix(out, M, N, dy.dtype, dev)
    ps = _state(state, dev)
    if stream is not None:
        _other_stream(dev, stream, dy, state, dx)
    _call("mxtrain_dropout_bwd", dev, dy.data_ptr(), _row_stride(dy, "dy"), _TYPES[dy.dtype], M, N, p,
          _word(seed, "seed"), _word(offset, "offset"), ps, dx.data_ptr(), ld_out, _stream_of(dev, stream))
    return dx
