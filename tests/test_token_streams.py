"""The token operators' binding without a GPU: what a call touches is recorded on
the stream it is called for, and what it refuses before it reaches the library."""
import pytest
import torch

import swiglu_activation_cast_amd as mx
import swiglu_activation_cast_amd._token_binding as kb

T, K, E, H, V = 6, 2, 3, 16, 10


def _routed():
    ids = torch.zeros((T, K), dtype=torch.int64)
    rank = torch.arange(T * K, dtype=torch.int32).view(T, K)
    return torch.randn(T, H), torch.randn(T * K, H), ids, rank, torch.rand(T, K)


def call_expert_sort():
    ids, ws = _routed()[2], torch.empty(64, dtype=torch.uint8)
    return [ids, ws], kb.mxtrain_expert_sort(ids, E, workspace=ws, stream=7)


def call_sort_dispatch():
    x, _, ids, _, _ = _routed()
    ws = torch.empty(64, dtype=torch.uint8)
    return [x, ids, ws], kb.mxtrain_sort_dispatch(x, ids, E, workspace=ws, stream=7)


def call_dispatch_fwd():
    x, _, _, rank, _ = _routed()
    return [x, rank], (kb.mxtrain_dispatch_fwd(x, rank, stream=7),)


def call_dispatch_bwd():
    _, rows, _, rank, _ = _routed()
    return [rows, rank], (kb.mxtrain_dispatch_bwd(rows, rank, stream=7),)


def call_combine_fwd():
    x, rows, _, rank, w = _routed()
    return [rows, rank, w, x], (kb.mxtrain_combine_fwd(rows, rank, w, residual=x, stream=7),)


def call_combine_bwd():
    x, rows, _, rank, w = _routed()
    return [x, rows, rank, w], kb.mxtrain_combine_bwd(x, rows, rank, w, stream=7)


def call_embedding_fwd():
    table, ids = torch.randn(V, H), torch.zeros(T, dtype=torch.int64)
    return [table, ids], (kb.mxtrain_embedding_fwd(table, ids, stream=7),)


def call_embedding_bwd():
    dy, ids, ws = torch.randn(T, H), torch.zeros(T, dtype=torch.int64), torch.empty(1 << 16, dtype=torch.uint8)
    return [dy, ids, ws], (kb.mxtrain_embedding_bwd(dy, ids, V, workspace=ws, stream=7),)


def call_dropout_fwd():
    x, res, state = torch.randn(T, H), torch.randn(T, H), torch.zeros(2, dtype=torch.int64)
    return [x, res, state], (kb.mxtrain_dropout_fwd(x, 0.1, 1, 2, residual=res, state=state, stream=7),)


def call_dropout_bwd():
    dy, state = torch.randn(T, H), torch.zeros(2, dtype=torch.int64)
    return [dy, state], (kb.mxtrain_dropout_bwd(dy, 0.1, 1, 2, state=state, stream=7),)


CALLS = [call_expert_sort, call_sort_dispatch, call_dispatch_fwd, call_dispatch_bwd, call_combine_fwd, call_combine_bwd,
         call_embedding_fwd, call_embedding_bwd, call_dropout_fwd, call_dropout_bwd]


@pytest.mark.parametrize("call", CALLS)
def test_everything_a_call_touches_is_recorded_on_its_stream(monkeypatch, call):
    recorded = []
    monkeypatch.setattr(kb, "_gpu", lambda t, *a, **k: t)
    monkeypatch.setattr(kb, "_call", lambda *a: None)
    monkeypatch.setattr(kb, "_other_stream", lambda device, stream, *ts: recorded.extend(ts))
    inputs, outputs = call()
    held = {id(t) for t in recorded}
    assert all(id(t) in held for t in (*inputs, *outputs))


@pytest.mark.parametrize("call", CALLS)
def test_every_call_passes_the_stream_last(monkeypatch, call):
    seen = []
    monkeypatch.setattr(kb, "_gpu", lambda t, *a, **k: t)
    monkeypatch.setattr(kb, "_call", lambda name, device, *a: seen.append((name, a)))
    monkeypatch.setattr(kb, "_other_stream", lambda *a: None)
    call()
    (name, args), = seen
    assert args[-1] == 7 and len(args) == len(kb._SIGNATURES[name][1])


def test_tensors_off_the_gpu_are_refused():
    for call in CALLS:
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_public_names():
    for name in kb._SIGNATURES:
        if not name.endswith(("_workspace", "_status_str")):
            assert name in mx.__all__ and callable(getattr(mx, name)), name
