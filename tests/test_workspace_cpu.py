"""Workspaces that the binding allocates itself come from the pool of the stream that the call is queued on: a
block from another stream's pool may still be in use there by work that is queued ahead."""
import pytest
import torch

from partial_activation_sync_caat_b200 import caat as C

BF = torch.bfloat16


class Stop(Exception):
    pass


def test_allocated_with_the_streams_pool(monkeypatch):
    current, seen = [None], []

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    class Buffer:
        def record_stream(self, stream):
            pass

        def data_ptr(self):
            return 256

        def numel(self):
            return 1024

        def element_size(self):
            return 1

    def empty(*_, **__):
        seen.append(current[-1])
        return Buffer()

    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch, "empty", empty)
    side = object()
    C._workspace(None, 1000, 0, side)
    C._workspace(None, 1000, 0, None)
    C.alloc_workspace(1000, "cuda", side)
    C.alloc_workspace(1000)
    assert seen == [side, None, side, None]


def layer(name, **kw):
    X, W, R, g = (torch.zeros(*s, dtype=BF) for s in ((2, 64, 128), (2, 256, 128), (2, 64, 256), (256,)))
    if name == "rowpar_forward":
        return C.caat_rowpar_forward(X, W, R, g, None, 2, 0.5, R, **kw)
    if name == "rowpar_backward":
        return C.caat_rowpar_backward(X, W, R, g, R, None, 2, 0.5, X, W, g.float(), **kw)
    if name == "mlp_forward":
        return C.caat_mlp_forward(R, torch.zeros(2, 512, 256, dtype=BF), torch.zeros(2, 256, 256, dtype=BF), R, g, None, 2, 0.5, R, **kw)
    if name == "tp_local":
        return C.caat_rowpar_tp_local(X[0], W[0], R[0], 0.5, None, R[0], **kw)
    return C.caat_rowpar_tp_local_push(X[0], W[0], R[0], 0.5, R[0], C.TpPeers(), **kw)


@pytest.mark.parametrize("name", ["rowpar_forward", "rowpar_backward", "mlp_forward", "tp_local", "tp_local_push"])
def test_every_call_names_its_stream(monkeypatch, name):
    seen = []

    def alloc(nbytes, device=None, stream=None):
        seen.append(stream)
        raise Stop

    monkeypatch.setattr(C, "alloc_workspace", alloc)
    for stream in ("side", None):
        with pytest.raises(Stop):
            layer(name, stream=stream)
    assert seen == ["side", None]


def test_buffers_of_the_layer_over_devices(monkeypatch):
    from partial_activation_sync_caat_b200.tp import TPRowParallel
    current, seen = [None], []

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    class Layer(TPRowParallel):
        def buffers(self, T, device):
            seen.append(current[-1])
            return super().buffers(T, device)

    monkeypatch.setattr(torch.cuda, "stream", Use)
    layer = Layer(64, 0.5, local_fn=lambda *_, **__: None, finish_fn=lambda *_, **__: None, reduce_fn=lambda zs: None)
    x = torch.zeros(4, 32, dtype=BF)
    layer.forward(x, x, x, x, x, stream="side")
    layer.forward(x, x, x, x, x)
    assert seen == ["side", None]
