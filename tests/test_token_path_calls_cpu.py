"""How the binding of the token path makes its calls: temporary workspaces, streams,
the tensors that its handles keep, and further refusals (no GPU needed)."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from sp_partitioned_transformer_gb300 import build

    build.build()
    import sp_partitioned_transformer_gb300 as tpmlp

    tpmlp.load()
    return tpmlp


@pytest.mark.parametrize("stream,on", [(None, None), ("side", "side"), (77, ("external", 77, "cpu"))])
def test_a_temporary_workspace_is_allocated_on_the_stream_that_uses_it(T, monkeypatch, stream, on):
    """A block of another stream's pool may still be in use there when the call starts."""
    current, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    def allocate(*shape, **kw):
        seen.append(current[-1])
        return empty(*shape, **kw)

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(torch, "empty", allocate)
    ws = T._temporary(1000, "cpu", stream)
    assert seen == [on] and ws.numel() == 1000 and ws.dtype is torch.uint8
    assert T._temporary(0, "cpu", stream).numel() == 256
