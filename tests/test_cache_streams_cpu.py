"""The stream argument of the cache calls: whose device a raw handle and the
default stream belong to (CPU only; nothing is launched)."""
import contextlib
import types

import pytest

from paged_kv_cache_03_gb300 import binding as B


@pytest.fixture
def calls(monkeypatch):
    import torch
    seen = []

    def made(name):
        def make(*args, device=None):
            *handle, dev = (*args, device) if device is not None else args
            return types.SimpleNamespace(kind=name, handle=handle, device=dev)
        return make

    @contextlib.contextmanager
    def current(stream):
        seen.append(stream)
        yield
    monkeypatch.setattr(torch.cuda, "ExternalStream", made("external"))
    monkeypatch.setattr(torch.cuda, "default_stream", made("default"))
    monkeypatch.setattr(torch.cuda, "stream", current)
    return seen


def on(device):
    import torch
    return types.SimpleNamespace(device=torch.device(device))


@B._streamed
def call(query, pool=None, *, workspace=None):
    return query


def test_raw_handles_belong_to_the_tensors_device(calls):
    x = on("cuda:1")
    assert call(x, stream=77) is x and call(query=x, stream=0) is x
    handle, default = calls
    assert (handle.kind, handle.handle, str(handle.device)) == ("external", [77], "cuda:1")
    assert (default.kind, default.handle, str(default.device)) == ("default", [], "cuda:1")


def test_streams_of_another_device_are_refused(calls):
    import torch
    x, stream = on("cuda:1"), types.SimpleNamespace(device=torch.device("cuda:0"))
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        call(x, stream=stream)
    assert not calls
    stream.device = x.device
    assert call(x, stream=stream) is x and calls == [stream]
    assert call(x) is x and len(calls) == 1


@pytest.mark.parametrize("recent", [-1, 21, 2 ** 32])
def test_recent_out_of_range(recent, monkeypatch):
    """(2 ** 32 would reach a C int as 0.)"""
    import torch
    monkeypatch.setattr(B, "_on_device", lambda *a: None)
    table, ctx = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="recent"):
        B._evict("x", None, (), (4, 1, 16), B.PA_BF16, on("cuda:0").device, table, ctx,
                 torch.zeros(1, 1, 32), 20, recent, table, None, torch.zeros(256, dtype=torch.uint8))
