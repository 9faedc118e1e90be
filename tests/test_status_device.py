"""prism_query_device_status takes a device in any spelling that torch.device takes."""
import importlib.util

import pytest
import torch

from delta_rule_sequence_b200 import prism as P


class _Library:
    """Stands in for libprism.so: keeps the stream it is asked about."""

    def prism_query_device_status(self, workspace, stream):
        self.asked = workspace, stream
        return P.PRISM_ERR_TIMEOUT


@pytest.fixture
def library(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(P, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(P, "_current_raw_stream", lambda index: 1000 + int(index.__index__()))
    return lib


@pytest.mark.parametrize("device", [None, "cuda", torch.device("cuda"), "cuda:0", torch.device("cuda", 0), 0])
def test_every_spelling_of_the_current_device(library, device):
    assert P.prism_query_device_status(None, device=device) == P.PRISM_ERR_TIMEOUT
    assert library.asked == (None, 1000)


def test_a_stream_with_the_device_unnumbered(library):
    class Stream:
        device, cuda_stream = torch.device("cuda", 0), 77

    assert P.prism_query_device_status(None, Stream(), device="cuda") == P.PRISM_ERR_TIMEOUT
    assert library.asked == (None, 77)
    assert P.prism_query_device_status(None, Stream()) == P.PRISM_ERR_TIMEOUT
    with pytest.raises(ValueError):
        P.prism_query_device_status(None, Stream(), device="cuda:1")


def test_other_devices_are_refused(library):
    with pytest.raises(ValueError):
        P.prism_query_device_status(None, device="cpu")
    assert not hasattr(library, "asked")


def test_a_torch_without_the_raw_stream_lookup(monkeypatch):
    """The lookup is not part of torch's public interface: without it the stream's object gives the handle."""
    source = importlib.util.find_spec(P.__name__)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    module = importlib.util.module_from_spec(source)
    source.loader.exec_module(module)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: type("Stream", (), {"cuda_stream": 2000 + index}))
    assert module._stream(None, torch.device("cuda", 3)) == 2003


@pytest.mark.gpu
def test_on_the_gpu():
    for device in (None, "cuda", "cuda:0", torch.device("cuda")):
        assert P.prism_query_device_status(None, device=device) == P.PRISM_OK
    s = torch.cuda.Stream()
    assert P.prism_query_device_status(None, s, device="cuda") == P.PRISM_OK
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert P.prism_query_device_status(ws) == P.PRISM_OK
