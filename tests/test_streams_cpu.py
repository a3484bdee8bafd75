"""Which torch stream stands for a call's ``stream`` argument, without a GPU: torch's own lookups are stood in for."""

import pytest
import torch

import affine_quantized_gemm_amd as Q
from affine_quantized_gemm_amd import rows

DEVICE = torch.device("cuda", 0)


class Handle:
    """A stream of another library, which has its address in ``cuda_stream``."""

    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def lookups(monkeypatch):
    def external(raw, device=None):
        # torch takes an address of 0 for none given and hands out one of its pool's streams
        return ("external", raw, device) if raw else ("pool", device)

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", device))


def of_the_cache(stream):
    cache = Q.KVCache.__new__(Q.KVCache)
    cache.device = DEVICE
    return cache._as_stream(stream)


def of_the_rows(stream):
    on = rows._On.__new__(rows._On)
    on.device, on.stream = DEVICE, stream
    on.raw = 0x50 if stream is None else int(getattr(stream, "cuda_stream", stream))
    return on.torch_stream()


@pytest.mark.parametrize("of", [of_the_cache, of_the_rows])
def test_the_default_stream_by_its_handle(lookups, of):
    assert of(0) == of(Handle(0)) == ("default", DEVICE)


@pytest.mark.parametrize("of", [of_the_cache, of_the_rows])
def test_other_handles(lookups, of):
    assert of(0x40) == of(Handle(0x40)) == ("external", 0x40, DEVICE)


def test_none_is_the_current_one(lookups):
    assert of_the_rows(None) == ("current", DEVICE)


def test_a_stream_of_torch_is_itself(lookups, monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", Handle)
    for s in (Handle(0), Handle(0x40)):
        assert of_the_cache(s) is s and of_the_rows(s) is s
