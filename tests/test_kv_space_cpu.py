"""The workspace that attention finds for itself, without a GPU: streams and their state of capture are stood in for."""

import contextlib

import pytest
import torch

import affine_quantized_gemm_amd as Q
from affine_quantized_gemm_amd import kv

HERE, THERE = 0x10, 0x20  # the current stream and another


@pytest.fixture
def cache(monkeypatch):
    """A cache on the CPU, of which only workspaces are asked."""
    c = Q.KVCache.__new__(Q.KVCache)
    c.device, c._spaces, c._most_space = torch.device("cpu"), {}, kv.ATTEND_ZEROED_BYTES + 32768 * 132
    g = kv._Geometry(0, 64, 128, 8, 64, 1, 9, 0x10000)
    c._geometry, c._c = g, kv.ctypes.byref(g)
    c.current, c.capturing = [HERE], set()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: c.current[-1] in c.capturing)

    @contextlib.contextmanager
    def on(stream):
        c.current.append(stream)
        yield
        c.current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    c._as_stream = lambda s: s
    return c


LONG, SHORT = (1, 1, 1, 32, 100000), (1, 1, 1, 32, 100)


def test_eager_calls_keep_one_a_stream(cache):
    a, n = cache._own_space(None, HERE, *LONG)
    assert n == a.numel() == cache._most_space and not a.any()
    assert cache._own_space(None, HERE, *SHORT)[0] is a
    b, _ = cache._own_space(THERE, THERE, *LONG)
    assert b is not a and cache._own_space(THERE, THERE, *LONG)[0] is b and set(cache._spaces) == {HERE, THERE}


@pytest.mark.parametrize("stream", [None, THERE])
def test_a_captured_call_has_one_of_its_own(cache, stream):
    """Of the call's stream, not of the current one: a kept workspace zeroed in a graph would not be zeroed yet."""
    raw = HERE if stream is None else THERE
    cache.capturing = {raw}
    need = cache.attend_workspace_bytes(*LONG)
    a, n = cache._own_space(stream, raw, *LONG)
    assert n == need == a.numel() > kv.ATTEND_ZEROED_BYTES and not a[:kv.ATTEND_ZEROED_BYTES].any()
    assert not cache._spaces and cache._own_space(stream, raw, *LONG)[0] is not a


@pytest.mark.parametrize("stream", [None, THERE])
def test_a_captured_call_that_needs_none_fills_none(cache, stream):
    cache.capturing = {HERE if stream is None else THERE}
    assert cache.attend_workspace_bytes(*SHORT) == 0
    assert cache._own_space(stream, HERE if stream is None else THERE, *SHORT) == (None, 0)


def test_an_eager_call_while_another_stream_is_captured(cache):
    cache.capturing = {HERE}
    a, n = cache._own_space(THERE, THERE, *LONG)
    assert n == cache._most_space and cache._spaces == {THERE: a}


# ---- sizes ----

@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_tables_of_more_tokens_than_positions_reach_are_refused(page):
    """Attention looks up to 256 tokens ahead of a position, in 32 bits: near 2^31 tokens its loops would not end."""
    L, A, most = Q._lib, 0x10000, (1 << 30) // page  # (addresses are never dereferenced)
    g = kv.ctypes.byref(kv._Geometry(0, 64, 128, 8, page, 1, 9, A))
    for width, status in ((most, Q.QMM_ERR_INVALID_ARG), (most + 1, Q.QMM_ERR_UNSUPPORTED),
                          (((1 << 31) - 1) // page, Q.QMM_ERR_UNSUPPORTED)):
        # (the width that is served is refused for a NULL operand)
        assert L.qmm_kv_attend(g, 0, 1, 1, 1, A, width, A, None, None, 128, 128, 8, 1.0, None, A, None, 100, A, 1 << 30, None) == status
        assert L.qmm_kv_append(g, 0, 1, 1, 1, A, width, A, None, None, 128, 128, A, 128, 128, None) == status
        assert L.qmm_kv_read(g, 0, 1, 1, 1, A, width, A, None, None, A, None) == status
        assert L.qmm_kv_reserve(g, 1, A, width, A, A, None, A, A, 1 << 30, None) == status
        assert L.qmm_kv_fork(g, 1, A, width, A, A, None, A, 1, A, A, 1 << 30, None) == status
        assert L.qmm_kv_free(g, 1, A, width, A, A, None, 1, None) == status
        assert L.qmm_kv_compact(g, 1, A, width, A, A, A, None, A, 1 << 30, None) == status
