"""Calls on a stream that is given by its handle, the default stream's 0 among them: their work, their workspace's zeroing and
their outputs are in that stream's order."""

import numpy as np
import pytest
import torch

import synth

from test_gpu_kv import filled, gpu_cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import affine_quantized_gemm_amd as Q
    return Q


@pytest.fixture(params=["default", "other"])
def given(request):
    """A stream, how a call is given it, and another one to be the current one meanwhile."""
    s = torch.cuda.default_stream() if request.param == "default" else torch.cuda.Stream()
    assert (s.cuda_stream == 0) == (request.param == "default")
    return s, s.cuda_stream, torch.cuda.Stream()


def late(stream, to, value):
    """`to` gets its value on the stream, behind some milliseconds of other work there."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(8):
            a = (a @ a).clamp_(max=1.0)
        to.copy_(value)


def test_log_probs(Q, given):
    """Rows cut into parts, whose counters have to be zero when the first call's workgroups come."""
    from affine_quantized_gemm_amd import rows
    stream, handle, current = given
    print(f"log_probs on stream {handle:#x}", flush=True)
    z = synth.normal((6, 50000), 2.0, "bf16", 1).cuda()
    want = Q.log_probs(z, top=5)
    torch.cuda.synchronize()
    rows._spaces.pop((torch.cuda.current_device(), handle), None)
    for _ in range(3):
        x = torch.zeros_like(z)
        torch.cuda.synchronize()
        late(stream, x, z)
        with torch.cuda.stream(current):
            got = Q.log_probs(x, top=5, stream=handle)
        torch.cuda.synchronize()
        assert all(a is b or torch.equal(a, b) for a, b in zip(got, want))
    assert not rows._spaces[(torch.cuda.current_device(), handle)][:rows.LOG_PROBS_ZEROED_BYTES].any()


def test_gated_gradient(Q, given):
    stream, handle, current = given
    print(f"gated_backward on stream {handle:#x}", flush=True)
    w = Q.quantize(synth.normal((2 * 512, 256), 0.06, "bf16", 2).cuda(), 4, 64)
    x, grad = synth.normal((6, 256), 1.0, "bf16", 3).cuda(), synth.normal((6, 512), 1.0, "bf16", 4).cuda()
    want = Q.gated_backward(x, *w, 4, 64, grad)
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    late(stream, y, x)
    with torch.cuda.stream(current):
        got = Q.gated_backward(y, *w, 4, 64, grad, stream=handle)
        # (what is freed behind the call and taken again here must not be the call's workspace)
        for _ in range(4):
            torch.full((6, 1024), 7.0, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_attention_over_a_window(Q, given):
    stream, handle, current = given
    print(f"attend on stream {handle:#x}", flush=True)
    lens = np.array([3000, 2000])
    c, tables = filled("bf16", 64, 64, 64, 2, lens, 48, 90, 5)
    q = synth.normal((8, 8, 64), 1.0, "bf16", 6).cuda()
    args = (i32(tables), i32(lens))
    want = gpu_cache(Q, c).attend(0, q, *args, window=1500, sinks=4, lse=True)
    cache, x = gpu_cache(Q, c), torch.zeros_like(q)  # (a cache without a workspace yet)
    torch.cuda.synchronize()
    for _ in range(2):
        x.zero_()
        torch.cuda.synchronize()
        late(stream, x, q)
        with torch.cuda.stream(current):
            got = cache.attend(0, x, *args, window=1500, sinks=4, lse=True, stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert set(cache._spaces) == {handle}


def test_gradient_of_no_columns(Q, given):
    """grad_x of a block without columns is zero, behind what the stream did to it before."""
    stream, handle, current = given
    wq, s = torch.empty(0, 8, dtype=torch.int32, device="cuda"), torch.empty(0, 1, dtype=torch.float16, device="cuda")
    x, none = torch.ones(3, 64, dtype=torch.float16, device="cuda"), torch.empty(3, 0, dtype=torch.float16, device="cuda")
    out, sevens = torch.zeros_like(x), torch.full_like(x, 7.0)
    torch.cuda.synchronize()
    late(stream, out, sevens)
    with torch.cuda.stream(current):
        Q.gated_backward(x, wq, s, s.clone(), 4, 64, none, out=out, stream=handle)
    torch.cuda.synchronize()
    assert not out.any()
    late(stream, out, sevens)
    with torch.cuda.stream(stream):  # the current one, not given
        Q.gated_backward(x, wq, s, s.clone(), 4, 64, none, out=out)
    torch.cuda.synchronize()
    assert not out.any()
