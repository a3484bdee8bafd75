"""The gated block, rotary positions, log probabilities and attention with a window without a GPU: the oracle pinned by
differences and closed forms, and the arguments that the C entry points and the binding refuse before any HIP call."""

import ctypes
import math

import numpy as np
import pytest
import torch

import affine_quantized_gemm_amd as Q
import synth
from affine_quantized_gemm_amd import kv, rows
from oracle import kv_oracle as KO
from oracle import qmm_oracle as O
from oracle import rows_oracle as RO

L = Q._lib
A, MIS8, MIS2, MIS1 = 0x10000, 0x10008, 0x10002, 0x10001  # addresses that are never dereferenced
OK, INV, UNS, MIS = Q.QMM_OK, Q.QMM_ERR_INVALID_ARG, Q.QMM_ERR_UNSUPPORTED, Q.QMM_ERR_MISALIGNED
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


# ---- the oracle ----

@pytest.mark.parametrize("name", ACTS)
def test_activation_slopes_are_differences(name):
    a = np.array([-30.0, -8.0, -3.0, -1.0, -0.3, 0.2, 0.7, 2.0, 5.0, 20.0])
    h = 1e-5
    v, slope, bend = RO.act(name, a)
    up, down = RO.act(name, a + h), RO.act(name, a - h)
    assert np.allclose((up[0] - down[0]) / (2 * h), slope, atol=1e-8)
    assert (np.abs(up[1] - down[1]) / (2 * h) <= bend + 1e-8).all() and (np.abs(slope) <= 1.2).all()
    x = torch.tensor(a)
    want = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
            "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[name](x)
    assert np.allclose(v, want.numpy(), rtol=1e-12, atol=1e-14)


def weights(dt, bits, gs, n, k, seed):
    w = synth.normal((n, k), k ** -0.5, dt, seed)
    return O.quantize(synth.to_oracle(w), dt, bits, gs)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradient_is_differences(name):
    wq, sc, bi = weights("f16", 4, 32, 2 * 6, 64, 1)
    x = O.to_f64(synth.to_oracle(synth.normal((3, 64), 1.0, "f16", 2)), "f16")
    grad = np.random.default_rng(3).normal(size=(3, 6))
    dx = RO.gated_backward(x, wq, sc, bi, "f16", 4, 32, name, grad)[0]
    h = 1e-5
    for k in (0, 17, 63):
        for r in (0, 2):
            up, down = x.copy(), x.copy()
            up[r, k] += h
            down[r, k] -= h
            f = lambda v: (grad * RO.gated(v, wq, sc, bi, "f16", 4, 32, name)[0]).sum()
            assert abs((f(up) - f(down)) / (2 * h) - dx[r, k]) < 1e-7


def test_rotary_oracle():
    x = np.zeros((2, 1, 32))
    x[:, 0, 0] = 1.0
    freq = np.full(16, math.pi / 2, dtype=np.float64).astype(np.float32)
    y = RO.rotary(x, np.array([[1, 2]]), freq, [16], "halves", False, 1.0, "f16")[0]
    assert np.allclose(y[0, 0, [0, 16]], [0, 1], atol=1e-6) and np.allclose(y[1, 0, [0, 16]], [-1, 0], atol=1e-6)
    y = RO.rotary(x, np.array([[1, 2]]), freq, [16], "adjacent", True, 2.0, "f16")[0]
    assert np.allclose(y[0, 0, [0, 1]], [0, -2], atol=1e-6)
    # turning back is the transposed map: (R x) . y = x . (R' y)
    g = np.random.default_rng(0)
    x, y, pos = g.normal(size=(5, 3, 48)), g.normal(size=(5, 3, 48)), g.integers(0, 1000, (3, 5))
    freq = g.random(16).astype(np.float32)
    for pairs in ("halves", "adjacent"):
        a = (RO.rotary(x, pos, freq, [4, 0, 12], pairs, False, 0.7, "f16")[0] * y).sum()
        assert np.isclose(a, (x * RO.rotary(y, pos, freq, [4, 0, 12], pairs, True, 0.7, "f16")[0]).sum())


def test_log_probs_oracle():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    r = RO.log_probs(z, np.array([[2, -100, 3]]), 3, 1.0)
    assert np.isclose(r["lse"][0], math.log(8)) and list(r["top_ids"][0]) == [2, 1, 0]
    assert np.allclose(r["tokens"], [[math.log(0.5), 0, math.log(0.125)]])
    assert np.isclose(r["entropy"][0], 0.5 * math.log(2) + 0.25 * math.log(4) + 0.25 * math.log(8))
    r = RO.log_probs(np.array([[-np.inf, 0.0, -np.inf], [-np.inf] * 3]), np.array([1, 0]), 2, 1.0)
    assert list(r["lse"]) == [0, -np.inf] and list(r["entropy"]) == [0, 0] and list(r["tokens"]) == [0, -np.inf]
    assert r["top_ids"].tolist() == [[1, 0], [0, 1]]


def test_log_probs_oracle_of_large_logits():
    """Equal largest logits of any size: the same log probabilities."""
    for size in (1.0, 1e20, 1e38):
        r = RO.log_probs(size * np.array([[1.0, 1.0, 1.0, -1.0]]) - 60 * np.array([0, 0, 0, 1.0]), np.array([0]), 1, 1.0)
        assert np.isclose(r["tokens"][0], -math.log(3)) and np.isclose(r["entropy"][0], math.log(3))


def test_log_probs_gradient_is_differences():
    g = np.random.default_rng(1)
    z, tokens = g.normal(size=(4, 9)) * 2, np.array([[1, 1], [8, -100], [0, 3], [9, -1]])
    z[2, 5] = -np.inf
    gt, gh, gl = g.normal(size=(4, 2)), g.normal(size=4), g.normal(size=4)

    def loss(v):
        r = RO.log_probs(v, tokens, 0, 1.3)
        return (gt * r["tokens"]).sum() + (gh * r["entropy"]).sum() + (gl * r["lse"]).sum()

    r = RO.log_probs(z, tokens, 0, 1.3)
    d = RO.log_probs_backward(z, tokens, r["lse"], r["entropy"], gt, gh, gl, 1.3, "f16")[0]
    h = 1e-6
    for i in range(4):
        for v in range(9):
            if np.isfinite(z[i, v]):
                up, down = z.copy(), z.copy()
                up[i, v] += h
                down[i, v] -= h
                assert abs((loss(up) - loss(down)) / (2 * h) - d[i, v]) < 1e-7
    assert d[2, 5] == 0


def test_window_oracle():
    every = list(range(12))
    at = lambda **kw: np.flatnonzero(KO.sees(positions=every, **kw)).tolist()
    assert at(word=1, length=10, n=1, window=3) == [7, 8, 9]
    assert at(word=1, length=10, n=1, window=3, sinks=2) == [0, 1, 7, 8, 9]
    assert at(word=1, length=10, n=1, window=100, sinks=2) == list(range(10))
    assert at(word=0b101, length=10, n=3, window=2, sinks=1) == [0, 7, 9]       # a tree: 8 is another branch
    assert at(word=0b101, length=10, n=3, window=4) == [5, 6, 7, 9]
    assert at(word=0, length=10, n=3, window=2) == [5, 6]
    assert at(word=0b111, length=10, n=3, window=2, sinks=8) == [*range(8), 8, 9]
    assert at(word=0b111, length=10, n=3) == list(range(10))


def test_bounds_are_of_the_size_of_the_roundings():
    """A bound says something: a twentieth of the values (a group of 64 of 1024 codes is a sixteenth), most of it for sums of
    codes with an offset of 1024 that all round the same way."""
    for dt, bits in (("f16", 4), ("bf16", 4), ("bf16", 8), ("f16", 8)):
        wq, sc, bi = weights(dt, bits, 64, 2 * 16, 1024, 5)
        x = O.to_f64(synth.to_oracle(synth.normal((4, 1024), 1.0, dt, 6)), dt)
        h, tol = RO.gated(x, wq, sc, bi, dt, bits, 64, "silu")
        assert np.median(tol) <= 100 * RO.UNIT[dt] * np.sqrt((h ** 2).mean())
    z = np.random.default_rng(2).normal(size=(2, 5000)) * 2
    r = RO.log_probs(z, np.array([1, 2]), 4, 1.0)
    for k in ("lse", "entropy", "tokens", "top_values"):
        assert (r["tol_" + k] <= 1e-4).all()


# ---- refusals ----

def gated(**kw):
    a = dict(dt=0, bits=4, gs=64, act=0, M=4, F=32, K=128, x=A, wq=A, s=A, b=A, h=A)
    a.update(kw)
    return L.qmm_gated(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNS), (dict(bits=5), UNS), (dict(gs=16), UNS), (dict(act=4), UNS), (dict(act=-1), UNS), (dict(M=65), UNS),
    (dict(M=-1), INV), (dict(F=-1), INV), (dict(K=-64), INV), (dict(K=96), UNS), (dict(K=32), UNS), (dict(K=64, gs=128), UNS),
    (dict(F=1 << 31), UNS), (dict(K=1 << 30), UNS), (dict(x=None), INV), (dict(wq=None), INV), (dict(s=None), INV), (dict(b=None), INV),
    (dict(h=None), INV), (dict(x=MIS8), MIS), (dict(wq=MIS8), MIS), (dict(s=MIS2), MIS), (dict(b=MIS2), MIS),
    (dict(h=MIS8), MIS), (dict(M=0, x=None, h=None), OK), (dict(F=0, wq=None, h=None), OK),
])
def test_gated_refusals(kw, status):
    assert gated(**kw) == status


def backward(**kw):
    a = dict(dt=0, bits=4, gs=64, act=0, M=4, F=32, K=128, x=A, wq=A, s=A, b=A, grad=A, dgu=A, dx=A, ws=A, bytes=1 << 30)
    a.update(kw)
    return L.qmm_gated_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNS), (dict(F=33), UNS), (dict(F=8), UNS), (dict(act=9), UNS), (dict(M=65), UNS), (dict(M=-1), INV),
    (dict(grad=None), INV), (dict(dgu=None), INV), (dict(dx=None), INV), (dict(grad=MIS8), MIS), (dict(dgu=MIS8), MIS),
    (dict(dx=MIS2), MIS), (dict(bytes=-1), INV), (dict(M=0, x=None, grad=None, ws=None, bytes=0), OK),
])
def test_gated_backward_refusals(kw, status):
    assert backward(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict(dx=None), INV), (dict(dx=MIS8), MIS), (dict(M=0, dx=None), OK)])
def test_gated_backward_without_columns_refusals(kw, status):
    """grad_x is written there too."""
    none = dict(F=0, x=None, wq=None, s=None, b=None, grad=None, dgu=None, ws=None, bytes=0)
    assert backward(**{**none, **kw}) == status


def test_gated_backward_workspace():
    size = L.qmm_gated_backward_workspace_bytes
    need = size(0, 4, 64, 6, 2048, 4096)
    assert need > 0 and need % 16 == 0
    big = dict(M=6, F=2048, K=4096)
    assert backward(**big, ws=None) == INV and backward(**big, bytes=need - 1) == INV and backward(**big, ws=MIS8) == MIS
    assert size(0, 4, 64, 0, 2048, 4096) == 0 and size(0, 4, 64, 6, 2040, 4096) == UNS and size(0, 4, 64, -1, 2048, 4096) == INV


def rotary(**kw):
    a = dict(dt=1, rows=5, heads=3, dim=64, turned=32, pairs=0, inverse=0, scale=1.0, x=A, xr=192, xh=64, pos=A, wide=0, ps=5,
             axes=2, sections=(ctypes.c_int32 * 2)(10, 6), freq=A, out=A, outr=192, outh=64)
    a.update(kw)
    return L.qmm_rotary(*a.values(), None)


def sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), UNS), (dict(rows=-1), INV), (dict(heads=-1), INV), (dict(dim=60), UNS), (dict(dim=2048), UNS), (dict(dim=8), UNS),
    (dict(turned=24), UNS), (dict(turned=0), UNS), (dict(turned=80), UNS), (dict(pairs=2), UNS), (dict(axes=0), UNS),
    (dict(axes=5), UNS), (dict(sections=None), INV), (dict(sections=sections(10, 7)), INV), (dict(sections=sections(20, -4)), INV),
    (dict(xr=-8), INV), (dict(xr=196), MIS), (dict(xh=60), MIS), (dict(outr=188), MIS), (dict(outh=4), MIS), (dict(ps=-5), INV),
    (dict(x=None), INV), (dict(out=None), INV), (dict(freq=None), INV), (dict(pos=None), INV), (dict(x=MIS8), MIS),
    (dict(out=MIS8), MIS), (dict(freq=MIS2), MIS), (dict(pos=MIS2), MIS), (dict(pos=A + 4, wide=1), MIS),
    (dict(outh=0), INV), (dict(outr=64), INV), (dict(outr=0), INV), (dict(outr=128, outh=64), INV),
    (dict(rows=0, x=None, out=None, pos=None), OK), (dict(heads=0, x=None, out=None), OK),
])
def test_rotary_refusals(kw, status):
    assert rotary(**kw) == status


def log_probs(**kw):
    a = dict(dt=0, rows=1000, vocab=500, scale=1.0, logits=A, stride=500, tokens=A, wide=1, given=1, top=4, lse=A, h=A, lp=A,
             values=A, ids=A, ws=A, bytes=1 << 30)
    a.update(kw)
    return L.qmm_log_probs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNS), (dict(rows=-1), INV), (dict(vocab=-1), INV), (dict(stride=-1), INV), (dict(given=-1), INV),
    (dict(top=-1), INV), (dict(given=65), UNS), (dict(top=65), UNS), (dict(vocab=3), UNS), (dict(vocab=1 << 31), UNS),
    (dict(vocab=0, top=0), UNS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.inf), INV),
    (dict(scale=math.nan), INV), (dict(logits=None), INV), (dict(logits=MIS1), MIS), (dict(tokens=None), INV),
    (dict(tokens=A + 4), MIS), (dict(lp=None), INV), (dict(lse=None), INV), (dict(h=None), INV), (dict(lse=MIS2), MIS),
    (dict(values=None), INV), (dict(ids=None), INV), (dict(ids=A + 4), MIS), (dict(bytes=-1), INV),
    (dict(rows=6, vocab=100000, ws=None), INV), (dict(rows=6, vocab=100000, bytes=rows.LOG_PROBS_WORKSPACE_BYTES - 1), INV),
    (dict(rows=6, vocab=100000, ws=MIS8), MIS), (dict(rows=0, logits=None, lse=None), OK),
])
def test_log_probs_refusals(kw, status):
    assert log_probs(**kw) == status


@pytest.mark.parametrize("scale", [2.0 ** -101, 2.0 ** 101, 3e38, 1e-44])
def test_log_probs_scales_out_of_range(scale):
    assert log_probs(scale=scale) == UNS and log_probs_backward(scale=scale) == UNS
    assert log_probs(scale=scale, rows=0) == UNS
    assert log_probs(scale=2.0 ** 100, rows=0) == OK and log_probs_backward(scale=2.0 ** -100, rows=0) == OK


def test_log_probs_workspace_is_for_few_rows():
    need = L.qmm_log_probs_needs_workspace
    assert need(6, 100000) == 1 and need(6, 100) == 0 and need(100000, 100000) == 0 and need(0, 100) == 0
    assert need(-1, 5) == INV and need(5, -1) == INV and need(5, 1 << 31) == UNS


def log_probs_backward(**kw):
    a = dict(dt=0, rows=6, vocab=500, scale=1.0, logits=A, stride=500, tokens=A, wide=1, given=1, lse=A, h=A, gt=A, gh=A, gl=A,
             out=A, outs=500)
    a.update(kw)
    return L.qmm_log_probs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNS), (dict(rows=-1), INV), (dict(vocab=-1), INV), (dict(given=65), UNS), (dict(scale=0.0), INV),
    (dict(outs=499), INV), (dict(outs=-1), INV), (dict(logits=None), INV), (dict(out=None), INV), (dict(out=MIS1), MIS),
    (dict(lse=None), INV), (dict(lse=MIS2), MIS), (dict(h=None), INV), (dict(gh=MIS2), MIS), (dict(gl=MIS2), MIS),
    (dict(tokens=None), INV), (dict(gt=MIS2), MIS), (dict(tokens=A + 4), MIS), (dict(rows=0, logits=None, out=None), OK),
    (dict(vocab=0, logits=None, out=None, stride=0, outs=0), OK),
])
def test_log_probs_backward_refusals(kw, status):
    assert log_probs_backward(**kw) == status


def window(**kw):
    g = ctypes.byref(kv._Geometry(0, 64, 128, 8, 64, 2, 9, A))
    a = dict(g=g, layer=0, seqs=2, max_new=3, rows=6, tables=A, width=4, lens=A, starts=None, q=A, qr=4096, qh=128, heads=32,
             scale=0.1, mask=None, window=100, sinks=4, out=A, lse=None, max_len=256, ws=A, bytes=1 << 30)
    a.update(kw)
    return L.qmm_kv_attend_window(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), INV), (dict(window=-5), INV), (dict(sinks=-1), INV), (dict(layer=2), INV), (dict(rows=5), INV),
    (dict(max_new=65, rows=130), UNS), (dict(heads=12), UNS), (dict(q=None), INV), (dict(out=MIS8), MIS), (dict(mask=A + 4), MIS),
    (dict(max_len=0), INV), (dict(rows=0, seqs=0, q=None, out=None, tables=None, lens=None), OK),
])
def test_window_refusals(kw, status):
    assert window(**kw) == status


def test_window_workspace():
    """The tokens that a window leaves, not the sequences' lengths, say how many parts there are; within the bound."""
    size = L.qmm_kv_attend_window_workspace_bytes
    for dim in (64, 128, 256):
        for kv_heads, group, n, seqs in ((1, 1, 1, 1), (8, 4, 1, 1), (8, 4, 64, 3), (5, 7, 17, 33), (100, 1, 5, 2)):
            g = ctypes.byref(kv._Geometry(0, 64, dim, kv_heads, 64, 2, 9, A))
            for span in (1, 100, 5000, 1 << 40):
                for sinks in (0, 4, 1 << 40):
                    need = size(g, seqs, n, seqs * n, kv_heads * group, 1 << 20, span, sinks)
                    assert 0 <= need <= kv.ATTEND_ZEROED_BYTES + 32768 * (dim + 4)
    g = ctypes.byref(kv._Geometry(0, 64, 128, 8, 64, 2, 9, A))
    assert size(g, 1, 1, 1, 32, 1 << 17, 1000, 4) < L.qmm_kv_attend_workspace_bytes(g, 1, 1, 1, 32, 1 << 17)
    assert size(g, 1, 1, 1, 32, 1 << 17, 0, 4) == INV and size(g, 1, 1, 1, 32, 1 << 17, 5, -1) == INV
    need = size(g, 2, 3, 6, 32, 1 << 17, 5000, 4)
    assert window(max_len=1 << 17, window=5000, bytes=need - 1) == INV and window(max_len=1 << 17, window=5000, ws=None) == INV


# ---- the binding ----

def test_python_refuses_before_the_library():
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16)
    words = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    ok = (half(4, 128), words(64, 16), half(64, 2), half(64, 2), 4, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        Q.gated(*ok)
    with pytest.raises(ValueError, match="2F"):
        Q.gated(half(4, 128), words(63, 16), half(63, 2), half(63, 2), 4, 64)
    with pytest.raises(ValueError, match="wq has shape"):
        Q.gated(half(4, 128), words(64, 15), half(64, 2), half(64, 2), 4, 64)
    with pytest.raises(ValueError, match="scales has"):
        Q.gated(half(4, 128), words(64, 16), half(64, 4), half(64, 2), 4, 64)
    with pytest.raises(Q.QmmError):
        Q.gated(half(4, 128).float(), *ok[1:])
    x, pos, freq = half(5, 3, 64), torch.zeros(5, dtype=torch.int64), torch.ones(16)
    with pytest.raises(ValueError, match="GPU tensor"):
        Q.rotary(x, pos, freq)
    with pytest.raises(ValueError, match="positions has shape"):
        Q.rotary(x, pos[:4], freq)
    with pytest.raises(ValueError, match="positions has dtype"):
        Q.rotary(x, pos.float(), freq)
    with pytest.raises(ValueError, match="freq has dtype"):
        Q.rotary(x, pos, freq.double())
    with pytest.raises(ValueError, match="3-D"):
        Q.rotary(x[0], pos, freq)
    with pytest.raises(ValueError, match="contiguous"):
        Q.rotary(half(5, 64, 3).transpose(1, 2), pos, freq)
    z = half(4, 100)
    with pytest.raises(ValueError, match="GPU tensor"):
        Q.log_probs(z, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="2-D"):
        Q.log_probs(z[0])
    with pytest.raises(Q.QmmError):
        Q.log_probs(z.float())


def test_constants_match_the_header():
    text = open(Q.LIB_PATH.replace("affine_quantized_gemm_amd/libqmm.so", "include/qmm.h")).read()
    assert f"#define QMM_LOG_PROBS_ZEROED_BYTES {rows.LOG_PROBS_ZEROED_BYTES}" in text
    assert "#define QMM_LOG_PROBS_WORKSPACE_BYTES (65536 + 1024 * 66 * 8)" in text
    assert rows.LOG_PROBS_WORKSPACE_BYTES == 65536 + 1024 * 66 * 8
    for names, prefix in ((rows.ACTS, "QMM_ACT_"), (rows.PAIRS, "QMM_PAIRS_")):
        for name, value in names.items():
            assert f"{prefix}{name.upper()} = {value}" in text
