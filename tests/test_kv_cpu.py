"""The paged K/V cache without a GPU: arguments that the C entry points refuse
(before any HIP call), sizes, and the oracle pinned by hand-worked cases."""

import ctypes

import numpy as np
import pytest
import torch

import affine_quantized_gemm_amd as Q
from affine_quantized_gemm_amd import kv
from oracle import kv_oracle as KO
from oracle import qmm_oracle as O

L = Q._lib
A, MIS8, MIS2 = 0x10000, 0x10008, 0x10002  # addresses that are never dereferenced
OK, INV, UNS, MIS = Q.QMM_OK, Q.QMM_ERR_INVALID_ARG, Q.QMM_ERR_UNSUPPORTED, Q.QMM_ERR_MISALIGNED


def geo(dt=0, gs=64, dim=128, kv_heads=8, page=64, layers=2, pages=0, pool=A):
    return ctypes.byref(kv._Geometry(dt, gs, dim, kv_heads, page, layers, pages, pool))


def test_record_bytes():
    for dim in (64, 128, 256):
        for gs in (32, 64, 128):
            for page in (32, 64, 128, 256):
                n = L.qmm_kv_record_bytes(geo(gs=gs, dim=dim, page=page))
                if gs > dim:
                    assert n == UNS
                else:
                    assert n == page * (dim + 8 * (dim // gs)) == 4 * KO.record_words(dim, gs, page)
                    assert n == 4 * Q.record_words(dim, gs, page) and n % 128 == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNS), (dict(dt=-1), UNS), (dict(dim=96), UNS), (dict(dim=0), UNS), (dict(dim=512), UNS),
    (dict(gs=16), UNS), (dict(gs=48), UNS), (dict(gs=128, dim=64), UNS), (dict(page=16), UNS), (dict(page=48), UNS),
    (dict(page=0), UNS), (dict(page=512), UNS), (dict(kv_heads=0), UNS), (dict(kv_heads=70000), UNS),
    (dict(layers=0), UNS), (dict(pages=-1), INV), (dict(pages=1 << 31), UNS),
])
def test_geometry_refused_everywhere(kw, status):
    g = geo(**kw)
    assert L.qmm_kv_record_bytes(g) == status
    assert L.qmm_kv_append(g, 0, 1, 1, 1, A, 4, A, None, A, 128, 128, A, 128, 128, None) == status
    assert L.qmm_kv_read(g, 0, 1, 1, 1, A, 4, A, None, A, A, None) == status
    assert L.qmm_kv_attend_workspace_bytes(g, 1, 1, 1, 8, 100) == status
    assert L.qmm_kv_attend(g, 0, 1, 1, 1, A, 4, A, None, A, 128, 128, 8, 1.0, None, A, None, 100, A, 1 << 30,
                           None) == status
    assert L.qmm_kv_pages_workspace_bytes(g, 4) == status
    assert L.qmm_kv_copy_pages(g, A, A, 3, None) == status
    assert L.qmm_kv_reserve(g, 1, A, 4, A, A, A, A, A, 1 << 30, None) == status
    assert L.qmm_kv_fork(g, 1, A, 4, A, A, A, A, 1, A, A, 1 << 30, None) == status
    assert L.qmm_kv_free(g, 1, A, 4, A, A, A, 1, None) == status
    assert L.qmm_kv_compact(g, 1, A, 4, A, A, A, A, A, 1 << 30, None) == status
    assert L.qmm_kv_record_bytes(None) == INV


def attend(**kw):
    a = dict(g=geo(pages=9), layer=0, seqs=2, max_new=3, rows=6, tables=A, width=4, lens=A, starts=None, q=A, qr=4096,
             qh=128, heads=32, scale=0.1, mask=None, out=A, lse=None, max_len=256, ws=A, bytes=1 << 30)
    a.update(kw)
    return L.qmm_kv_attend(a["g"], a["layer"], a["seqs"], a["max_new"], a["rows"], a["tables"], a["width"], a["lens"],
                           a["starts"], a["q"], a["qr"], a["qh"], a["heads"], a["scale"], a["mask"], a["out"],
                           a["lse"], a["max_len"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(seqs=-1), INV), (dict(max_new=-1), INV), (dict(rows=-6), INV),
    (dict(rows=5), INV), (dict(rows=7, starts=A), INV), (dict(width=-1), INV), (dict(max_new=65, rows=130), UNS),
    (dict(heads=0), UNS), (dict(heads=12), UNS), (dict(heads=-8), UNS), (dict(max_len=0), INV),
    (dict(max_len=1 << 32), UNS), (dict(width=1 << 28), UNS), (dict(seqs=1 << 28, rows=3 << 28), UNS),
    (dict(tables=None), INV), (dict(lens=None), INV), (dict(q=None), INV), (dict(out=None), INV),
    (dict(tables=MIS2), MIS), (dict(lens=MIS2), MIS), (dict(starts=MIS2), MIS), (dict(q=MIS8), MIS),
    (dict(qr=4100), MIS), (dict(qh=132), MIS), (dict(qr=-4096), INV), (dict(out=MIS8), MIS), (dict(mask=A + 4), MIS),
    (dict(lse=MIS2), MIS), (dict(g=geo(pages=9, pool=None)), INV), (dict(g=geo(pages=9, pool=MIS8)), MIS),
    (dict(rows=0, seqs=0, q=None, out=None, tables=None, lens=None), OK),
    (dict(rows=0, max_new=0, q=None, out=None, lens=None), OK),
])
def test_attend_refusals(kw, status):
    assert attend(**kw) == status


def test_attend_workspace_refusals():
    g = geo(pages=9)
    long = 1 << 17
    need = L.qmm_kv_attend_workspace_bytes(g, 2, 3, 6, 32, long)
    assert need > 0 and need % 16 == 0
    assert attend(g=g, max_len=long, ws=None) == INV
    assert attend(g=g, max_len=long, bytes=need - 1) == INV
    assert attend(g=g, max_len=long, ws=MIS8) == MIS
    assert L.qmm_kv_attend_workspace_bytes(g, 0, 3, 0, 32, long) == 0
    assert L.qmm_kv_attend_workspace_bytes(g, 2, 3, 6, 32, 0) == INV
    assert L.qmm_kv_attend_workspace_bytes(g, 2, 3, 6, 33, 5) == UNS
    assert L.qmm_kv_attend_workspace_bytes(g, 2, 65, 130, 32, 5) == UNS


def test_attend_workspace_bound():
    """What the header promises no call exceeds, over head layouts, rows, sequences and lengths."""
    for dim in (64, 128, 256):
        for kv_heads in (1, 2, 5, 8, 16, 100):
            for group in (1, 3, 7, 16, 40):
                for rows in (1, 5, 17, 64):
                    for seqs in (1, 2, 7, 33, 200, 300):
                        for most in (1, 129, 5000, 1 << 30):
                            n = L.qmm_kv_attend_workspace_bytes(geo(dim=dim, kv_heads=kv_heads), seqs, rows, seqs * rows,
                                                                kv_heads * group, most)
                            assert 0 <= n <= kv.ATTEND_ZEROED_BYTES + 32768 * (dim + 4)


def test_append_and_read_refusals():
    g = geo(pages=9)
    ap = L.qmm_kv_append
    assert ap(g, 0, 1, 2, 2, A, 4, A, None, None, 128, 128, A, 128, 128, None) == INV
    assert ap(g, 0, 1, 2, 2, A, 4, A, None, A, 128, 128, MIS8, 128, 128, None) == MIS
    assert ap(g, 0, 1, 2, 2, A, 4, A, None, A, 128, 4, A, 128, 128, None) == MIS
    assert ap(g, 0, 1, 2, 2, A, 4, A, None, A, 128, 128, A, -128, 128, None) == INV
    assert ap(g, 0, 1, 2, 0, A, 4, A, A, None, 128, 128, None, 128, 128, None) == OK
    rd = L.qmm_kv_read
    assert rd(g, 0, 1, 2, 2, A, 4, A, None, A, None, None) == INV
    assert rd(g, 0, 1, 2, 2, A, 4, A, None, MIS8, A, None) == MIS
    assert rd(g, 3, 1, 2, 2, A, 4, A, None, A, A, None) == INV


def test_page_call_refusals():
    g = geo(pages=9)
    need = L.qmm_kv_pages_workspace_bytes(g, 5)
    assert need >= 5 * 12 and L.qmm_kv_pages_workspace_bytes(g, 0) > 0 and L.qmm_kv_pages_workspace_bytes(g, -1) == INV
    assert L.qmm_kv_copy_pages(g, A, A, -1, None) == INV
    assert L.qmm_kv_copy_pages(g, None, A, 1, None) == INV
    assert L.qmm_kv_copy_pages(g, MIS2, A, 1, None) == MIS
    assert L.qmm_kv_copy_pages(g, None, None, 0, None) == OK
    rs = L.qmm_kv_reserve
    assert rs(g, 5, A, 4, A, A, A, A, None, 0, None) == INV
    assert rs(g, 5, A, 4, A, A, A, A, A, need - 16, None) == INV
    assert rs(g, 5, A, 4, None, A, A, A, A, need, None) == INV
    assert rs(g, 5, A, 4, A, A, A, MIS2, A, need, None) == MIS
    assert rs(g, 0, None, 4, None, A, None, None, None, 0, None) == OK
    fk = L.qmm_kv_fork
    assert fk(g, 5, A, 4, A, A, A, None, 2, A, A, need, None) == INV
    assert fk(g, 5, A, 4, A, A, A, A, -2, A, A, need, None) == INV
    assert fk(g, 5, A, 4, A, A, A, A, 5, A, A, 16, None) == INV
    assert fk(g, 5, A, 4, A, A, None, None, 0, None, None, 0, None) == OK
    fr = L.qmm_kv_free
    assert fr(g, 5, A, 4, A, A, None, 2, None) == INV
    assert fr(g, 5, A, 4, A, A, A, -2, None) == INV
    assert fr(g, 5, A, 4, A, None, A, 2, None) == INV
    cm = L.qmm_kv_compact
    big = L.qmm_kv_pages_workspace_bytes(g, 0)
    assert cm(g, 5, A, 4, A, A, A, None, A, big, None) == INV
    assert cm(g, 5, A, 4, A, None, A, A, A, big, None) == INV
    assert cm(g, 5, A, 4, A, A, A, A, A, big - 16, None) == INV
    assert cm(g, 5, A, -4, A, A, A, A, A, big, None) == INV


def test_python_refuses_before_the_library():
    with pytest.raises(Q.QmmError):
        Q.record_words(96, 32, 64)
    with pytest.raises(Q.QmmError):
        Q.record_words(128, 64, 64, torch.float32)
    w = Q.record_words(128, 64, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        Q.KVCache(torch.zeros(1, 2, 3, w, dtype=torch.int32), 128, 64, 64)
    with pytest.raises(ValueError, match="shape"):
        Q.KVCache(torch.zeros(1, 2, 3, w + 1, dtype=torch.int32), 128, 64, 64)
    with pytest.raises(ValueError, match="dtype"):
        Q.KVCache(torch.zeros(1, 2, 3, w, dtype=torch.int64), 128, 64, 64)
    with pytest.raises(ValueError, match="4-D"):
        Q.KVCache(torch.zeros(2, 3, w, dtype=torch.int32), 128, 64, 64)


# ---- the oracle ----

@pytest.mark.parametrize("dim,gs,page", [(64, 32, 32), (128, 64, 64), (256, 128, 32)])
def test_oracle_layout_is_a_bijection(dim, gs, page):
    c = KO.new_cache(1, 1, 1, dim, gs, page, "f16")
    seen = set()
    for part in (0, 1):
        for slot in range(page):
            word, shift = KO._code_at(c, part, slot)
            seen |= {(int(w), int(s)) for w, s in zip(word, shift)}
            half = KO._half_at(c, part, slot)
            for h in list(half) + list(half + 4):
                seen |= {(int(h) // 2, 16 * (int(h) % 2) + 4 * x) for x in range(4)}
    assert len(seen) == KO.record_words(dim, gs, page) * 8  # every 4 bits of the record once
    assert max(w for w, _ in seen) == KO.record_words(dim, gs, page) - 1


def test_oracle_layout_by_hand():
    # D = 128, page 64: K value 77 of token 5 is word (5, j = 1, s = 2), bits 20..23;
    # V value 77 of token 6 is word (u = 1, i = 13, p = 1, c = 1), low half, n = 0
    c = KO.new_cache(1, 1, 1, 128, 64, 64, "f16")
    w, s = KO._code_at(c, 0, 5)
    assert (w[77], s[77]) == (5 * 16 + 1 * 4 + 2, 20)
    w, s = KO._code_at(c, 1, 6)
    assert (w[77], s[77]) == (64 * 16 + ((16 + 13) * 2 + 1) * 2 + 1, 0)
    assert list(KO._half_at(c, 1, 6)) == [2 * (2048 + 128) + 16 + 2, 2 * (2048 + 128) + 16 + 8 + 2]


def test_oracle_stores_what_the_quantizer_says():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 128)).astype(np.float16)
    c = KO.new_cache(1, 2, 1, 128, 32, 32, "f16", fill=0xFFFFFFFF)
    for t in range(3):
        KO.store(c, 0, 1, 0, t, 0, x[t])
        KO.store(c, 0, 1, 0, t, 1, x[t])
    wq, s, b = O.quantize(x, "f16", 4, 32)
    want = O.dequantize_exact(wq, s, b, "f16", 4, 32, 128)
    for part in (0, 1):
        for t in range(3):
            q, sc, z = KO.load(c, 0, 1, 0, t, part)
            assert np.array_equal(q * sc + z, want[t])
    assert (c["pool"][0, 0] == 0xFFFFFFFF).all()


def test_oracle_attention_by_hand():
    # one token: its own value; none visible: zeros and -inf; equal scores: the mean
    c = KO.new_cache(1, 1, 1, 64, 64, 32, "f16")
    x = np.linspace(-1, 1, 64).astype(np.float16)
    for t in range(2):
        KO.store(c, 0, 0, 0, t, 0, np.zeros(64, np.float16))
        KO.store(c, 0, 0, 0, t, 1, x * (t + 1))
    tables = np.array([[0]], dtype=np.int32)
    v = [KO.load(c, 0, 0, 0, t, 1) for t in range(2)]
    v = [q * s + z for q, s, z in v]
    out, lse, _, _ = KO.attend(c, 0, np.ones((2, 1, 64)), tables, [2], [0, 2], 0.5)
    assert np.allclose(out[0, 0], v[0]) and np.allclose(out[1, 0], (v[0] + v[1]) / 2)
    assert lse[0, 0] == 0 and np.isclose(lse[1, 0], np.log(2))
    out, lse, _, _ = KO.attend(c, 0, np.ones((2, 1, 64)), tables, [2], [0, 2], 0.5, mask=np.array([0, 1]))
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and np.allclose(out[1, 0], v[0])


def test_oracle_pages_by_hand():
    tables, lens = np.full((3, 4), -1, np.int32), np.zeros(3, np.int32)
    refs = np.zeros(6, np.int32)
    refs[1] = 1  # someone else's
    assert list(KO.reserve(tables, lens, refs, [40, 0, 32], 32)) == [1, 1, 1]
    assert tables.tolist() == [[0, 2, -1, -1], [-1] * 4, [3, -1, -1, -1]] and lens.tolist() == [40, 0, 32]
    pool = np.arange(6)[None]
    assert list(KO.fork(pool, tables, lens, refs, [0], [1], 32)) == [1]
    assert tables[1].tolist() == [0, 4, -1, -1] and refs.tolist() == [2, 1, 1, 1, 1, 0] and pool[0, 4] == 2
    KO.free(tables, lens, refs, [0])
    assert refs.tolist() == [1, 1, 0, 1, 1, 0] and lens.tolist() == [0, 40, 32]
    out, counts, live = KO.compact(pool, tables, refs)
    assert live == 4 and counts.tolist() == [1, 1, 1, 1, 0, 0]
    assert out.tolist() == [[-1] * 4, [0, 2, -1, -1], [3, -1, -1, -1]]
