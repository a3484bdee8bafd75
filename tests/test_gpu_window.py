"""Attention with a window and sinks over the 4-bit cache, against the oracle's bound; what no row sees is not read."""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import kv_oracle as KO
from oracle import qmm_oracle as O

from test_gpu_kv import FORMATS, POISON, filled, gpu_cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import affine_quantized_gemm_amd as Q
    return Q


def check(Q, c, tables, lens, new, heads, seed, window, sinks=0, mask=None, bounds=()):
    dim, dt = c["dim"], c["dt"]
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1])
    q = synth.normal((rows, heads, dim), 1.0, dt, seed)
    scale = 1 / math.sqrt(dim)
    out, lse, tol, ltol = KO.attend_bound(c, 0, O.to_f64(synth.to_oracle(q), dt), tables, lens, starts, scale, mask, window, sinks)
    cache = gpu_cache(Q, c)
    kw = {"starts": i32(starts), "max_new": int(max(new))} if len(set(new)) != 1 else {}
    m = None if mask is None else torch.tensor(mask, dtype=torch.int64, device="cuda")
    args = (0, q.cuda(), i32(tables), i32(lens))
    got, glse = cache.attend(*args, mask=m, lse=True, window=window, sinks=sinks, **kw)
    again = cache.attend(*args, mask=m, window=window, sinks=sinks, **kw)
    empty = np.isneginf(lse)
    more = [cache.attend(*args, mask=m, lse=True, window=window, sinks=sinks, max_len=n, **kw) for n in bounds]
    for y, s in [(got, glse), *more]:
        g, gl = O.to_f64(synth.to_oracle(y), dt), s.cpu().numpy().astype(np.float64)
        assert np.isfinite(g).all()
        err = np.abs(g - out)
        print(f"  window {window}+{sinks}: worst err/bound {np.max(err[~empty] / tol[~empty], initial=0):.3f}", flush=True)
        assert (err <= tol).all()
        assert np.array_equal(np.isneginf(gl), empty) and (g[empty] == 0).all()
        assert (np.abs(gl[~empty] - lse[~empty]) <= ltol[~empty]).all()
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    return got


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_window_formats(Q, dt, dim, gs):
    """Ragged rows and lengths; windows of one token, inside a step, over steps and beyond the sequence."""
    print(f"window {dt} D={dim} gs={gs}", flush=True)
    lens = np.array([1, 5, 33, 64, 97, 130, 300, 517])
    new = np.array([1, 4, 6, 5, 3, 1, 2, 7])
    c, tables = filled(dt, dim, gs, 32, 1, lens, 17, 45, 60)
    for window, sinks in ((1, 0), (3, 4), (40, 0), (100, 1), (128, 33), (1000, 4)):
        check(Q, c, tables, lens, new, 3, 61, window, sinks)


@pytest.mark.parametrize("window", [1, 31, 32, 33, 64, 95, 200, 511])
@pytest.mark.parametrize("sinks", [0, 1, 32, 70, 600])
def test_window_ends(Q, window, sinks):
    """Sinks and windows that end in, at and beside steps and pages, meet, overlap or reach past the sequence."""
    lens = np.array([20, 100, 257, 512, 600])
    c, tables = filled("f16" if window % 2 else "bf16", 64, 64, 64, 1, lens, 10, 30, 62)
    check(Q, c, tables, lens, np.full(5, 1), 2, 63, window, sinks)
    check(Q, c, tables, lens, np.full(5, 20), 2, 64, window, sinks)


@pytest.mark.parametrize("rows,heads,kv_heads", [(1, 8, 2), (5, 10, 1), (17, 4, 4), (33, 9, 1), (64, 3, 1)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_window_long(Q, rows, heads, kv_heads, dt):
    """Long sequences beside short ones, cut into parts by what the window leaves, by tokens and by rows."""
    print(f"window long {dt} rows={rows} heads={heads}/{kv_heads}", flush=True)
    lens = np.array([2100, rows, 700, 1400 + rows])
    c, tables = filled(dt, 128, 64, 64, kv_heads, lens, 34, 80, 65)
    for window, sinks in ((900, 5), (64, 0)):
        check(Q, c, tables, lens, np.full(4, rows), heads, 66, window, sinks, bounds=(2100, 100))


def test_window_many_sequences(Q):
    """By rows (a workgroup a sequence), and more sequences than are cut."""
    lens = np.array([40 + 7 * (b % 20) for b in range(70)])
    c, tables = filled("f16", 64, 32, 32, 1, lens, 6, 420, 67)
    check(Q, c, tables, lens, np.full(70, 40), 1, 68, 50, 3)
    lens = np.array([9 + b % 90 for b in range(300)])
    c, tables = filled("bf16", 64, 64, 32, 1, lens, 4, 900, 69)
    check(Q, c, tables, lens, np.full(300, 2), 2, 70, 30, 2)


def test_window_trees(Q):
    """Draft trees: a row keeps its own token, its ancestors and what of the cache fills the window; rows that see nothing new,
    words that name tokens which are not there."""
    lens, new = np.array([60, 300, 13, 75]), np.array([13, 40, 13, 64])
    g = np.random.default_rng(71)
    words = []
    for n in new:
        m = []
        for i in range(n):
            m.append((1 << i) | (m[g.integers(max(0, i - 4), i)] if i else 0))
        words += m
    words[3], words[20], words[60] = 0, 1 << 5, words[60] | 1 << 63 | 1 << 50
    words[-1] = (1 << 64) - 1
    mask = [w - (1 << 64) if w >> 63 else w for w in words]
    c, tables = filled("bf16", 128, 64, 64, 2, lens, 5, 20, 72)
    for window, sinks in ((1, 0), (4, 2), (20, 0), (70, 40), (500, 1)):
        check(Q, c, tables, lens, new, 4, 73, window, sinks, mask=mask)


def test_window_without_new_tokens_or_places(Q):
    """Sequences of no rows, shorter than their new tokens, longer than the table; entries that name no page."""
    lens, new = np.array([0, 50, 3, 200, 90]), np.array([0, 0, 6, 5, 4])
    c, tables = filled("f16", 64, 64, 32, 1, np.array([0, 50, 3, 128, 90]), 4, 14, 74)
    tables[4, 1] = -1
    check(Q, c, tables, lens, new, 2, 75, 40, 3)
    check(Q, c, tables, lens, new, 2, 75, 100, 0)
    tables[3, :] = [99, -5, 2, 1000]
    check(Q, c, tables, lens, new, 2, 75, 100, 40)


def test_pages_outside_the_window_are_not_read(Q):
    """Pages that no row sees may be given up: what they hold, NaN or another sequence's, has no part."""
    dim, gs, page = 128, 64, 64
    lens, new = np.array([1000, 700]), np.array([5, 5])
    c, tables = filled("bf16", dim, gs, page, 2, lens, 16, 40, 76)
    window, sinks = 150, 10
    want = check(Q, c, tables, lens, new, 4, 77, window, sinks)
    for b in range(2):
        low = int(lens[b] - 5 - window + 1) // page  # the first row's window begins here
        for col in range(1, low):
            c["pool"][0, tables[b, col]] = POISON
            tables[b, col] = -1 if col % 2 else tables[b, col]
    q = synth.normal((10, 4, dim), 1.0, "bf16", 77).cuda()
    got = gpu_cache(Q, c).attend(0, q, i32(tables), i32(lens), window=window, sinks=sinks)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dt,page,new", [("bf16", 64, 1), ("f16", 64, 6), ("bf16", 32, 4), ("f16", 32, 1)])
def test_a_window_that_begins_with_a_page(Q, dt, page, new):
    """The page before the first row's first token holds nothing that a row sees: NaN there has no part, bit for bit, and with
    a mask, where the page is read, no more than another form of the steps has."""
    lens = np.array([8 * page + new + 31, 5 * page + new + 12])
    c, tables = filled(dt, 128, 64, page, 1, lens, 10, 20, 85)
    mask = [(2 << i) - 1 for _ in lens for i in range(new)]
    q = synth.normal((2 * new, 3, 128), 1.0, dt, 86).cuda()
    for b in range(2):
        window = int(lens[b] - new + 1) % page + page
        first = int(lens[b]) - new + 1 - window  # of the first row
        assert first % page == 0 and first > 0
        want = check(Q, c, tables, lens, np.full(2, new), 3, 86, window, 2)
        m = check(Q, c, tables, lens, np.full(2, new), 3, 86, window, 2, mask=mask)
        kept = c["pool"].copy()
        c["pool"][0, tables[b, first // page - 1]] = POISON
        cache = gpu_cache(Q, c)
        got = cache.attend(0, q, i32(tables), i32(lens), window=window, sinks=2)
        assert torch.equal(got[b * new:(b + 1) * new].view(torch.int16), want[b * new:(b + 1) * new].view(torch.int16))
        got = cache.attend(0, q, i32(tables), i32(lens), window=window, sinks=2, mask=torch.tensor(mask, device="cuda"))
        step = 2.0 ** (-10 if dt == "f16" else -7)  # (another form of the steps: within two roundings)
        assert ((got - m).float().abs() <= step * (m.float().abs() + 0.5))[b * new:(b + 1) * new].all()
        c["pool"][...] = kept


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_infinite_values_outside_the_window_have_no_part(Q, dt):
    """Tokens beside the window, in a step that is read for others, infinite or NaN: as if they were not there."""
    dim, gs, page = 128, 64, 64
    lens, new = np.array([333, 200]), np.array([3, 3])
    c, tables = filled(dt, dim, gs, page, 1, lens, 6, 14, 78)
    window, sinks = 77, 6
    want = check(Q, c, tables, lens, new, 5, 79, window, sinks)
    starts = np.array([0, 1, 2])
    for b in range(2):
        for t in (sinks, sinks + 1, int(lens[b]) - 3 - window, int(lens[b]) - 3 - window - 1):  # beside the sinks, before every window
            k = np.full((2, 1, dim), 0x7E00 if dt == "f16" else 0x7FC0, np.uint16)
            v = np.full((2, 1, dim), 0x7C00 if dt == "f16" else 0x7F80, np.uint16)
            page_of = tables[b, t // page]
            half = c["pool"].view(np.uint16)
            for part in (0, 1):
                at = KO._half_at(c, part, t % page)
                half[0, page_of, 0, at] = (k if t % 2 else v)[0, 0, 0]
                half[0, page_of, 0, at + 4] = (v if t % 2 else k)[0, 0, 0]
    q = synth.normal((6, 5, dim), 1.0, dt, 79).cuda()
    got, lse = gpu_cache(Q, c).attend(0, q, i32(tables), i32(lens), window=window, sinks=sinks, lse=True)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    # the form of a step may change with a scale that is not finite, so not bit for bit: within two roundings of the output
    step = 2.0 ** (-10 if dt == "f16" else -7)
    assert ((got - want).float().abs() <= step * (want.float().abs() + 0.5)).all()


def test_a_window_beyond_the_sequence_is_none(Q):
    lens, new = np.array([500, 77, 9]), np.array([6, 1, 9])
    c, tables = filled("f16", 128, 64, 64, 2, lens, 8, 20, 80)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = synth.normal((16, 8, 128), 1.0, "f16", 81).cuda()
    cache = gpu_cache(Q, c)
    args = (0, q, i32(tables), i32(lens))
    kw = dict(starts=i32(starts), max_new=9, lse=True)
    a, la = cache.attend(*args, **kw)
    for window in (500, 1 << 31, 1 << 62):
        b, lb = cache.attend(*args, window=window, sinks=7, **kw)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    b, lb = cache.attend(*args, window=1, sinks=1 << 40, **kw)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


def test_window_refusals(Q):
    c, tables = filled("f16", 64, 64, 32, 1, np.array([20]), 1, 2, 82)
    cache, q = gpu_cache(Q, c), torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    for kw in (dict(window=0), dict(window=-1), dict(window=5, sinks=-1), dict(sinks=4)):
        with pytest.raises(ValueError):
            cache.attend(0, q, i32(tables), i32([20]), **kw)
    with pytest.raises(Q.QmmError):
        cache.attend_workspace_bytes(1, 1, 1, 2, 100, 0, 4)


def test_window_in_graphs_and_beside_others(Q):
    """Two captured calls and eager ones, with a window and without, on the cache's own workspaces: the eager results again."""
    lens, new = np.array([3000, 2000]), np.array([4, 4])
    c, tables = filled("bf16", 64, 64, 64, 2, lens, 48, 90, 83)
    cache = gpu_cache(Q, c)
    q = synth.normal((8, 8, 64), 1.0, "bf16", 84).cuda()
    args = (0, q, i32(tables), i32(lens))
    run = lambda: [cache.attend(*args, window=1500, sinks=4, lse=True), cache.attend(*args, lse=True), cache.attend(*args, window=64, lse=True)]
    flat = lambda r: [t for pair in r for t in pair]
    want = [t.clone() for t in flat(run())]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = flat(run())
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
            eager = flat(run())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(eager, want))
