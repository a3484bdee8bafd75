"""The paged 4-bit K/V cache on the GPU against the CPU oracle: appended
records bit for bit, values read back bit for bit, attention within the bound
the oracle derives per element, page bookkeeping exactly."""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import kv_oracle as KO
from oracle import qmm_oracle as O

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = [(dim, gs) for dim in (64, 128, 256) for gs in (32, 64, 128) if gs <= dim]
POISON = 0x7FFF7FFF  # both halves NaN in fp16 and bf16


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import affine_quantized_gemm_amd as Q
    return Q


def gpu_pool(c):
    return torch.from_numpy(c["pool"].view(np.int32).copy()).cuda()


def gpu_cache(Q, c):
    return Q.KVCache(gpu_pool(c), c["dim"], c["gs"], c["page"], DT[c["dt"]])


def words(cache):
    return cache.pool.cpu().numpy().view(np.uint32)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def tables_for(lens, page, width, pages, seed):
    """Random pages for each sequence, -1 past its end."""
    order = np.random.default_rng(seed).permutation(pages)
    t, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(lens):
        m = -(-max(int(n), 0) // page)
        t[b, :m] = order[at:at + m]
        at += m
    return t


def values(rows, heads, dim, dt, seed, kind="normal"):
    if kind == "normal":
        return synth.normal((rows, heads, dim), 1.0, dt, seed, outlier_frac=0.01, outlier_scale=8.0)
    return synth.special_groups(kind, rows * heads, dim, 32, dt, seed).view(rows, heads, dim)


def filled(dt, dim, gs, page, kv_heads, lens, width, pages, seed, layers=1):
    """A cache whose sequences hold values; everything else is poison."""
    c = KO.new_cache(layers, pages, kv_heads, dim, gs, page, dt, fill=POISON)
    tables = tables_for(lens, page, width, pages, seed)
    starts = np.concatenate([[0], np.cumsum(np.maximum(lens, 0))])
    n = int(starts[-1])
    off = synth.normal((1, kv_heads, dim), 1.5, "f16", seed + 3).float()
    k = (synth.normal((n, kv_heads, dim), 1.0, dt, seed + 1).float() + off).to(DT[dt])
    v = values(n, kv_heads, dim, dt, seed + 2)
    KO.append(c, layers - 1, synth.to_oracle(k), synth.to_oracle(v), tables, np.maximum(lens, 0), starts)
    return c, tables


# ---- append and read ----

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,gs", FORMATS)
@pytest.mark.parametrize("kind", ["normal", "mixed", "constant", "tiny"])
def test_append_is_bit_exact_and_touches_nothing_else(Q, dt, dim, gs, kind):
    print(f"append {dt} D={dim} gs={gs} {kind}", flush=True)
    page, kv_heads, width = 32, 3, 4
    lens = np.array([1, 33, 64, 7, 100, 0, 5, 90])
    new = np.array([1, 2, 5, 7, 37, 0, 3, 90])  # from one token to several pages, at every offset in a bundle
    starts = np.concatenate([[0], np.cumsum(new)])
    tables = tables_for(lens, page, width, 24, 5)
    k, v = (values(int(starts[-1]), kv_heads, dim, dt, 40 + i, kind) for i in (0, 1))
    c = KO.new_cache(2, 24, kv_heads, dim, gs, page, dt, fill=0xA5C3A5C3)
    cache = gpu_cache(Q, c)
    KO.append(c, 1, synth.to_oracle(k), synth.to_oracle(v), tables, lens, starts)
    cache.append(1, k.cuda(), v.cuda(), i32(tables), i32(lens), starts=i32(starts), max_new=90)
    assert np.array_equal(words(cache), c["pool"])
    kg, vg = cache.read(1, int(starts[-1]), i32(tables), i32(lens), starts=i32(starts), max_new=90)
    ko, vo = KO.read(c, 1, tables, lens, starts, kv_heads)
    for got, want in ((kg, ko), (vg, vo)):  # s*q + b is rounded to fp32, then to the type
        want = O.f32_to_dt_rne(want.astype(np.float32), dt)
        assert np.array_equal(synth.to_oracle(got).view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("page,seqs,new", [(32, 5, 1), (64, 3, 4), (128, 2, 6), (256, 1, 300)])
def test_append_uniform_rows_strided_operands(Q, page, seqs, new):
    """k and v as slices of one projection's output, padded rows; one row count for all."""
    dim, gs, kv_heads, dt = 128, 64, 2, "bf16"
    lens = np.array([new + 17 * b for b in range(seqs)])
    width = -(-int(lens.max()) // page)
    tables = tables_for(lens, page, width, 20, 6)
    both = synth.normal((seqs * new, (5 + 2 * kv_heads) * dim + 8), 1.0, dt, 7).cuda()
    k = both[:, 3 * dim:(3 + kv_heads) * dim].view(-1, kv_heads, dim)
    v = both[:, 5 * dim:(5 + kv_heads) * dim].view(-1, kv_heads, dim)
    c = KO.new_cache(1, 20, kv_heads, dim, gs, page, dt, fill=1)
    cache = gpu_cache(Q, c)
    starts = np.arange(seqs + 1) * new
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, lens, starts)
    cache.append(0, k, v, i32(tables), i32(lens))
    assert np.array_equal(words(cache), c["pool"])


def test_append_and_read_skip_what_has_no_place(Q):
    """Positions before 0, past the table, on entries that name no page: skipped, read as zeros."""
    dim, gs, page, kv_heads = 64, 64, 32, 2
    tables = np.array([[3, 99], [-1, 2], [1, 0], [4, -7]], np.int32)  # 5 pages
    lens, new = np.array([60, 40, 66, 3]), np.array([40, 40, 5, 6])
    starts = np.concatenate([[0], np.cumsum(new)])
    k, v = (values(int(starts[-1]), kv_heads, dim, "f16", 50 + i) for i in (0, 1))
    c = KO.new_cache(1, 5, kv_heads, dim, gs, page, "f16", fill=9)
    cache = gpu_cache(Q, c)
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, lens, starts)
    cache.append(0, k.cuda(), v.cuda(), i32(tables), i32(lens), starts=i32(starts), max_new=40)
    assert np.array_equal(words(cache), c["pool"])
    kg, vg = cache.read(0, int(starts[-1]), i32(tables), i32(lens), starts=i32(starts), max_new=40)
    ko, vo = KO.read(c, 0, tables, lens, starts, kv_heads)
    assert np.array_equal(kg.cpu().numpy(), ko.astype(np.float32).astype(np.float16))
    assert np.array_equal(vg.cpu().numpy(), vo.astype(np.float32).astype(np.float16))


# ---- attention ----

def check_attend(Q, c, tables, lens, new, heads, seed, mask=None, scale=None, width_bound=True, layer=0, max_len=None):
    dim, dt = c["dim"], c["dt"]
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1])
    q = synth.normal((rows, heads, dim), 1.0, dt, seed)
    scale = 1 / math.sqrt(dim) if scale is None else scale
    out, lse, tol, ltol = KO.attend(c, layer, O.to_f64(synth.to_oracle(q), dt), tables, lens, starts, scale, mask)
    cache = gpu_cache(Q, c)
    ragged = len(set(new)) != 1
    kw = {"starts": i32(starts), "max_new": int(max(new))} if ragged else {}
    m = None if mask is None else torch.tensor(mask, dtype=torch.int64, device="cuda")
    args = (layer, q.cuda(), i32(tables), i32(lens))
    got, glse = cache.attend(*args, mask=m, scale=scale, lse=True, max_len=max_len, **kw)
    again = cache.attend(*args, mask=m, scale=scale, max_len=max_len, **kw)
    g = O.to_f64(synth.to_oracle(got), dt)
    assert np.isfinite(g).all()
    err = np.abs(g - out)
    print(f"  worst err/bound {np.max(err / np.maximum(tol, 1e-30), initial=0):.3f}", flush=True)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-30)).max()
    gl = glse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (g[empty] == 0).all()
    assert (np.abs(gl[~empty] - lse[~empty]) <= ltol[~empty]).all()
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))  # the same bits again, with and without lse
    return got


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_attend_formats(Q, dt, dim, gs):
    """Ragged rows and lengths around tile and page ends, shared heads, poison past the ends."""
    print(f"attend {dt} D={dim} gs={gs}", flush=True)
    lens = np.array([1, 5, 31, 32, 33, 64, 97, 130])
    new = np.array([1, 4, 1, 6, 5, 3, 1, 2])
    c, tables = filled(dt, dim, gs, 32, 2, lens, 5, 24, 60)
    check_attend(Q, c, tables, lens, new, 6, 61)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (7, 1), (8, 2), (24, 2), (64, 4)])
@pytest.mark.parametrize("rows", [1, 3, 8, 17])
def test_attend_head_layouts(Q, heads, kv_heads, rows):
    print(f"attend heads={heads}/{kv_heads} rows={rows}", flush=True)
    lens = np.array([rows, 50, 77])
    c, tables = filled("f16" if rows % 2 else "bf16", 128, 64, 64, kv_heads, lens, 2, 6, 70)
    check_attend(Q, c, tables, lens, np.full(3, rows), heads, 71)


@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_attend_page_sizes_and_layers(Q, page):
    print(f"attend page={page}", flush=True)
    lens = np.array([page, page + 1, 2 * page - 1, 3])
    c, tables = filled("f16", 64, 32, page, 1, lens, 2, 8, 80, layers=2)
    check_attend(Q, c, tables, lens, np.array([1, 2, 6, 3]), 4, 81, layer=1)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 5, 64])
def test_attend_long(Q, dt, rows):
    """Long sequences beside short ones, split over workgroups; a bound on the lengths that is kept, and one that is not."""
    print(f"attend long {dt} rows={rows}", flush=True)
    lens = np.array([2500, rows, 700, 1999 + rows])
    c, tables = filled(dt, 128, 64, 64, 1, lens, 42, 90, 90)
    new = np.full(4, rows)
    a = check_attend(Q, c, tables, lens, new, 2, 91)
    check_attend(Q, c, tables, lens, new, 2, 91, max_len=2500)
    check_attend(Q, c, tables, lens, new, 2, 91, max_len=100)
    assert a.shape == (4 * rows, 2, 128)


@pytest.mark.parametrize("dt,dim,gs,heads,rows", [
    ("f16", 128, 64, 10, 5), ("bf16", 64, 32, 6, 7), ("f16", 64, 64, 3, 14),  # 3 and 4 tiles of rows over long sequences
    ("bf16", 128, 128, 5, 20), ("f16", 128, 32, 9, 33), ("bf16", 256, 64, 3, 30),  # more
])
def test_attend_many_rows_long(Q, dt, dim, gs, heads, rows):
    """Ragged rows that leave tiles, wavefronts and workgroups without any, over long sequences and short ones."""
    print(f"attend {dt} D={dim} gs={gs} heads={heads} rows={rows}", flush=True)
    new = np.array([rows, 1, rows // 2, rows])
    lens = np.array([1600, 1100, rows, 300])
    c, tables = filled(dt, dim, gs, 64, 1, lens, 26, 56, 95)
    check_attend(Q, c, tables, lens, new, heads, 96)
    check_attend(Q, c, tables, lens, new, heads, 96, max_len=900)


@pytest.mark.parametrize("dt,dim,gs,kv_heads,group,rows,longest", [
    ("f16", 128, 64, 8, 1, 64, 40), ("bf16", 64, 32, 7, 3, 20, 150),  # 4 tiles of rows a sequence
    ("f16", 64, 64, 8, 5, 9, 260), ("bf16", 128, 32, 5, 7, 31, 129),  # 3, and 14
    ("bf16", 256, 64, 4, 3, 30, 70), ("f16", 256, 128, 8, 1, 33, 33),  # heads of 256: 6 and 3
])
def test_attend_many_rows_and_sequences(Q, dt, dim, gs, kv_heads, group, rows, longest):
    """Enough sequences for workgroups by rows; ragged ends of both, empty sequences, draft trees."""
    print(f"attend {dt} D={dim} gs={gs} kv_heads={kv_heads} group={group} rows={rows}", flush=True)
    rng = np.random.default_rng(7)
    seqs = 48
    new = rng.integers(0, rows + 1, seqs)
    new[:6] = rows, 1, rows, 0, 0, rows
    lens = np.maximum(new, rng.integers(0, longest + 1, seqs))
    lens[:6] = max(rows, longest), 1, rows, 0, longest, 32 * -(-rows // 32)
    width = -(-int(lens.max()) // 64) + 1
    c, tables = filled(dt, dim, gs, 64, kv_heads, lens, width, int((-(-lens // 64)).sum()) + 2, 97)
    most = int(lens.max())
    check_attend(Q, c, tables, lens, new, group * kv_heads, 98, max_len=most)
    masks = rng.integers(0, 1 << 62, int(new.sum())) * rng.integers(0, 2, int(new.sum()))
    check_attend(Q, c, tables, lens, new, group * kv_heads, 98, mask=masks, max_len=most)


def test_attend_many_sequences(Q):
    """More sequences than are planned over: one part each, however long."""
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 40, 300)
    lens[[0, 257]] = 900, 1300
    c, tables = filled("f16", 64, 32, 32, 1, lens, 41, int((-(-lens // 32)).sum()), 99)
    check_attend(Q, c, tables, lens, np.ones(300, int), 4, 100)


def test_pool_beyond_32_bits(Q):
    """Pages whose words lie past 2^31 bytes, 2^32 bytes and 2^31 words: append, read, attend, copy."""
    lens, new, pages = np.array([300, 513, 256]), np.array([3, 1, 5]), 13200
    c, tables = filled("f16", 256, 32, 256, 8, lens, 3, 6, 101)
    small = gpu_cache(Q, c)
    big = Q.KVCache.empty(1, pages, 8, 256, 32, 256)
    assert big.pool.numel() > 2 ** 31
    place = torch.tensor([pages - 1, 4000, 7000, pages - 2, 9000, pages - 7], device="cuda")
    big.pool[:, place] = small.pool
    far = torch.where(i32(tables) < 0, i32(tables), place.to(torch.int32)[i32(tables).long()])
    starts = np.concatenate([[0], np.cumsum(new)])
    kw = {"starts": i32(starts), "max_new": 5}
    k, v, q = (values(9, h, 256, "f16", 102 + h).cuda() for h in (8, 8, 16))
    got = []
    for cache, t in ((small, i32(tables)), (big, far)):
        cache.append(0, k, v, t, i32(lens), **kw)
        got.append((*cache.read(0, 9, t, i32(lens), **kw), cache.attend(0, q, t, i32(lens), **kw)))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(big.pool[:, place], small.pool)
    big.copy_pages(i32([pages - 1, 4000]), i32([4001, pages - 3]))
    assert torch.equal(big.pool[:, [4001, pages - 3]], small.pool[:, :2])


def test_attend_on_two_streams(Q):
    """Calls in flight on two streams, each cut into parts with counters of its own."""
    lens = np.array([1536])
    c, tables = filled("f16", 128, 64, 64, 2, lens, 24, 24, 110)
    cache = gpu_cache(Q, c)
    t = [i32(tables), i32(tables[:, ::-1].copy())]
    n = i32(lens)
    q = [synth.normal((1, 8, 128), 1.0, "f16", 112 + i).cuda() for i in range(2)]
    want = [cache.attend(0, q[i], t[i], n) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(cache.attend(0, q[i], t[i], n))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g.view(torch.int16), want[i].view(torch.int16)) for g in got[i])


def test_attend_masks(Q):
    """Draft trees; rows that see only what was before, or nothing at all."""
    rng = np.random.default_rng(1)
    new = np.array([13, 64, 4, 7, 1, 2])
    lens = np.array([40, 64, 4, 100, 1, 35])  # sequences 1, 2 and 4 have nothing before the new tokens
    mask = []
    for b, n in enumerate(new):
        for i in range(n):
            word = (1 << i) | int(rng.integers(0, 1 << 62)) & ((1 << i) - 1)
            if b == 2 or (b == 1 and i in (0, 5, 63)) or b == 4:
                word = 0  # sees nothing
            elif b == 3:
                word = 0 if i % 2 else (1 << i)  # sees what was before
            elif b == 5:
                word = -1  # every bit: new tokens that exist, later ones too
            mask.append(word - (1 << 64) if word >> 63 and word > 0 else word)
    mask = np.array(mask, dtype=np.int64)
    for dt, dim, gs in (("f16", 128, 64), ("bf16", 64, 64)):
        print(f"attend masks {dt}", flush=True)
        c, tables = filled(dt, dim, gs, 32, 2, lens, 4, 16, 100)
        check_attend(Q, c, tables, lens, new, 4, 101, mask=mask)


@pytest.mark.parametrize("dt,gs", [("f16", 32), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("heads", [2, 40])
def test_attend_infinite_values(Q, dt, gs, heads):
    """Draft tokens of infinite and NaN values: the rows that do not see them are as if they were not; a value that all
    rows see takes its own group only."""
    print(f"attend infinite {dt} gs={gs} heads={heads}", flush=True)
    inf, nan = float("inf"), float("nan")
    masks = torch.tensor([0b1, 0b11, 0b101, 0b1000, 0b10001, 0b100001], dtype=torch.int64, device="cuda")
    k, v = (values(300, 1, 128, dt, 150 + i) for i in (0, 1))
    q = synth.normal((6, heads, 128), 1.0, dt, 152).cuda()
    tables, lens = i32(np.arange(5)[None]), i32([300])
    out = []
    for bad in (False, True):
        cache = Q.KVCache.empty(1, 5, 1, 128, gs, 64, DT[dt])
        if bad:  # the fourth and sixth new tokens
            k[297], v[297], k[299], v[299, 0, :gs] = nan, inf, inf, -inf
        cache.append(0, k.cuda(), v.cuda(), tables, lens)
        out.append(cache.attend(0, q, tables, lens, mask=masks, lse=True))
    (a, la), (b, lb) = out
    others = [0, 1, 2, 4]
    assert torch.isfinite(a).all()
    assert torch.equal(a[others].view(torch.int16), b[others].view(torch.int16)) and torch.equal(la[others], lb[others])
    assert not torch.isfinite(b[3]).any() and not torch.isfinite(b[5, :, :gs]).any()
    # before the new tokens, where every row sees it: one group of one token
    if gs < 128:
        v[297], k[297], k[299], v[299], v[20, 0, gs:2 * gs] = 0, 0, 0, 0, inf
        cache.append(0, k.cuda(), v.cuda(), tables, lens)
        c = cache.attend(0, q, tables, lens, mask=masks)
        seen = torch.ones(128, dtype=torch.bool)
        seen[gs:2 * gs] = False
        assert not torch.isfinite(c[..., ~seen]).any()
        assert torch.equal(c[others][..., seen].view(torch.int16), a[others][..., seen].view(torch.int16))


def test_attend_nothing_to_see(Q):
    """No tokens, lengths below the new rows, no page, a table of width 0."""
    lens, new = np.array([0, 0, 2, 40, -5]), np.array([1, 3, 5, 2, 2])
    c, tables = filled("f16", 64, 32, 32, 1, lens, 2, 6, 110)
    tables[3, 0] = 77  # its first 32 tokens have no page
    check_attend(Q, c, tables, lens, new, 2, 111)
    check_attend(Q, c, np.zeros((5, 0), np.int32), lens, new, 2, 111)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attend_large_and_small_scores(Q, dt):
    """Scores in the hundreds (one token takes all) and of no size (the mean)."""
    lens, new = np.array([150, 61]), np.array([2, 6])
    c, tables = filled(dt, 128, 32, 32, 2, lens, 5, 9, 120)
    for scale in (8.0, -8.0, 1e-6, 0.0):
        print(f"attend {dt} scale={scale}", flush=True)
        check_attend(Q, c, tables, lens, new, 8, 121, scale=scale)


@pytest.mark.parametrize("dt,size", [("f16", 2.0 ** -9), ("f16", 512.0), ("bf16", 2.0 ** -40), ("bf16", 2.0 ** 40)])
def test_attend_value_ranges(Q, dt, size):
    """Values far from 1 (K scaled the other way in bf16, so that scores keep their size)."""
    print(f"attend values {dt} {size}", flush=True)
    lens = np.array([70, 3])
    tables = tables_for(lens, 32, 3, 5, 130)
    c = KO.new_cache(1, 5, 1, 64, 32, 32, dt, fill=POISON)
    k = synth.normal((73, 1, 64), 1.0, dt, 131)
    v = (synth.normal((73, 1, 64), 1.0, dt, 132).float() * size).to(DT[dt])
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, lens, [0, 70, 73])
    q = synth.normal((2, 2, 64), 1.0, dt, 133)
    out, _, tol, _ = KO.attend(c, 0, O.to_f64(synth.to_oracle(q), dt), tables, lens, [0, 1, 2], 0.125)
    got = gpu_cache(Q, c).attend(0, q.cuda(), i32(tables), i32(lens))
    assert (np.abs(O.to_f64(synth.to_oracle(got), dt) - out) <= tol).all()


def test_attend_strided_q_out_and_stream(Q):
    """q as a slice of a projection, a given out, a stream of its own."""
    lens, new = np.array([70, 33]), np.array([3, 3])
    c, tables = filled("bf16", 128, 64, 64, 2, lens, 2, 5, 140)
    cache = gpu_cache(Q, c)
    qkv = synth.normal((6, 9 * 128), 1.0, "bf16", 141).cuda()
    q = qkv[:, 128:5 * 128].view(6, 4, 128)
    want = cache.attend(0, q.contiguous(), i32(tables), i32(lens))
    out = torch.full_like(want, float("nan"))
    t, n = i32(tables), i32(lens)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cache.attend(0, q, t, n, out=out, stream=st)
    st.synchronize()
    assert got is out and torch.equal(out, want)
    got = cache.attend(0, q, t, n, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_step_in_a_graph(Q):
    """append + attend captured once, replayed as the lengths grow; each replay against the eager calls."""
    dim, gs, page, kv_heads, heads = 128, 64, 32, 2, 8
    c = KO.new_cache(1, 12, kv_heads, dim, gs, page, "f16", fill=POISON)
    graph_cache, eager = gpu_cache(Q, c), gpu_cache(Q, c)
    tables = i32(np.random.default_rng(3).permutation(12).reshape(2, 6))
    lens = i32([1, 3])  # as the first replay, so that the warm-up call writes no other place
    q, k, v = (torch.zeros(2, h, dim, dtype=torch.float16, device="cuda") for h in (heads, kv_heads, kv_heads))
    out = torch.zeros_like(q)
    ws = graph_cache.attend_workspace(2, 1, 2, heads, 192)
    step = lambda: (graph_cache.append(0, k, v, tables, lens),
                    graph_cache.attend(0, q, tables, lens, out=out, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in range(1, 190, 9):
        for x, s in ((q, 0), (k, 1), (v, 2)):
            x.copy_(synth.normal(tuple(x.shape), 1.0, "f16", 1000 * s + t))
        lens.copy_(i32([t, t + 2]))
        g.replay()
        eager.append(0, k, v, tables, lens)
        want = eager.attend(0, q, tables, lens, max_len=192)
        torch.cuda.synchronize()
        assert torch.equal(graph_cache.pool, eager.pool)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), t


def test_graph_without_a_given_workspace(Q):
    """A captured call that is cut into parts brings its own zeroed workspace; eager calls go on between replays."""
    lens = np.array([1000, 1040])
    c, tables = filled("bf16", 128, 64, 64, 2, lens, 18, 33, 145)
    cache = gpu_cache(Q, c)
    t, n = i32(tables), i32(lens)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert cache.attend_workspace_bytes(2, 1, 2, 8, 18 * 64) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attend(0, q, t, n)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cache.attend(0, q, t, n)
    for r in range(6):
        q.copy_(synth.normal(tuple(q.shape), 1.0, "bf16", 146 + r))
        n.copy_(i32([1000 - 130 * r, 40 + 200 * r]))
        g.replay()
        want = cache.attend(0, q, t, n)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), r


def test_python_refusals(Q):
    cache = Q.KVCache.empty(1, 4, 2, 128, 64, 32, torch.float16)
    t, n = i32(np.zeros((2, 2))), i32([1, 1])
    q = torch.zeros(2, 4, 128, dtype=torch.float16, device="cuda")
    k = torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda")
    bad = [
        lambda: cache.attend(0, q[:, :, :64], t, n), lambda: cache.attend(0, q.bfloat16(), t, n),
        lambda: cache.attend(0, q.cpu(), t, n), lambda: cache.attend(0, q, t.long(), n),
        lambda: cache.attend(0, q, t, n[:1]), lambda: cache.attend(0, q, t.t(), n), lambda: cache.attend(1, q, t, n),
        lambda: cache.attend(0, q.transpose(1, 2).contiguous().transpose(1, 2), t, n),
        lambda: cache.attend(0, torch.zeros(3, 4, 128, dtype=torch.float16, device="cuda"), t, n),
        lambda: cache.attend(0, q, t, n, starts=i32([0, 1, 2])),
        lambda: cache.attend(0, q, t, n, starts=i32([0, 1]), max_new=1),
        lambda: cache.attend(0, q, t, n, mask=i32([1, 1])), lambda: cache.attend(0, q, t, n, out=q[:1]),
        lambda: cache.attend(0, q, t, n, lse=torch.zeros(2, 4, device="cuda").half()),
        lambda: cache.append(0, k, k[:, :1], t, n), lambda: cache.append(0, q, q, t, n),
        lambda: cache.append(0, k.float(), k.float(), t, n), lambda: cache.read(0, 3, t, n),
        lambda: cache.copy_pages(n, n[:1]), lambda: cache.free(t, n, i32([0, 0, 0]), n),
        lambda: cache.fork(t, n, i32([0] * 4), n, n.long()), lambda: cache.reserve(t, n, i32([0] * 4), i32([1])),
        lambda: cache.compact(t, i32([0] * 4), tables_out=t[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    for call in (lambda: cache.attend(0, torch.zeros(2, 3, 128, dtype=torch.float16, device="cuda"), t, n),  # 3 / 2 heads
                 lambda: cache.attend(0, torch.zeros(130, 4, 128, dtype=torch.float16, device="cuda"), t, n),  # 65 rows
                 lambda: cache.attend(0, torch.zeros(2, 4, 130, dtype=torch.float16, device="cuda")[:, :, 1:129], t, n)):
        with pytest.raises(Q.QmmError):
            call()


# ---- pages ----

def page_state(seed, seqs, width, pages, page, hold):
    """Tables, lengths and counts of a pool in use: sequences with random lengths, some pages held twice."""
    rng = np.random.default_rng(seed)
    tables, lens, refs = np.full((seqs, width), -1, np.int32), np.zeros(seqs, np.int32), np.zeros(pages, np.int32)
    order = list(rng.permutation(pages))
    for s in range(hold):
        n = int(rng.integers(0, width * page + 1))
        m = -(-n // page)
        if m > len(order):
            break
        for x in range(m):
            tables[s, x] = order.pop()
            refs[tables[s, x]] += 1
        lens[s] = n
    return tables, lens, refs


@pytest.mark.parametrize("pages,width,seqs", [(7, 2, 5), (700, 9, 60), (5000, 17, 300)])
@pytest.mark.parametrize("layers", [1, 3])
def test_pages_against_the_oracle(Q, pages, width, seqs, layers):
    """Rounds of reserve, fork, cut back, free and compact, each against the oracle, through exhaustion of the pool."""
    page, dim, gs, kv_heads = 32, 64, 64, 1
    rng = np.random.default_rng(pages + layers)
    c = KO.new_cache(layers, pages, kv_heads, dim, gs, page, "f16")
    c["pool"][:] = rng.integers(0, 1 << 32, c["pool"].shape, dtype=np.uint32)
    cache = gpu_cache(Q, c)
    tables, lens, refs = page_state(pages, seqs, width, pages, page, seqs // 2)
    gt, gl, gr = i32(tables), i32(lens), i32(refs)
    pool = c["pool"]

    def same(what):
        assert np.array_equal(gt.cpu().numpy(), tables), what
        assert np.array_equal(gl.cpu().numpy(), lens), what
        assert np.array_equal(gr.cpu().numpy(), refs), what

    for turn in range(4):
        print(f"pages={pages} width={width} layers={layers} turn={turn} live={(refs > 0).sum()}", flush=True)
        add = rng.integers(-1, 2 * page, seqs).astype(np.int32)
        add[rng.random(seqs) < 0.3] = 0
        ok = cache.reserve(gt, gl, gr, i32(add))
        assert np.array_equal(ok.cpu().numpy(), KO.reserve(tables, lens, refs, add, page))
        same("reserve")
        # rejected drafts: lengths cut back, inside the last page or off it
        for s in range(seqs):
            if lens[s] > 3 and rng.random() < 0.5:
                lens[s] -= int(rng.integers(1, 4))
        gl.copy_(i32(lens))
        empty = [s for s in range(seqs) if lens[s] == 0 and (tables[s] < 0).all()]
        held = [s for s in range(seqs) if s not in empty]
        dst = rng.permutation(empty)[: max(1, len(empty) // 2)] if empty else np.zeros(0, int)
        src = rng.choice(held, len(dst)) if held and len(dst) else dst[:0]
        dst = dst[: len(src)]
        if len(src) > 2:
            src[1], dst[0] = seqs + 5, dst[0]  # no such sequence
        ok = cache.fork(gt, gl, gr, i32(src), i32(dst))
        assert np.array_equal(ok.cpu().numpy(), KO.fork(pool, tables, lens, refs, src, dst, page))
        same("fork")
        which = rng.permutation(seqs)[: seqs // 4]
        which = np.concatenate([which, which[:2], [-3, seqs]])  # some twice, some that are none
        cache.free(gt, gl, gr, i32(which))
        KO.free(tables, lens, refs, list(dict.fromkeys(which)))
        same("free")
        live = i32([0])
        to, ro, n = KO.compact(pool, tables, refs)
        if turn % 2:  # into other tensors, then in place
            ot, orf = cache.compact(gt, gr, live=live)
            same("compact leaves its inputs")
            assert ot is not gt and np.array_equal(ot.cpu().numpy(), to) and np.array_equal(orf.cpu().numpy(), ro)
            gt, gr = ot, orf
        else:
            cache.compact(gt, gr, tables_out=gt, refs_out=gr, live=live)
        tables, refs = to, ro
        same("compact")
        assert int(live) == n
        assert np.array_equal(words(cache), pool)


@pytest.mark.parametrize("kv_heads,dim,gs,page", [(1, 64, 64, 32), (5, 128, 64, 64), (2, 256, 32, 256)])
def test_copy_pages(Q, kv_heads, dim, gs, page):
    c = KO.new_cache(2, 11, kv_heads, dim, gs, page, "bf16")
    c["pool"][:] = np.random.default_rng(9).integers(0, 1 << 32, c["pool"].shape, dtype=np.uint32)
    cache = gpu_cache(Q, c)
    src, dst = [10, 3, -1, 4, 0, 11], [1, 2, 5, 6, -1, 7]
    cache.copy_pages(i32(src), i32(dst))
    for s, d in ((10, 1), (3, 2), (4, 6)):
        c["pool"][:, d] = c["pool"][:, s]
    assert np.array_equal(words(cache), c["pool"])


def test_forked_sequences_attend_alike_and_then_apart(Q):
    """A fork reads what its source reads; tokens appended to one do not show in the other."""
    dim, gs, page, kv_heads, heads = 128, 64, 32, 2, 8
    cache = Q.KVCache.empty(2, 16, kv_heads, dim, gs, page, torch.bfloat16)
    tables, lens, refs = i32(np.full((3, 4), -1)), i32([0, 0, 0]), i32([0] * 16)
    draw = lambda n, h, s: synth.normal((n, h, dim), 1.0, "bf16", s).cuda()
    cache.reserve(tables, lens, refs, i32([45, 0, 0]))
    k, v = draw(45, kv_heads, 1), draw(45, kv_heads, 2)
    for layer in (0, 1):
        cache.append(layer, k, v, tables, lens, starts=i32([0, 45, 45, 45]), max_new=45)
    assert cache.fork(tables, lens, refs, i32([0, 0]), i32([1, 2])).tolist() == [1, 1]
    assert lens.tolist() == [45, 45, 45] and refs.tolist()[:4] == [3, 1, 1, 1]
    q = draw(3, heads, 3)
    q[1:] = q[0]
    same = cache.attend(1, q, tables, lens)
    assert torch.equal(same[0], same[1]) and torch.equal(same[0], same[2])
    cache.reserve(tables, lens, refs, i32([1, 1, 1]))
    k, v = draw(3, kv_heads, 4), draw(3, kv_heads, 5)
    cache.append(1, k, v, tables, lens)
    apart = cache.attend(1, q, tables, lens)
    assert not torch.equal(apart[0], apart[1]) and not torch.equal(apart[1], apart[2])
    kb, vb = cache.read(1, 3, tables, lens)
    assert (kb - k).abs().max() < 0.5 and (vb - v).abs().max() < 0.5
    cache.free(tables, lens, refs, i32([0, 1, 2]))
    assert refs.tolist() == [0] * 16 and lens.tolist() == [0, 0, 0] and (tables == -1).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_speculative_decoding_example(Q, dt):
    """Forked sequences, draft trees, cut back lengths, freed and compacted pages: every token that came out is the
    likeliest one of a plain pass over its whole text.

    Both passes quantize keys and values that differ by roundings, so a code may be the neighbour: a step of about
    0.4 standard deviations in one of 128 values moves a score by 0.4 / sqrt(128) = 0.035, and as much of one
    token's share of the sums; over both layers the logits move by well under a tenth of their deviation."""
    from affine_quantized_gemm_amd import spec_decode as S
    print(f"speculative decoding {dt}", flush=True)
    model = S.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=512, vocab=512, dtype=DT[dt])
    s = S.Sequences(model, 3, 70 + 1 + 45 * 7, 3)
    prompt = torch.randint(0, 512, (70,), generator=torch.Generator().manual_seed(1)).cuda()
    s.fork(s.prefill(prompt)[-1])
    for _ in range(25):
        s.step()
    ended = s.texts()
    s.end([1])
    assert s.refs[:int((s.refs > 0).sum())].min() > 0  # the live pages are the lowest
    for _ in range(15):
        s.step()
    texts = s.texts()
    assert len(texts) == 2 and texts[0][:len(ended[0])] == ended[0] and texts[1][:len(ended[2])] == ended[2]
    assert len({e[70] for e in ended}) == 3
    assert sum(len(t) - 71 for t in texts) > 2 * 40 * 1.5  # drafts were accepted
    for text in [*texts, ended[1]]:
        logits = S.logits_of(model, text[:-1])[70:].float()
        got = logits.gather(1, torch.tensor(text[71:], device="cuda")[:, None])[:, 0]
        assert ((logits.amax(1) - got) <= 0.1 * logits.std(1)).all()
