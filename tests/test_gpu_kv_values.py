"""Attention over the paged K/V cache within the bound that follows its roundings (``kv_oracle.attend_bound``), on
ordinary values and on those where a running reference or a small type goes wrong."""

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
BOTH = pytest.mark.parametrize("dt", ["f16", "bf16"])


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import affine_quantized_gemm_amd as Q
    return Q


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def normal(shape, dt, seed, std=1.0):
    return synth.normal(shape, std, dt, seed)


def cache_of(k, v, gs, dt, lens, page=64, seed=1):
    """A cache that holds the sequences' k and v [tokens, kv_heads, dim], and its tables; poison elsewhere."""
    lens = np.asarray(lens)
    need = -(-lens // page)
    pages = int(need.sum()) + 1
    c = KO.new_cache(1, pages, k.shape[1], k.shape[2], gs, page, dt, fill=0x7FFF7FFF)
    order, at = np.random.default_rng(seed).permutation(pages), 0
    tables = np.full((len(lens), int(need.max()) + 1), -1, np.int32)
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, lens, np.concatenate([[0], np.cumsum(lens)]))
    return c, tables


def call(Q, c, q, tables, lens, new, mask=None, scale=None, max_len=None):
    """(out, lse) of the kernel."""
    cache = Q.KVCache(torch.from_numpy(c["pool"].view(np.int32).copy()).cuda(), c["dim"], c["gs"], c["page"], DT[c["dt"]])
    kw = {"starts": i32(np.concatenate([[0], np.cumsum(new)])), "max_new": int(max(new))} if len(set(new)) > 1 else {}
    m = None if mask is None else torch.tensor(mask, dtype=torch.int64, device="cuda")
    return cache.attend(0, q.cuda(), i32(tables), i32(lens), mask=m, scale=scale, max_len=max_len, lse=True, **kw)


def check(Q, c, q, tables, lens, new, mask=None, scale=None, max_len=None, oracle=None):
    """The kernel against the oracle, within its bound; returns the kernel's and the oracle's results."""
    dt = c["dt"]
    scale = 1 / math.sqrt(c["dim"]) if scale is None else scale
    if oracle is None:
        oracle = KO.attend_bound(c, 0, O.to_f64(synth.to_oracle(q), dt), tables, lens,
                                 np.concatenate([[0], np.cumsum(new)]), scale, mask)
    out, lse, tol, ltol = oracle
    got, glse = call(Q, c, q, tables, lens, new, mask, scale, max_len)
    g, gl = O.to_f64(synth.to_oracle(got), dt), glse.cpu().numpy().astype(np.float64)
    seen = ~np.isneginf(lse)
    bad = ~(np.abs(g - out) <= tol)
    with np.errstate(invalid="ignore"):
        print(f"  err/bound {np.nanmax(np.abs(g - out) / np.maximum(tol, 1e-300)):.3f}, "
              f"lse {np.nanmax(np.abs(gl[seen] - lse[seen]) / ltol[seen], initial=0):.3f}, "
              f"not finite {np.count_nonzero(~np.isfinite(g))}", flush=True)
    assert not bad.any(), f"{np.count_nonzero(bad)} of {bad.size} beyond the bound"
    assert np.array_equal(np.isneginf(gl), ~seen) and (g[~seen] == 0).all()
    assert (np.abs(gl[seen] - lse[seen]) <= ltol[seen]).all()
    return got, oracle


def offset_keys(n, kv_heads, dim, dt, seed):
    """Keys as a model leaves them: channels with offsets."""
    return (normal((n, kv_heads, dim), dt, seed).float() + normal((1, kv_heads, dim), "f16", seed + 1, 1.5).float()).to(DT[dt])


# ---- the bound, at ordinary values ----

@BOTH
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_formats(Q, dt, dim, gs):
    print(f"formats {dt} D={dim} gs={gs}", flush=True)
    lens, new = np.array([1, 33, 70, 130]), np.array([1, 4, 6, 2])
    n = int(lens.sum())
    c, tables = cache_of(offset_keys(n, 2, dim, dt, 10), normal((n, 2, dim), dt, 12), gs, dt, lens, page=32)
    check(Q, c, normal((13, 6, dim), dt, 13), tables, lens, new)


@BOTH
@pytest.mark.parametrize("rows,heads", [(1, 2), (5, 2), (5, 8), (40, 1)])
def test_long(Q, dt, rows, heads):
    """Cut over workgroups and not, one tile of rows and more."""
    print(f"long {dt} rows={rows} heads={heads}", flush=True)
    lens, new = np.array([1700, 600 + rows]), np.full(2, rows)
    n = int(lens.sum())
    c, tables = cache_of(offset_keys(n, 1, 128, dt, 20), normal((n, 1, 128), dt, 22), 64, dt, lens)
    q = normal((2 * rows, heads, 128), dt, 23)
    _, oracle = check(Q, c, q, tables, lens, new)
    check(Q, c, q, tables, lens, new, max_len=64, oracle=oracle)


@BOTH
def test_by_rows(Q, dt):
    """Enough short sequences for workgroups by rows."""
    print(f"by rows {dt}", flush=True)
    lens = np.array([40 + b % 9 for b in range(40)])
    n = int(lens.sum())
    c, tables = cache_of(offset_keys(n, 4, 64, dt, 30), normal((n, 4, 64), dt, 32), 32, dt, lens)
    check(Q, c, normal((40 * 18, 8, 64), dt, 33), tables, lens, np.full(40, 18), max_len=48)


@BOTH
@pytest.mark.parametrize("scores", ["flat", "rising", "falling"])
@pytest.mark.parametrize("sizes", ["rising", "falling"])
def test_ramps(Q, dt, scores, sizes):
    """Scores and values' sizes that rise or fall along a sequence by many times what a reference lets through."""
    print(f"ramps {dt} scores {scores} sizes {sizes}", flush=True)
    n, dim = 700, 64
    at = torch.linspace(0, 1, n)[:, None, None]
    k = normal((n, 1, dim), dt, 90, 0.2).float()
    k = k + {"flat": 0 * at, "rising": 5 * at, "falling": 5 - 5 * at}[scores]
    e = 14 * at - 7 if dt == "f16" else 60 * at - 30
    v = normal((n, 1, dim), dt, 92).float() * 2.0 ** (e if sizes == "rising" else -e)
    q = (normal((1, 5, dim), dt, 93).float() * 0.2 + 1.0).to(DT[dt])
    c, tables = cache_of(k.to(DT[dt]), v.to(DT[dt]), 32, dt, [n])
    check(Q, c, q, tables, np.array([n]), np.array([1]), scale=0.5)


@pytest.mark.parametrize("dt,size", [("f16", 2.0 ** -14), ("f16", 2.0 ** -9), ("f16", 300.0), ("f16", 1e4),
                                     ("bf16", 2.0 ** -60), ("bf16", 2.0 ** 60)])
def test_sizes(Q, dt, size):
    print(f"size {dt} {size}", flush=True)
    k, v = normal((400, 1, 128), dt, 100), (normal((400, 1, 128), dt, 102).float() * size).to(DT[dt])
    c, tables = cache_of(k, v, 64, dt, [400])
    check(Q, c, normal((1, 20, 128), dt, 103), tables, np.array([400]), np.array([1]))


# ---- flat groups: scales of 0 ----

@BOTH
@pytest.mark.parametrize("dim,gs", [(64, 32), (128, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("value", ["zero", "constant", "large"])
def test_flat_values(Q, dt, dim, gs, value):
    """V constant over each group: everywhere, in one token, in the first 32, in a run of parts."""
    print(f"flat {dt} D={dim} gs={gs} {value}", flush=True)
    level = {"zero": 0.0, "constant": 1.0, "large": 3e4 if dt == "f16" else 2.0 ** 24}[value]
    for n, flat in ((1, [(0, 1)]), (20, [(0, 20)]), (300, [(0, 300)]), (300, [(0, 32)]), (300, [(64, 128), (250, 300)]),
                    (1500, [(0, 128), (512, 1024)])):
        k, v = offset_keys(n, 1, dim, dt, 40), normal((n, 1, dim), dt, 42)
        for a, b in flat:
            v[a:b] = (level * normal((b - a, 1, dim // gs), dt, 43).float()).clamp(-6e4, 6e4 if dt == "f16" else 1e9).to(
                DT[dt]).repeat_interleave(gs, 2)
        c, tables = cache_of(k, v, gs, dt, [n])
        for heads in (3, 17):
            check(Q, c, normal((1, heads, dim), dt, 44), tables, np.array([n]), np.array([1]))


@BOTH
def test_flat_head_beside_others(Q, dt):
    """A kv head of zeros (padding) next to one that holds values; draft trees."""
    lens, new = np.array([90, 5]), np.array([5, 5])
    k, v = offset_keys(95, 2, 128, dt, 50), normal((95, 2, 128), dt, 52)
    k[:, 1], v[:, 1] = 0, 0
    c, tables = cache_of(k, v, 64, dt, lens)
    check(Q, c, normal((10, 4, 128), dt, 53), tables, lens, new, mask=np.array([1, 3, 5, 9, 17, 1, 2, 4, 8, 0]))


# ---- values of very different size ----

OUTLIERS = [("f16", 1e4), ("f16", 6e4), ("bf16", 1e6), ("bf16", 1e20), ("bf16", 1e30)]


@pytest.mark.parametrize("dt,size", OUTLIERS)
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("n", [20, 300])
def test_unseen_outlier_has_no_part(Q, dt, size, gs, n):
    """A finite draft token of any size: the rows that do not see it are bit for bit as if it were not."""
    print(f"unseen outlier {dt} {size} gs={gs} n={n}", flush=True)
    lens, new = np.array([n]), np.array([4])
    mask = np.array([0b1, 0b11, 0b101, 0b1000])  # the fourth sees the outlier, itself, alone among the new ones
    k, v, q = offset_keys(n, 1, 128, dt, 60), normal((n, 1, 128), dt, 62), normal((4, 10, 128), dt, 63)
    got = []
    for bad in (False, True):
        if bad:
            k[n - 1] = (k[n - 1].float() * 100).to(DT[dt])
            v[n - 1] = (torch.sign(v[n - 1].float()) * (0.5 + 0.5 * torch.rand(1, 128)) * size).to(DT[dt])
        c, tables = cache_of(k, v, gs, dt, lens)
        oracle = KO.attend_bound(c, 0, O.to_f64(synth.to_oracle(q), dt), tables, lens, [0, 4], 128 ** -0.5, mask)
        got.append((check(Q, c, q, tables, lens, new, mask=mask, oracle=oracle)[0], call(Q, c, q, tables, lens, new, mask)[1]))
    for a, b in zip(*got):
        assert torch.equal(a[:3].view(torch.uint8), b[:3].view(torch.uint8))


@pytest.mark.parametrize("dt,size", OUTLIERS)
@pytest.mark.parametrize("where", [0, 7, 200, 299])
def test_outlier_without_weight(Q, dt, size, where):
    """A token that all rows see with a weight of nothing: it takes no precision from the others."""
    print(f"weightless outlier {dt} {size} at {where}", flush=True)
    k, v = normal((300, 1, 128), dt, 70), normal((300, 1, 128), dt, 72)
    q = (normal((1, 6, 128), dt, 73).float() * 0.3 + 1.0).to(DT[dt])
    k[where] = -40.0  # scores near -450
    v[where] = (v[where].float() * size / 4).clamp(-size, size).to(DT[dt])
    c, tables = cache_of(k, v, 64, dt, [300])
    check(Q, c, q, tables, np.array([300]), np.array([1]))


@pytest.mark.parametrize("dt,big,small", [("f16", 1e4, 1e-2), ("f16", 1e4, 1.0), ("f16", 1.0, 2.0 ** -12),
                                          ("bf16", 1e10, 1e-10), ("bf16", 1e4, 1.0), ("bf16", 1.0, 1e-12)])
@pytest.mark.parametrize("dim,gs,heads", [(128, 32, 4), (128, 64, 20), (256, 32, 3)])
def test_groups_of_different_size(Q, dt, big, small, dim, gs, heads):
    """Every group keeps its own precision, over a long flat tail of weights too."""
    print(f"groups {dt} {big}/{small} D={dim} gs={gs} heads={heads}", flush=True)
    k, v, q = normal((900, 1, dim), dt, 80, 0.5), normal((900, 1, dim), dt, 82).float(), normal((1, heads, dim), dt, 83)
    v[..., :gs] *= big / 4
    v[..., gs:] *= small
    v[0] /= big / small  # the first tokens are smaller in all groups
    c, tables = cache_of(k, v.to(DT[dt]), gs, dt, [900])
    check(Q, c, q, tables, np.array([900]), np.array([1]))


@BOTH
@pytest.mark.parametrize("dim,gs", [(64, 32), (128, 32), (128, 64), (256, 32), (256, 64)])
def test_sizes_by_rows(Q, dt, dim, gs):
    """Workgroups by rows: a head of zeros, one of small values, one with a large group, an ordinary one; ragged rows."""
    print(f"sizes by rows {dt} D={dim} gs={gs}", flush=True)
    lens, new = np.array([40 + b % 9 for b in range(40)]), np.array([18 - b % 3 for b in range(40)])
    n = int(lens.sum())
    k, v = offset_keys(n, 4, dim, dt, 104), normal((n, 4, dim), dt, 106).float()
    v[:, 0] = 0
    v[:, 1] *= 2.0 ** -13
    v[:, 2, :gs] *= 2.0 ** 10
    c, tables = cache_of(k, v.to(DT[dt]), gs, dt, lens)
    check(Q, c, normal((int(new.sum()), 8, dim), dt, 107), tables, lens, new, max_len=48)


@BOTH
def test_sizes_beside_holes(Q, dt):
    """Steps without a page, before, between and after those of unusual size; cut into parts and not."""
    print(f"sizes beside holes {dt}", flush=True)
    n = 1500
    k, v = offset_keys(n, 1, 128, dt, 108), normal((n, 1, 128), dt, 109).float()
    v[200:700] *= 2.0 ** -14
    v[900:1000] = 0
    c, tables = cache_of(k, v.to(DT[dt]), 64, dt, [n])
    tables[0, [0, 4, 5, 12, 23]] = -1
    tables[0, 8] = 999
    q = normal((2, 10, 128), dt, 110)
    _, oracle = check(Q, c, q, tables, np.array([n]), np.array([2]))
    check(Q, c, q, tables, np.array([n]), np.array([2]), max_len=32, oracle=oracle)


# ---- the ends of the types' ranges ----

@pytest.mark.parametrize("size", [1e30, 1e36, 1e38])
@pytest.mark.parametrize("kind", ["flat", "spread", "one", "late"])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_values_near_the_largest(Q, size, kind, n):
    """bf16 values near its largest, that carry weight: sums of them are kept below fp32's."""
    print(f"near the largest {size} {kind} n={n}", flush=True)
    dt = "bf16"
    k, v = offset_keys(n, 1, 128, dt, 160), normal((n, 1, 128), dt, 162).float()
    top = (v / v.abs().max() * size).to(DT[dt]).float()
    if kind == "flat":
        v = top[..., :2].repeat_interleave(64, 2)
    elif kind == "spread":
        v = top
    elif kind == "one":
        v[n // 2] = top[n // 2]
    else:  # constant groups, of a size that comes after the first steps
        v = v[..., :2].repeat_interleave(64, 2)
        v[n // 2:] = top[n // 2:, :, :2].repeat_interleave(64, 2)
    c, tables = cache_of(k, v.to(DT[dt]), 64, dt, [n])
    check(Q, c, normal((1, 20, 128), dt, 163), tables, np.array([n]), np.array([1]))


@pytest.mark.parametrize("dt,size", [("f16", 3e3), ("f16", 6e4), ("bf16", 1e5), ("bf16", 1e12)])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_scores_beyond_whole_numbers(Q, dt, size, n):
    """Scores so large that fp32 holds no units of them: the largest, here far ahead, takes all."""
    print(f"large scores {dt} {size} n={n}", flush=True)
    k, v, q = normal((n, 1, 128), dt, 170), normal((n, 1, 128), dt, 171), normal((2, 10, 128), dt, 172)
    k, q = ((x.float() / x.float().abs().max() * size).to(DT[dt]) for x in (k, q))
    c, tables = cache_of(k, v, 64, dt, [n])
    q, mask = torch.cat([q, -q]), [0b1000] * 4  # the last token and those before the new ones
    got, lse = call(Q, c, q, tables, [n], [4], mask=mask)
    out, want, _, ltol = KO.attend_bound(c, 0, O.to_f64(synth.to_oracle(q), dt), tables, [n], [0, 4], 128 ** -0.5, mask)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    g = O.to_f64(synth.to_oracle(got), dt)
    tie = 2.0 ** -11 if dt == "f16" else 2.0 ** -8
    assert (np.abs(g - out) <= 2 * tie * np.abs(v.float().numpy()).max()).all()
    assert (np.abs(lse.cpu().numpy() - want) <= ltol).all()


# ---- offsets: the middles of the groups are large, their spread is small ----

@BOTH
@pytest.mark.parametrize("n,sharp", [(1, 1.0), (40, 1.0), (40, 30.0), (600, 1.0), (600, 6.0), (600, 30.0)])
def test_offset_values_of_narrow_groups(Q, dt, n, sharp):
    """The weights of the middles add up to what they are divided by, whatever the type rounds (one token that comes
    after the first of its part and takes almost all the weight; many alike)."""
    print(f"offset {dt} n={n} sharp={sharp}", flush=True)
    jitter = normal((n, 1, 128), "f16", 112).float()
    v = (normal((1, 1, 4), "f16", 113).float().repeat_interleave(32, 2) * 20 * (1 + 2.0 ** -9 * jitter)).to(DT[dt])
    c, tables = cache_of(offset_keys(n, 1, 128, dt, 110), v, 32, dt, [n])
    for heads in (5, 17):
        check(Q, c, normal((1, heads, 128), dt, 114), tables, np.array([n]), np.array([1]), scale=sharp / 128 ** 0.5)


@BOTH
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_offset_values_of_every_format(Q, dt, dim, gs):
    """As above, 8 tokens whose scores rise by a third of a power of two each."""
    print(f"offset {dt} D={dim} gs={gs}", flush=True)
    n, rise = 8, math.log(2) / 3
    v = (normal((1, 1, dim // gs), "f16", 115).float().repeat_interleave(gs, 2) * 20 *
         (1 + 2.0 ** -9 * normal((n, 1, dim), "f16", 116).float())).to(DT[dt])
    k = torch.full((n, 1, dim), 0.0)
    k[..., :gs] = torch.arange(n)[:, None, None] * rise * 16 / gs
    c, tables = cache_of(k.to(DT[dt]), v, gs, dt, [n])
    q = torch.full((1, 3, dim), 1.0)
    q[0, :, gs:] = 0
    q[0, 1] *= 0.75
    q[0, 2] *= 4.5
    check(Q, c, q.to(DT[dt]), tables, np.array([n]), np.array([1]), scale=1 / 16)


# ---- NaN ----

@BOTH
def test_lse_of_nan_scores(Q, dt):
    """NaN scores give NaN, not the -infinity of a row that sees nothing: one part, several, by rows."""
    for seqs, n, rows, heads in ((1, 50, 2, 2), (1, 3000, 2, 2), (2, 1000, 5, 8), (40, 40, 18, 8)):
        print(f"nan scores {dt} seqs={seqs} n={n} rows={rows}", flush=True)
        k, v = normal((seqs * n, 1, 64), dt, 120), normal((seqs * n, 1, 64), dt, 121)
        k[n // 2] = float("nan")  # the first sequence only; every row sees it
        page = 64
        width = -(-n // page)
        cache = Q.KVCache.empty(1, seqs * width, 1, 64, 64, page, DT[dt])
        tables, lens = i32(np.arange(seqs * width).reshape(seqs, width)), i32([n] * seqs)
        cache.append(0, k.cuda(), v.cuda(), tables, lens)
        q = normal((seqs * rows, heads, 64), dt, 122)
        if seqs > 1:
            q[rows, 0] = float("nan")  # a row of the second
        out, lse = cache.attend(0, q.cuda(), tables, lens, lse=True, max_len=n)
        nan = torch.zeros(seqs * rows, heads, dtype=torch.bool)
        nan[:rows] = True
        if seqs > 1:
            nan[rows, 0] = True
        assert torch.equal(torch.isnan(lse).cpu(), nan) and torch.isfinite(lse[~nan]).all()
        assert torch.equal(torch.isnan(out).all(-1).cpu(), nan) and torch.isfinite(out[~nan]).all()


@BOTH
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_one_nan_stays_a_nan(Q, dt, dim, gs):
    """A NaN among finite values: its group reads back as NaN, all else as without it, and attention shows it."""
    n, kv_heads = 70, 2
    k, v = normal((n, kv_heads, dim), dt, 130), normal((n, kv_heads, dim), dt, 131)
    rng = np.random.default_rng(132)
    places = {(int(rng.integers(n)), int(rng.integers(kv_heads)), d) for d in (0, 7, dim // 2 + 5, dim - 1)}
    tables, lens = i32([[1, 0]]), i32([n])
    pools, got = [], []
    for bad in (False, True):
        if bad:
            for t, h, d in places:
                v[t, h, d] = float("nan")
        cache = Q.KVCache(torch.zeros(1, 2, kv_heads, Q.record_words(dim, gs, 64, DT[dt]), dtype=torch.int32, device="cuda"),
                          dim, gs, 64, DT[dt])
        cache.append(0, k.cuda(), v.cuda(), tables, lens)
        got.append([x.cpu() for x in cache.read(0, n, tables, lens)])
        pools.append(cache)
    group = torch.zeros(n, kv_heads, dim, dtype=torch.bool)
    for t, h, d in places:
        group[t, h, d // gs * gs:d // gs * gs + gs] = True
    assert torch.equal(got[0][0], got[1][0])
    assert torch.isnan(got[1][1][group]).all() and torch.equal(got[0][1][~group], got[1][1][~group])
    q = normal((1, 4, dim), dt, 133).cuda()
    out = [c.attend(0, q, tables, lens).cpu() for c in pools]
    lost = group.any(0)[None].repeat_interleave(2, 1)
    assert torch.isnan(out[1][lost]).all()
    assert torch.equal(out[0][~lost].view(torch.int16), out[1][~lost].view(torch.int16))
    k[3, 0, 1] = float("nan")  # a key: every score of its head
    pools[0].append(0, k.cuda(), normal((n, kv_heads, dim), dt, 131).cuda(), tables, lens)
    out, lse = pools[0].attend(0, q, tables, lens, lse=True)
    assert torch.isnan(out[:, :2]).all() and torch.isnan(lse[:, :2]).all() and torch.isfinite(out[:, 2:]).all()


# ---- graphs ----

@BOTH
def test_graph_of_a_step_over_real_values(Q, dt):
    """append + attend captured once, replayed as the lengths grow, every position that is seen written before:
    finite, bit for bit the eager calls, and within the oracle's bound."""
    print(f"graph {dt}", flush=True)
    dim, gs, page, kv_heads, heads, n0 = 128, 64, 32, 2, 8, [1170, 45]
    k, v = offset_keys(sum(n0), kv_heads, dim, dt, 140), normal((sum(n0), kv_heads, dim), dt, 142)
    c = KO.new_cache(1, 48, kv_heads, dim, gs, page, dt, fill=0x7FFF7FFF)
    tables = np.full((2, 40), -1, np.int32)
    tables[0], tables[1, :8] = np.random.default_rng(4).permutation(40), np.arange(40, 48)
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, n0, [0, n0[0], sum(n0)])
    make = lambda: Q.KVCache(torch.from_numpy(c["pool"].view(np.int32).copy()).cuda(), dim, gs, page, DT[dt])
    captured, eager = make(), make()
    t, lens = i32(tables), i32([n + 1 for n in n0])
    q, kn, vn = (torch.zeros(2, h, dim, dtype=DT[dt], device="cuda") for h in (heads, kv_heads, kv_heads))
    out, lse = torch.zeros_like(q), torch.zeros(2, heads, device="cuda")
    ws = captured.attend_workspace(2, 1, 2, heads, 1280)
    step = lambda: (captured.append(0, kn, vn, t, lens),
                    captured.attend(0, q, t, lens, out=out, lse=lse, max_len=1280, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(12):
        new = np.array([n + 1 + r for n in n0])
        data = [normal(tuple(x.shape), dt, 150 + 3 * r + i) for i, x in enumerate((q, kn, vn))]
        for x, d in zip((q, kn, vn), data):
            x.copy_(d)
        lens.copy_(i32(new))
        g.replay()
        eager.append(0, kn, vn, t, lens)
        want, wlse = eager.attend(0, q, t, lens, lse=True, max_len=1280)
        torch.cuda.synchronize()
        assert torch.equal(captured.pool, eager.pool)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse), r
        KO.append(c, 0, synth.to_oracle(data[1]), synth.to_oracle(data[2]), tables, new, [0, 1, 2])
        if r % 5 == 0:
            o, ls, tol, ltol = KO.attend_bound(c, 0, O.to_f64(synth.to_oracle(data[0]), dt), tables, new, [0, 1, 2],
                                               dim ** -0.5)
            assert (np.abs(O.to_f64(synth.to_oracle(out), dt) - o) <= tol).all()
            assert (np.abs(lse.cpu().numpy() - ls) <= ltol).all()


def test_captured_calls_on_a_given_stream(Q):
    """attend(stream=s) while s is captured and another stream is current: cut into parts and not, against eager calls
    on that stream between the replays and after them."""
    dt = "bf16"
    for n in (60, 2500):
        print(f"captured stream n={n}", flush=True)
        c, tables = cache_of(offset_keys(n, 1, 128, dt, 200), normal((n, 1, 128), dt, 201), 64, dt, [n])
        cache = Q.KVCache(torch.from_numpy(c["pool"].view(np.int32).copy()).cuda(), 128, 64, 64, DT[dt])
        t, lens = i32(tables), i32([n])
        q, out = torch.zeros(1, 8, 128, dtype=DT[dt], device="cuda"), torch.zeros(1, 8, 128, dtype=DT[dt], device="cuda")
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.capture_begin()
            with torch.cuda.stream(torch.cuda.Stream()):
                cache.attend(0, q, t, lens, out=out, stream=s)
            g.capture_end()
        for r in range(4):
            q.copy_(normal(tuple(q.shape), dt, 202 + r))
            torch.cuda.synchronize()
            want = cache.attend(0, q, t, lens, stream=s)
            with torch.cuda.stream(s):
                g.replay()
            again = cache.attend(0, q, t, lens, stream=s)
            torch.cuda.synchronize()
            assert torch.isfinite(want).all() and torch.equal(want, again) and torch.equal(want, out), r
