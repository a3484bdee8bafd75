"""The gated block, rotary positions and log probabilities on the GPU against 64-bit plain forms, within bounds that follow
the kernels' roundings; their edges, strides, streams and graphs."""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import qmm_oracle as O
from oracle import rows_oracle as RO

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = [(dt, bits, gs) for dt in ("f16", "bf16") for bits in (4, 6, 8) for gs in (32, 64, 128)]


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import affine_quantized_gemm_amd as Q
    return Q


def f64(t, dt):
    return O.to_f64(synth.to_oracle(t), dt)


def within(got, want, tol, what=""):
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    print(f"  {what} worst err/bound {np.max(err / np.maximum(tol, 1e-300), initial=0):.3f}", flush=True)
    assert (err <= tol).all(), (what, (err / np.maximum(tol, 1e-300)).max())


# ---- gated block ----

def block(dt, bits, gs, rows, ffn, hidden, seed, std=1.0):
    w = synth.normal((2 * ffn, hidden), hidden ** -0.5, dt, seed, outlier_frac=0.01, outlier_scale=8.0)
    x = synth.normal((rows, hidden), std, dt, seed + 1)
    wq, sc, bi = O.quantize(synth.to_oracle(w), dt, bits, gs)
    gpu = tuple(synth.from_oracle(a, dt if a.dtype != np.uint32 else None).cuda() for a in (wq, sc, bi))
    return x, (wq, sc, bi), gpu


def check_gated(Q, dt, bits, gs, rows, ffn, hidden, seed, act="silu", std=1.0, back=False):
    print(f"gated {dt} {bits}-bit gs={gs} M={rows} F={ffn} K={hidden} {act}", flush=True)
    x, w, gpu = block(dt, bits, gs, rows, ffn, hidden, seed, std)
    h, tol = RO.gated(f64(x, dt), *w, dt, bits, gs, act)
    got = Q.gated(x.cuda(), *gpu, bits, gs, act=act)
    y = f64(got, dt)
    within(y, h, tol, "h")
    if h.size >= 64 and act != "relu":  # a rounding is at most UNIT of each value; what is before it is far below
        assert ((y - h) ** 2).mean() <= (1.05 * RO.UNIT[dt]) ** 2 * (h ** 2).mean() + 2.0 ** -50
    assert torch.equal(got, Q.gated(x.cuda(), *gpu, bits, gs, act=act))
    if back:
        grad = synth.normal((rows, ffn), 0.5, dt, seed + 2)
        dx, tx, d, td = RO.gated_backward(f64(x, dt), *w, dt, bits, gs, act, f64(grad, dt))
        gx, gd = Q.gated_backward(x.cuda(), *gpu, bits, gs, grad.cuda(), act=act)
        within(f64(gd, dt), d, td, "grad_gate_up")
        within(f64(gx, dt), dx, tx, "grad_x")
        if act != "relu":
            err = ((f64(gx, dt) - dx) ** 2).mean()
            assert err <= (1.1 * RO.UNIT[dt]) ** 2 * (dx ** 2).mean() + 2.0 ** -50
    return got


@pytest.mark.parametrize("dt,bits,gs", FORMATS)
def test_gated_formats(Q, dt, bits, gs):
    """Whole superblocks of K and others, one and several row tiles, columns that end inside a tile."""
    check_gated(Q, dt, bits, gs, 5, 33, 256, 1)
    check_gated(Q, dt, bits, gs, 1, 16, 128, 2)
    check_gated(Q, dt, bits, gs, 21, 47, 768, 3, back=False)
    check_gated(Q, dt, bits, gs, 64, 80, 512, 4, back=True)
    check_gated(Q, dt, bits, gs, 17, 48, 384, 5, back=True)


@pytest.mark.parametrize("rows", [1, 2, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_gated_rows(Q, rows):
    check_gated(Q, "bf16", 4, 64, rows, 96, 1024, 10, back=True)
    check_gated(Q, "f16", 8, 32, rows, 32, 320, 11)


@pytest.mark.parametrize("hidden", [64, 192, 256, 320, 512, 1280, 2048, 4096, 4352, 11008, 14336])
def test_gated_depths(Q, hidden):
    """From less than a superblock to several chunks of x, whole ones and not."""
    check_gated(Q, "f16", 4, 64, 6, 40, hidden, 20)
    check_gated(Q, "bf16", 6, 64, 40, 16, hidden, 21)
    check_gated(Q, "bf16", 4, 32, 16, 272, hidden, 22)


@pytest.mark.parametrize("ffn", [1, 15, 16, 17, 100, 1000, 4099])
def test_gated_widths(Q, ffn):
    check_gated(Q, "f16", 4, 64, 3, ffn, 256, 30)
    check_gated(Q, "bf16", 8, 128, 33, ffn, 256, 31)


def test_gated_many_tiles(Q):
    """More column tiles than workgroups: the weights of a workgroup's next tile are asked for in the one before."""
    check_gated(Q, "bf16", 4, 64, 4, 40000, 256, 32)
    check_gated(Q, "f16", 4, 128, 20, 70000, 128, 33)
    check_gated(Q, "f16", 8, 64, 40, 33000, 512, 34)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_activations(Q, act, dt):
    check_gated(Q, dt, 4, 64, 6, 64, 256, 40, act=act, back=True)
    check_gated(Q, dt, 8, 64, 6, 64, 256, 41, act=act, std=8.0, back=True)  # far into both tails
    check_gated(Q, dt, 8, 64, 6, 64, 256, 42, act=act, std=0.05, back=True)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_nan_in_the_gate(Q, act, dt):
    """One column's gate is NaN by its weights, the other product's is not: h is NaN there, and both gradients and grad_x."""
    x, _, (wq, sc, bi) = block(dt, 4, 64, 5, 32, 256, 43)
    sc = sc.clone()
    sc[9, 1] = math.nan
    grad = synth.normal((5, 32), 1.0, dt, 44).cuda()
    h = Q.gated(x.cuda(), wq, sc, bi, 4, 64, act=act)
    dx, d = Q.gated_backward(x.cuda(), wq, sc, bi, 4, 64, grad, act=act)
    at = torch.arange(32, device="cuda") == 9
    assert torch.isnan(h[:, at]).all() and torch.isfinite(h[:, ~at]).all()
    both = torch.cat([at, at])
    assert torch.isnan(d[:, both]).all() and torch.isfinite(d[:, ~both]).all() and torch.isnan(dx).all()


@pytest.mark.parametrize("rows,hidden", [(5, 256), (5, 192), (40, 512), (64, 320)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_rows_keep_to_themselves(Q, dt, rows, hidden):
    """A row of x or of the incoming gradient that is NaN or infinite has no part in the others, bit for bit."""
    x, _, gpu = block(dt, 4, 32, rows, 48, hidden, 45)
    x, grad = x.cuda(), synth.normal((rows, 48), 1.0, dt, 46).cuda()
    others = torch.arange(rows, device="cuda") != 3
    h, (dx, d) = Q.gated(x, *gpu, 4, 32), Q.gated_backward(x, *gpu, 4, 32, grad)
    for bad in (math.nan, math.inf):
        y, g = x.clone(), grad.clone()
        y[3, 7] = bad
        g[3, ::2] = bad
        assert torch.equal(Q.gated(y, *gpu, 4, 32)[others], h[others])
        for a, b in ((y, grad), (x, g)):
            ex, ed = Q.gated_backward(a, *gpu, 4, 32, b)
            assert torch.equal(ex[others], dx[others]) and torch.equal(ed[others], d[others])
            assert not torch.isfinite(ex[3]).any()


def test_gated_gradient_is_differences(Q):
    """grad_x of fp16 against differences of h itself, along random directions."""
    dt, rows, ffn, hidden = "f16", 4, 256, 512
    x, _, gpu = block(dt, 8, 64, rows, ffn, hidden, 50)
    g = np.random.default_rng(51)
    grad = torch.from_numpy(g.normal(size=(rows, ffn))).to(DT[dt])
    dx = f64(Q.gated_backward(x.cuda(), *gpu, 8, 64, grad.cuda())[0], dt)
    for k in range(4):
        step = torch.from_numpy(g.normal(size=(rows, hidden))) * 2.0 ** -4
        up, down = ((x.double() + s * step).to(DT[dt]) for s in (1, -1))
        real = (up.double() - down.double()).numpy()
        hu, hd = (f64(Q.gated(v.cuda(), *gpu, 8, 64), dt) for v in (up, down))
        got, want = (f64(grad, dt) * (hu - hd)).sum(), (dx * real).sum()
        # each h is rounded to 2^-11 of itself; the difference of third order is below 2^-8 of the change's size
        size = math.sqrt((f64(grad, dt) ** 2 * (hu ** 2 + hd ** 2)).sum()) * 2.0 ** -11 * 4
        assert abs(got - want) <= size + 2.0 ** -6 * np.linalg.norm(dx) * np.linalg.norm(real) / math.sqrt(rows * hidden) * 4, k


def test_gated_empty_and_out(Q):
    x, _, gpu = block("f16", 4, 64, 3, 32, 128, 60)
    assert Q.gated(x[:0].cuda(), *gpu, 4, 64).shape == (0, 32)
    dx, d = Q.gated_backward(x[:0].cuda(), *gpu, 4, 64, torch.empty(0, 32, dtype=torch.float16, device="cuda"))
    assert dx.shape == (0, 128) and d.shape == (0, 64)
    buffer = torch.full((4, 32), 7.0, dtype=torch.float16, device="cuda")
    y = Q.gated(x.cuda(), *gpu, 4, 64, out=buffer[:3])
    assert y.data_ptr() == buffer.data_ptr() and (buffer[3] == 7).all()
    none = tuple(t[:0].contiguous() for t in gpu)
    assert Q.gated(x.cuda(), *none, 4, 64).shape == (3, 0)
    dx, d = Q.gated_backward(x.cuda(), *none, 4, 64, torch.empty(3, 0, dtype=torch.float16, device="cuda"))
    assert d.shape == (3, 0) and not dx.any()
    for bad in (dict(act="tanh"), dict(out=buffer), dict(out=buffer[:3].bfloat16()), dict(out=torch.empty(3, 32, dtype=torch.float16))):
        with pytest.raises(ValueError):
            Q.gated(x.cuda(), *gpu, 4, 64, **bad)
    with pytest.raises(ValueError, match="contiguous"):
        Q.gated(torch.empty(128, 3, dtype=torch.float16, device="cuda").t(), *gpu, 4, 64)
    with pytest.raises(Q.QmmError):
        Q.gated(torch.empty(65, 128, dtype=torch.float16, device="cuda"), *gpu, 4, 64)
    with pytest.raises(ValueError, match="grad has shape"):
        Q.gated_backward(x.cuda(), *gpu, 4, 64, buffer)
    with pytest.raises(Q.QmmError):
        Q.gated_backward(x.cuda(), *gpu, 4, 64, buffer[:3], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_gated_equals_the_products(Q):
    """Beside small_m and torch: gate and up by the same weights, within what small_m rounds."""
    dt, bits, gs, hidden = "bf16", 4, 64, 1024
    x, w, gpu = block(dt, bits, gs, 6, 128, hidden, 61)
    both = f64(Q.small_m(x.cuda(), *gpu, bits, gs), dt)
    g, u = both[:, :128], both[:, 128:]
    want = RO.act("silu", g)[0] * u
    got = f64(Q.gated(x.cuda(), *gpu, bits, gs), dt)
    # small_m rounds a product to 2^-8 of itself, besides fp32 sums (RO.product's bound), and holds a group's sum of x, and
    # 128 times that against the scale, in two bf16 numbers: within 2^-16 of them
    _, e = RO.product(f64(x, dt), *w, dt, bits, gs)
    sums = np.abs(f64(x, dt).reshape(6, -1, gs).sum(2))
    e += 2.0 ** -16 * sums @ (np.abs(O.to_f64(w[2], dt)) + 128 * O.to_f64(w[1], dt)).T
    e += 2.0 ** -8 * (np.abs(both) + e)
    tol = 1.1 * e[:, :128] * (np.abs(u) + e[:, 128:]) + (np.abs(RO.act("silu", g)[0]) + 1.1 * e[:, :128]) * e[:, 128:]
    assert (np.abs(got - want) <= tol + RO.rounding(got, 0, dt) + 2.0 ** -20 * np.abs(want)).all()


# ---- rotary positions ----

def check_rotary(Q, dt, rows, heads, dim, sections, seed, pairs="halves", inverse=False, scale=1.0, far=10000, wide=True,
                 x=None, out=None):
    g = np.random.default_rng(seed)
    half = sum(sections)
    x = synth.normal((rows, heads, dim), 1.0, dt, seed).cuda() if x is None else x
    pos = g.integers(-far // 2, far, (len(sections), rows))
    freq = (10000.0 ** (-np.arange(half) / half)).astype(np.float32)
    before = x.clone()
    y, tol = RO.rotary(f64(x, dt), pos, freq, sections, pairs, inverse, scale, dt)
    p = torch.tensor(pos, dtype=torch.int64 if wide else torch.int32).cuda()
    if len(sections) == 1:
        p = p[0]
    got = Q.rotary(x, p, torch.from_numpy(freq).cuda(), sections=None if len(sections) == 1 else sections, pairs=pairs,
                   inverse=inverse, scale=scale, out=out)
    within(f64(got, dt), y, tol, f"{dt} {rows}x{heads}x{dim} {sections} {pairs}")
    if out is None or out.data_ptr() != x.data_ptr():
        assert torch.equal(x, before)
    return got


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("dim,sections", [(64, (32,)), (128, (16, 24, 24)), (80, (40,)), (256, (128,)), (128, (10, 6)),
                                          (96, (1, 0, 7, 8)), (16, (8,)), (1024, (500, 12)), (24, (8,))])
def test_rotary_layouts(Q, dt, pairs, dim, sections):
    check_rotary(Q, dt, 7, 3, dim, sections, 70, pairs)
    check_rotary(Q, dt, 1, 1, dim, sections, 71, pairs, inverse=True, scale=0.75, wide=False)
    check_rotary(Q, dt, 130, 5, dim, sections, 72, pairs, far=1 << 20)


@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 40), (3, 7), (33, 65), (300, 40), (5000, 3), (2, 200), (4100, 9)])
def test_rotary_sizes(Q, rows, heads):
    check_rotary(Q, "bf16", rows, heads, 64, (32,), 80)
    check_rotary(Q, "f16", rows, heads, 32, (8,), 81)


@pytest.mark.parametrize("far", [1 << 24, (1 << 31) - 1, 1 << 40])
def test_rotary_far_positions(Q, far):
    check_rotary(Q, "f16", 9, 2, 128, (64,), 82, far=far, wide=far > (1 << 31))


def test_rotary_strides_and_in_place(Q):
    """The q and k heads of one projection's output, turned where they are; what lies beside them stays."""
    dt, rows, heads, others, dim = "bf16", 37, 10, 4, 128
    whole = synth.normal((rows, heads + others, dim), 1.0, dt, 90).cuda()
    rest = whole[:, heads:].clone()
    x = whole[:, :heads]
    want = check_rotary(Q, dt, rows, heads, dim, (16, 24, 24), 91, x=x.clone())
    got = check_rotary(Q, dt, rows, heads, dim, (16, 24, 24), 91, x=x, out=x)
    assert torch.equal(got, want) and got.data_ptr() == whole.data_ptr() and torch.equal(whole[:, heads:], rest)
    # heads first in memory, as x and as out; one row for all
    t = synth.normal((heads, rows, dim), 1.0, dt, 92).cuda().transpose(0, 1)
    check_rotary(Q, dt, rows, heads, dim, (64,), 93, x=t, out=torch.empty(heads, rows, dim, dtype=DT[dt], device="cuda").transpose(0, 1))
    check_rotary(Q, dt, rows, heads, dim, (64,), 94, x=synth.normal((1, heads, dim), 1.0, dt, 95).cuda().expand(rows, heads, dim))
    assert Q.rotary(whole[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), torch.ones(64, device="cuda")).shape == (0, 14, 128)
    freq, pos = torch.ones(64, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    with pytest.raises(Q.QmmError):
        Q.rotary(x, pos, freq, out=torch.empty(1, heads, dim, dtype=DT[dt], device="cuda").expand(rows, heads, dim))
    with pytest.raises(Q.QmmError):
        Q.rotary(x, pos, torch.ones(65, device="cuda"))
    with pytest.raises(Q.QmmError):
        Q.rotary(torch.empty(rows, heads, 132, dtype=DT[dt], device="cuda")[..., 4:], pos, freq)
    with pytest.raises(ValueError, match="sections"):
        Q.rotary(x, pos[None].expand(2, rows).contiguous(), freq, sections=(30, 30))
    with pytest.raises(ValueError, match="pairs"):
        Q.rotary(x, pos, freq, pairs="both")
    with pytest.raises(ValueError, match="is on"):
        Q.rotary(x, pos.cpu(), freq)


def test_rotary_there_and_back(Q):
    """Turned back, within two roundings; the gradient's map is the transposed one."""
    dt, x = "f16", synth.normal((50, 4, 64), 1.0, "f16", 96).cuda()
    pos, freq = torch.arange(50, device="cuda") * 1000, 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    y = Q.rotary(Q.rotary(x, pos, freq), pos, freq, inverse=True)
    assert ((y - x).float().abs() <= 2.0 ** -10 * (x.float().abs() + x.float().abs().roll(32, -1)) + 1e-6).all()


# ---- log probabilities ----

def check_log_probs(Q, dt, z, tokens, top, scale=1.0, back=True, seed=0):
    """z: a GPU tensor [rows, vocab] of the type (any strides of rows)."""
    rows, vocab = z.shape
    print(f"log_probs {dt} {rows}x{vocab} top={top} scale={scale}", flush=True)
    zz = f64(z, dt)
    t = None if tokens is None else tokens.cpu().numpy()
    want = RO.log_probs(zz, t, top, scale)
    got = Q.log_probs(z, tokens, top=top, scale=scale)
    again = Q.log_probs(z, tokens, top=top, scale=scale)
    names = ["lse", "entropy"] + (["tokens"] if tokens is not None else []) + (["top_values"] if top else [])
    for n in names:
        a, b, tol = getattr(got, n).double().cpu().numpy(), want[n], want["tol_" + n] + 2.0 ** -23 * np.abs(np.where(np.isfinite(want[n]), want[n], 0))
        assert np.array_equal(np.isneginf(a), np.isneginf(b)), n
        live = np.isfinite(b)
        within(a[live], b[live], tol[live], n)
        assert torch.equal(getattr(got, n), getattr(again, n))
    if top:
        assert np.array_equal(got.top_ids.cpu().numpy(), want["top_ids"])
    if back:
        g = np.random.default_rng(seed)
        gt = None if tokens is None else g.normal(size=t.shape).astype(np.float32)
        gh, gl = (g.normal(size=rows).astype(np.float32) for _ in range(2))
        lse, h = got.lse.cpu().numpy().astype(np.float64), got.entropy.cpu().numpy().astype(np.float64)
        for use in ((gt, None, None), (gt, gh, gl), (None, gh, None)):
            if all(u is None for u in use):
                continue
            d, tol = RO.log_probs_backward(zz, t if use[0] is not None else None, lse, h, *use, scale, dt)
            cuda = [None if u is None else torch.from_numpy(u).cuda() for u in use]
            y = Q.log_probs_backward(z, tokens if use[0] is not None else None, got.lse, got.entropy, cuda[0],
                                     grad_entropy=cuda[1], grad_lse=cuda[2], scale=scale)
            within(f64(y, dt), d, tol, "gradient")
    return got


def logits(rows, vocab, dt, seed, barred=0.0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    z = std * torch.randn(rows, vocab, generator=g)
    z[torch.arange(rows), torch.randint(0, vocab, (rows,), generator=g)] += 9
    if barred:
        z[torch.rand(rows, vocab, generator=g) < barred] = -math.inf
    return z.to(DT[dt]).cuda()


def some_tokens(rows, vocab, n, seed, wide=True):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (rows, n) if n else (rows,), generator=g)
    t.view(rows, -1)[::3, 0] = -100
    if n > 1:
        t[:, 1] = t[:, 0]  # the same token twice
    return (t if wide else t.int()).cuda()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 100, 1000, 1023, 1024, 1025, 2055, 8192, 8200, 50257])
def test_log_probs_vocabularies(Q, dt, vocab):
    """Parts, slices and pieces that end anywhere; few rows and many."""
    for rows, n, top in ((1, 0, min(5, vocab)), (3, 2, min(64, vocab)), (40, 1, 0)):
        check_log_probs(Q, dt, logits(rows, vocab, dt, vocab + rows), some_tokens(rows, vocab, n, 5, wide=rows != 3), top)


@pytest.mark.parametrize("rows", [1, 6, 64, 300, 600, 1500])
def test_log_probs_rows(Q, rows):
    check_log_probs(Q, "bf16", logits(rows, 4099, "bf16", rows), some_tokens(rows, 4099, 1, 6), 3, scale=1.3)
    check_log_probs(Q, "f16", logits(rows, 3001, "f16", rows, barred=0.7), None, 20, scale=0.5)


def test_log_probs_whole_vocabulary(Q):
    check_log_probs(Q, "bf16", logits(6, 151936, "bf16", 1), some_tokens(6, 151936, 0, 7), 8)
    check_log_probs(Q, "f16", logits(2, 151941, "f16", 2, barred=0.5), some_tokens(2, 151941, 8, 8), 64)


@pytest.mark.parametrize("top", [1, 2, 5, 20, 33, 63, 64])
def test_log_probs_orders(Q, top):
    """Selections that work hardest: rising, falling, all alike, two values, the best in one lane, all but a few barred."""
    vocab = 9001
    g = torch.Generator().manual_seed(top)
    i = torch.arange(vocab)
    rows = [i * 2.0 ** -8, -i * 2.0 ** -8, torch.zeros(vocab), (i % 7 == 3).float(), torch.where(i % 512 < 8, 10.0 + i * 2.0 ** -9, 0.0),
            torch.where(i % 1000 == 999, 1.0, -math.inf), torch.where(i == 8999, 1.0, -math.inf), torch.randn(vocab, generator=g),
            torch.where(i % 2 == 0, 0.0, -0.0), torch.randint(-3, 3, (vocab,), generator=g).float(), -torch.rand(vocab, generator=g) * 1e4]
    for dt in ("f16", "bf16"):
        z = torch.stack(rows).to(DT[dt]).cuda()
        check_log_probs(Q, dt, z, None, top, back=False)
        many = z.repeat(100, 1)  # a workgroup a row
        a, b = Q.log_probs(many, top=top), Q.log_probs(z, top=top)
        assert torch.equal(a.top_ids.view(100, -1, top), b.top_ids.expand(100, -1, top))


def test_log_probs_special_rows(Q):
    """A row without any token, with NaN, with infinity; values at the type's ends; none has a part in its neighbours."""
    for dt in ("f16", "bf16"):
        big = 65504.0 if dt == "f16" else 1e30
        z = logits(8, 3000, dt, 3)
        clean = z.clone()
        z[1] = -math.inf
        z[2, 77] = math.nan
        z[3, 2999] = math.inf
        z[4, 5] = big
        z[5, ::2] = -big
        z[6] = z[6].abs() * 2.0 ** -14
        t = torch.full((8,), 5, device="cuda")
        keep = [0, 4, 5, 6, 7]
        r = Q.log_probs(z, t, top=4)
        for i in (2, 3):
            assert all(torch.isnan(v[i]).all() for v in r[:4]) and (r.top_ids[i] == -1).all()
        assert r.lse[1] == -math.inf and r.entropy[1] == 0 and r.tokens[1] == -math.inf and r.top_ids[1].tolist() == [0, 1, 2, 3]
        assert r.tokens[4] == 0 and r.entropy[4] == 0 and r.top_ids[4, 0] == 5
        check_log_probs(Q, dt, z[keep].contiguous(), t[keep].contiguous(), 4, scale=1.0)
        one = torch.ones(8, device="cuda")
        d = Q.log_probs_backward(z, t, r.lse, r.entropy, one, grad_entropy=one, grad_lse=one)
        assert not d[1].any() and torch.isnan(d[2]).all() and torch.isnan(d[3]).all() and torch.isfinite(d[keep]).all()
        c = Q.log_probs(clean, t, top=4)
        for i in (0, 7):
            assert all(torch.equal(a[i], b[i]) for a, b in zip(r, c))


@pytest.mark.parametrize("size", [1.0, 2.0 ** 28, 2.0 ** 60, 2.0 ** 100])
def test_log_probs_large_gradients_beside_barred_tokens(Q, size):
    """Barred tokens and ones far below the others have no gradient, however large (a loss's scale) the entropy's is."""
    z = logits(6, 1500, "bf16", 6, barred=0.3)
    z[0, 1:] = -math.inf
    z[1, 3:700] = -1e30
    r = Q.log_probs(z)
    g = np.random.default_rng(7)
    gh, gl = (torch.from_numpy(size * g.normal(size=6)).float().cuda() for _ in range(2))
    d, tol = RO.log_probs_backward(f64(z, "bf16"), None, r.lse.double().cpu().numpy(), r.entropy.double().cpu().numpy(), None,
                                   gh.double().cpu().numpy(), gl.double().cpu().numpy(), 1.0, "bf16")
    y = f64(Q.log_probs_backward(z, None, r.lse, r.entropy, None, grad_entropy=gh, grad_lse=gl), "bf16")
    within(y, d, tol, f"gradient of size {size:.0e}")
    assert not y[torch.isinf(z).cpu().numpy()].any()


@pytest.mark.parametrize("scale", [0.25, 2.0 ** -60, 2.0 ** -100, 2.0 ** 100])
def test_log_probs_of_the_largest_differences(Q, scale):
    """bf16 logits further apart than fp32's largest, whose scaled difference is not: finite log probabilities.  With the
    largest scale, the smallest logits."""
    size = 3e38 if scale < 1 else 2.0 ** -95
    z = size * torch.randn(5, 700, generator=torch.Generator().manual_seed(8)).clamp_(-1, 1)
    z[1] = -size
    z[1, 9] = size
    z[2, ::2] = -math.inf
    z = z.bfloat16().cuda()
    t = torch.arange(5, device="cuda") * 7 + 1
    got = check_log_probs(Q, "bf16", z, t, 64, scale=scale, back=False)
    assert torch.isfinite(got.tokens).all()


def test_log_probs_strides_and_alignment(Q):
    """Rows that begin anywhere, are spread out or one and the same; gradients into such rows, in place."""
    dt, vocab = "bf16", 2777
    wide = logits(9, 3100, dt, 4)
    t = some_tokens(9, vocab, 1, 9)
    for first in (0, 1, 3, 8, 13):
        check_log_probs(Q, dt, wide[:, first:first + vocab], t, 6)
    check_log_probs(Q, dt, wide[:1, :vocab].expand(9, vocab), t, 6)
    check_log_probs(Q, dt, wide[::2, 5:5 + vocab], t[:5], 6)
    r = Q.log_probs(wide[:, 1:1 + vocab], t)
    g = torch.rand(9, 1, device="cuda")
    want = Q.log_probs_backward(wide[:, 1:1 + vocab], t, r.lse, r.entropy, g)
    for first in (0, 1, 4):  # other alignments of the result
        out = torch.full((9, vocab + 8), 3.0, dtype=DT[dt], device="cuda")
        y = Q.log_probs_backward(wide[:, 1:1 + vocab], t, r.lse, r.entropy, g, out=out[:, first:first + vocab])
        assert torch.equal(y, want) and (out[:, :first] == 3).all() and (out[:, first + vocab:] == 3).all()
    place = wide.clone()
    y = Q.log_probs_backward(place[:, 1:1 + vocab], t, r.lse, r.entropy, g, out=place[:, 1:1 + vocab])
    assert torch.equal(y, want) and torch.equal(place[:, 0], wide[:, 0]) and torch.equal(place[:, 1 + vocab:], wide[:, 1 + vocab:])
    with pytest.raises(Q.QmmError):
        Q.log_probs_backward(wide, None, r.lse, r.entropy, None, grad_lse=r.lse, out=wide[:1].expand(9, 3100))


def test_log_probs_of_nothing(Q):
    r = Q.log_probs(torch.empty(0, 50, dtype=torch.float16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=3)
    assert r.lse.shape == (0,) and r.top_ids.shape == (0, 3) and r.tokens.shape == (0,)
    z = logits(4, 50, "f16", 5)
    r = Q.log_probs(z)
    assert r.tokens is None and r.top_ids is None
    r = Q.log_probs(z, torch.empty(4, 0, dtype=torch.int64, device="cuda"))
    assert r.tokens.shape == (4, 0)
    for bad in (dict(top=51), dict(top=65), dict(top=-1)):
        with pytest.raises(Q.QmmError):
            Q.log_probs(z, **bad)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(tokens=torch.zeros(3, dtype=torch.int64, device="cuda")),
                dict(tokens=torch.zeros(4, device="cuda")), dict(tokens=torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            Q.log_probs(z, **bad)
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="together"):
        Q.log_probs_backward(z, t, r.lse, r.entropy, None)
    with pytest.raises(ValueError, match="needs the entropy"):
        Q.log_probs_backward(z, None, r.lse, None, None, grad_entropy=r.lse)
    with pytest.raises(ValueError, match="lse"):
        Q.log_probs_backward(z, None, None, None, None)
    with pytest.raises(ValueError, match="dtype"):
        Q.log_probs_backward(z, None, r.lse.double(), None, None)


def test_log_probs_workspaces(Q):
    """One workspace for calls of many sizes; two streams with their own; every call leaves the counters zero."""
    cases = [(logits(r, v, "bf16", r), t) for r, v, t in ((1, 151936, 64), (6, 50000, 8), (300, 5000, 1), (2, 9000, 0), (500, 3000, 5))]
    want = [Q.log_probs(z, top=t) for z, t in cases]
    ws = Q.log_probs_workspace()
    for _ in range(2):
        for (z, t), w in zip(cases, want):
            r = Q.log_probs(z, top=t, workspace=ws)
            assert all(a is b or torch.equal(a, b) for a, b in zip(r, w))
    assert not ws[:65536].any()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (z, t), w in zip(cases, want):
            for s in (a, b):
                got.append((Q.log_probs(z, top=t, stream=s), w))
    torch.cuda.synchronize()
    for r, w in got:
        assert all(x is y or torch.equal(x, y) for x, y in zip(r, w))
    with pytest.raises(Q.QmmError):
        Q.log_probs(cases[0][0], workspace=ws[:1000])


# ---- together: streams, graphs ----

def step_of(Q, seed=0):
    """A block's rows as they go through a step: products, positions, gate, logits, and back."""
    dt = "bf16"
    x, _, gpu = block(dt, 4, 64, 6, 512, 256, 100 + seed)
    head = synth.normal((5000, 256), 0.06, dt, 101)
    hq = Q.quantize(head.cuda(), 4, 64)
    down = Q.quantize(synth.normal((256, 512), 0.05, dt, 102).cuda(), 4, 64)
    qkv = Q.quantize(synth.normal((6 * 64, 256), 0.06, dt, 103).cuda(), 4, 64)
    pos = torch.tensor([[5, 6, 7, 7, 8, 9], [1, 1, 2, 2, 3, 3]], device="cuda")
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    tokens = torch.tensor([1, 2, -100, 4, 4999, 5], device="cuda")
    x = x.cuda()

    def run():
        q = Q.rotary(Q.small_m(x, *qkv, 4, 64).view(6, 6, 64), pos, freq, sections=(20, 12))
        h = Q.gated(x, *gpu, 4, 64)
        z = Q.small_m(Q.small_m(h, *down, 4, 64), *hq, 4, 64)
        r = Q.log_probs(z, tokens, top=5)
        one = torch.ones(6, device="cuda")
        dz = Q.log_probs_backward(z, tokens, r.lse, r.entropy, one, grad_entropy=one)
        dh = Q.small_m_nt(Q.small_m_nt(dz[:, :4992].contiguous(), *(t[:4992] for t in hq), 4, 64), *down, 4, 64)
        dx, d = Q.gated_backward(x, *gpu, 4, 64, dh)
        return [q, h, z, *r, dz, dh, dx, d, Q.rotary(q, pos, freq, sections=(20, 12), inverse=True)]

    return run, x


def test_a_step_in_graphs(Q):
    """Two captured steps, replayed in turn with eager work between: every replay gives the eager results, bit for bit."""
    run, x = step_of(Q)
    first = x.clone()
    eager = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    other = synth.normal(tuple(x.shape), 1.0, "bf16", 99).cuda()
    x.copy_(other)
    eager2 = [t.clone() for t in run()]
    for k in range(6):
        use, want = ((first, eager), (other, eager2))[k % 2]
        x.copy_(use)
        for g, out in graphs:
            g.replay()
            run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_a_step_on_another_stream(Q):
    """Calls on a stream that is not the current one, given as such, beside the same calls on the current one."""
    run, x = step_of(Q, 1)
    want = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        with torch.cuda.stream(s):
            got.append(run())
        run()
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    z = want[2]
    s.wait_stream(torch.cuda.current_stream())
    r = Q.log_probs(z, None, top=3, stream=s)
    h = Q.gated(x, *block("bf16", 4, 64, 6, 512, 256, 101)[2], 4, 64, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r.top_ids, Q.log_probs(z, top=3).top_ids) and torch.equal(h, want[1])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_decoding_with_a_window(Q, dt):
    """The speculative decoder with a window and sinks in its layers: every token is the likeliest one of a plain pass over
    its text, and came with that pass's log probability.

    Both passes quantize keys and values that differ by roundings: the logits move by well under a tenth of their
    deviation (a neighbouring code moves a score by 0.4 / sqrt(128), and as much of one token's share of the sums).  A
    log probability, z - lse, moves by at most twice as much as the logits."""
    from affine_quantized_gemm_amd import spec_decode as S
    print(f"decoding with a window {dt}", flush=True)
    model = S.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=512, vocab=512, dtype=DT[dt],
                      window=48, sinks=4)
    s = S.Sequences(model, 3, 70 + 1 + 45 * 7, 3)
    prompt = torch.randint(0, 512, (70,), generator=torch.Generator().manual_seed(1)).cuda()
    s.fork(s.prefill(prompt)[-1])
    for _ in range(12):
        s.step()
    s.end([1])
    for _ in range(8):
        s.step()
    for text, said in zip(s.texts(), s.scores()):
        assert len(text) == len(said) > 71 + 20
        logits = S.logits_of(model, text[:-1]).float()
        far = 0.1 * logits.std(1)
        got = logits.gather(1, torch.tensor(text[1:], device="cuda")[:, None])[:, 0]
        assert (logits.amax(1) - got <= far)[70:].all()
        off = (got - logits.logsumexp(1) - torch.tensor(said[1:], device="cuda")).abs()
        assert (off <= 2 * far).all(), off.max()
        # the window is one: without it the same text has other logits
        whole = S.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, head_dim=128, ffn=512, vocab=512, dtype=DT[dt])
        assert torch.equal(S.logits_of(whole, text[:-1]).float()[:40], logits[:40])
        assert not torch.equal(S.logits_of(whole, text[:-1]).float()[60:], logits[60:])


@pytest.mark.parametrize("when", ["fork", "step"])
def test_decoding_of_nan_logits(Q, when):
    """A token picked from NaN: no text is given out, and no index is outside the vocabulary meanwhile."""
    from affine_quantized_gemm_amd import spec_decode as S
    print(f"decoding of NaN logits, {when}", flush=True)
    model = S.Decoder(layers=1, hidden=256, heads=2, kv_heads=1, head_dim=128, ffn=256, vocab=256)
    s = S.Sequences(model, 2, 20 + 1 + 8 * 7, 3)
    logits = s.prefill(torch.arange(20, device="cuda"))[-1]
    if when == "fork":
        logits = torch.full_like(logits, math.nan)
    s.fork(logits)
    if when == "step":
        s.step()
        assert all(len(t) >= 22 for t in s.texts())
        model.head[1][7] = math.nan  # one column of scales' values
    for _ in range(3):
        s.step()
        assert int(s.history.min()) >= 0 and int(s.history.max()) < 256
    with pytest.raises(AssertionError, match="NaN or infinite"):
        s.texts()


def test_gradient_of_no_columns_on_a_stream(Q):
    """A block without columns: grad_x is zero, in the order of the stream that was given."""
    x = torch.ones(3, 64, dtype=torch.float16, device="cuda")
    wq, s = torch.empty(0, 8, dtype=torch.int32, device="cuda"), torch.empty(0, 1, dtype=torch.float16, device="cuda")
    out = torch.full_like(x, 7.0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    dx, dgu = Q.gated_backward(x, wq, s, s.clone(), 4, 64, torch.empty(3, 0, dtype=torch.float16, device="cuda"), out=out, stream=stream)
    with torch.cuda.stream(stream):
        got = dx.clone()
    stream.synchronize()
    assert dx is out and dgu.shape == (3, 0) and not got.any()


@pytest.mark.parametrize("rows,hidden", [(1, 64), (5, 192), (64, 4096)])
def test_gradient_of_no_columns_from_c(Q, rows, hidden):
    """The C entry writes grad_x of a block without columns itself, and nothing beside it."""
    buffer = torch.full((rows + 1, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        status = Q._lib.qmm_gated_backward(1, 4, 64, 0, rows, 0, hidden, None, None, None, None, None, None, buffer.data_ptr(), None, 0,
                                           torch.cuda.current_stream().cuda_stream)
        assert status == Q.QMM_OK and not buffer[:rows].any() and (buffer[rows] == 7).all()


# ---- more rows than one launch holds (2^32 threads) ----

BEYOND = (1 << 32) // 256 + 700  # workgroups of 256


def test_log_probs_of_very_many_rows(Q):
    """Two logits a row: around the end of the first launch and at the last rows as in calls of those rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(BEYOND, 2, generator=g, device="cuda").bfloat16()
    t = torch.randint(-1, 3, (BEYOND,), generator=g, device="cuda")
    gt, gh, gl = (torch.randn(BEYOND, generator=g, device="cuda") for _ in range(3))
    print(f"log_probs {tuple(z.shape)}", flush=True)
    r = Q.log_probs(z, t, top=1)
    assert torch.equal(r.top_ids[:, 0], (z[:, 1] > z[:, 0]).long())
    assert torch.allclose(r.lse, z.float().logsumexp(1), rtol=1e-5, atol=1e-5)
    print("log_probs_backward", flush=True)
    d = Q.log_probs_backward(z, t, r.lse, r.entropy, gt, grad_entropy=gh, grad_lse=gl)
    for at in (slice(0, 1000), slice(BEYOND - 1500, BEYOND), slice(BEYOND // 2, BEYOND // 2 + 600)):
        s = Q.log_probs(z[at], t[at], top=1)
        assert all(torch.equal(a[at], b) for a, b in zip(r, s))
        assert torch.equal(d[at], Q.log_probs_backward(z[at], t[at], s.lse, s.entropy, gt[at], grad_entropy=gh[at], grad_lse=gl[at]))


def test_log_probs_gradient_of_very_many_workgroups(Q):
    """Rows of two workgroups, one row of logits for all, int32 tokens."""
    rows, vocab = BEYOND // 2 + 500, 4096
    z = logits(1, vocab, "bf16", 2).expand(rows, vocab)
    t = torch.randint(0, vocab, (rows, 2), dtype=torch.int32, device="cuda")
    lse = z[:1].float().logsumexp(1).expand(rows).contiguous()
    gt = torch.randn(rows, 2, device="cuda")
    print(f"log_probs_backward {tuple(z.shape)}", flush=True)
    d = Q.log_probs_backward(z, t, lse, None, gt)
    for at in (slice(0, 100), slice(rows - 1000, rows)):
        assert torch.equal(d[at], Q.log_probs_backward(z[at], t[at], lse[at], None, gt[at]))


def test_rotary_of_very_many_rows(Q):
    """A workgroup a row: 512 turned values of one head."""
    x = synth.normal((1, 1, 512), 1.0, "f16", 97).cuda().expand(BEYOND, 1, 512)
    pos = torch.randint(0, 1 << 20, (2, BEYOND), dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-torch.arange(256, device="cuda") / 256)
    print(f"rotary {tuple(x.shape)}", flush=True)
    y = Q.rotary(x, pos, freq, sections=(100, 156))
    for at in (slice(0, 100), slice(BEYOND - 1500, BEYOND)):
        assert torch.equal(y[at], Q.rotary(x[at], pos[:, at].contiguous(), freq, sections=(100, 156)))


# ---- the largest sizes that are taken ----

@pytest.mark.parametrize("dt,bits,gs", [("bf16", 8, 64), ("f16", 4, 32), ("bf16", 6, 64)])
@pytest.mark.parametrize("hidden", [1 << 24, (1 << 24) - 64 * 7])
def test_gated_of_the_longest_rows(Q, dt, bits, gs, hidden):
    """K of 2^24 and a little less (not of whole superblocks): rows of x that are zero but for a few places, so that products
    are sums of a few weights; and the gradient's columns at both ends."""
    rows, ffn = 64, 16
    print(f"gated {dt} {bits}-bit gs={gs} K={hidden}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    wq = torch.randint(-2 ** 31, 2 ** 31 - 1, (2 * ffn, hidden * bits // 32), dtype=torch.int32, device="cuda", generator=g)
    sc = (torch.rand(2 * ffn, hidden // gs, device="cuda", generator=g) / 2 ** bits).to(DT[dt])
    bi = (torch.rand(2 * ffn, hidden // gs, device="cuda", generator=g) - 0.5).to(DT[dt])
    places = torch.tensor([0, 63, 64, hidden // 2 + 5, hidden - 257, hidden - 64, hidden - 1], device="cuda")
    x = torch.zeros(rows, hidden, dtype=DT[dt], device="cuda")
    x[:, places] = torch.randn(rows, 7, device="cuda", generator=g).to(DT[dt])
    w = Q.dequantize(wq, sc, bi, bits, gs)[:, places].double()  # (rounded to the type: 2^-8 or 2^-11 of each)
    xs = x[:, places].double()
    y, size = xs @ w.T, xs.abs() @ w.abs().T
    gate, up = y[:, :ffn], y[:, ffn:]
    want = torch.nn.functional.silu(gate) * up
    # a weight's rounding, and fp32 sums of x (q + off) beside (b - off s) x: off s is at most 1024 * 2^-4 here
    e = RO.UNIT[dt] * size + 2.0 ** -20 * xs.abs().sum(1, keepdim=True) * 64
    tol = 1.2 * e[:, :ffn] * (up.abs() + e[:, ffn:]) + gate.abs() * e[:, ffn:] + 2 * RO.UNIT[dt] * want.abs() + 1e-6
    h = Q.gated(x, wq, sc, bi, bits, gs)
    assert ((h.double() - want).abs() <= tol).all()
    for few in (slice(0, 5), slice(17, 40)):
        assert ((Q.gated(x[few].contiguous(), wq, sc, bi, bits, gs).double() - want[few]).abs() <= tol[few]).all()
    del w
    grad = torch.randn(rows, ffn, device="cuda", generator=g).to(DT[dt])
    dx, d = Q.gated_backward(x, wq, sc, bi, bits, gs, grad)
    for at in (slice(0, 512), slice(hidden - 640, hidden)):
        words, gr = slice(at.start * bits // 32, at.stop * bits // 32), slice(at.start // gs, at.stop // gs)
        wd = Q.dequantize(wq[:, words].contiguous(), sc[:, gr].contiguous(), bi[:, gr].contiguous(), bits, gs).double()
        ref, size = d.double() @ wd, d.double().abs() @ wd.abs()
        assert ((dx[:, at].double() - ref).abs() <= 3 * RO.UNIT[dt] * size + 1e-6).all()


def test_gated_of_very_many_columns(Q):
    """40 million columns: offsets beyond 32 bits in the weights, the result and the gradients."""
    ffn, hidden, rows = 40000016, 64, 33
    g = torch.Generator(device="cuda").manual_seed(2)
    wq = torch.randint(-2 ** 31, 2 ** 31 - 1, (2 * ffn, 8), dtype=torch.int32, device="cuda", generator=g)
    sc = torch.rand(2 * ffn, 2, device="cuda", generator=g, dtype=torch.float32).div_(16).half()
    bi = torch.rand(2 * ffn, 2, device="cuda", generator=g, dtype=torch.float32).sub_(0.5).half()
    x = torch.randn(rows, hidden, device="cuda", generator=g).half()
    print(f"gated F={ffn}", flush=True)
    h = Q.gated(x, wq, sc, bi, 4, 32)
    grad = torch.randn(rows, ffn, device="cuda", generator=g, dtype=torch.float16)
    dx, d = Q.gated_backward(x, wq, sc, bi, 4, 32, grad)
    for c in (0, ffn // 2 + 8, ffn - 1008):
        at = torch.cat([torch.arange(c, c + 1008, device="cuda"), torch.arange(ffn + c, ffn + c + 1008, device="cuda")])
        some = tuple(t[at].contiguous() for t in (wq, sc, bi))
        # (another split of the same sums: within two roundings)
        few = Q.gated(x, *some, 4, 32)
        assert ((h[:, c:c + 1008] - few).float().abs() <= 2.0 ** -10 * few.float().abs() + 1e-4).all()
        few = Q.gated_backward(x, *some, 4, 32, grad[:, c:c + 1008].contiguous())[1]
        assert ((d[:, at] - few).float().abs() <= 2.0 ** -10 * few.float().abs() + 1e-4).all()
    # grad_x as the sum over pieces of the columns, in 64 bits
    ref, size = torch.zeros(rows, hidden, dtype=torch.float64, device="cuda"), torch.zeros(rows, hidden, dtype=torch.float64, device="cuda")
    step = 2500000
    for c in range(0, 2 * ffn, step):
        wd = Q.dequantize(wq[c:c + step], sc[c:c + step], bi[c:c + step], 4, 32).double()
        n = wd.shape[0] // 16  # (a long sum as 16 products)
        p, wd = d[:, c:c + step].double().view(rows, 16, n).transpose(0, 1).contiguous(), wd.view(16, n, hidden)
        ref, size = ref + (p @ wd).sum(0), size + (p.abs() @ wd.abs()).sum(0)
    # d and the weights are rounded here, each by another amount, and sums are in fp32
    assert ((dx.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -16 * size + 1e-3).all()


def test_log_probs_of_the_longest_rows(Q):
    """1.5 billion logits: columns beyond 2^30, sums of as many equal terms."""
    vocab = 1500000001
    z = torch.zeros(1, vocab, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([[0, vocab - 1, vocab, vocab // 2]], device="cuda")
    print(f"log_probs of {vocab}", flush=True)
    r = Q.log_probs(z, t, top=3)
    assert r.top_ids.tolist() == [[0, 1, 2]]
    for v in (r.lse, r.entropy, -r.tokens[0, 0], -r.tokens[0, 1], -r.top_values[0, 2]):
        assert abs(float(v) - math.log(vocab)) < 1e-4
    assert r.tokens[0, 2] == 0
    z.fill_(-math.inf)
    best = [vocab - 1, vocab - 2, 1 << 30, 12345]
    z[0, best] = torch.tensor([3.0, 2.0, 1.0, 0.0], dtype=torch.bfloat16, device="cuda")
    r = Q.log_probs(z, t, top=5)
    assert r.top_ids.tolist() == [[*best, 0]]
    want = torch.tensor([3.0, 2.0, 1.0, 0.0]).double().log_softmax(0)
    assert np.allclose(r.top_values[0, :4].cpu().numpy(), want.numpy(), atol=1e-6) and r.top_values[0, 4] == -math.inf
    assert abs(float(r.entropy) + float((want.exp() * want).sum())) < 1e-6
    d = Q.log_probs_backward(z, t, r.lse, r.entropy, torch.ones(1, 4, device="cuda"))
    assert d[0, vocab - 1].item() == pytest.approx(1 - 3 * math.exp(want[0]), rel=2.0 ** -8) and int((d != 0).sum()) == 6


def test_log_probs_of_64_tokens(Q):
    """As many given tokens as there may be, some of them the same, some padding; their gradient."""
    for dt, rows, vocab in (("f16", 3, 5000), ("bf16", 70, 777)):
        check_log_probs(Q, dt, logits(rows, vocab, dt, 9), some_tokens(rows, vocab, 64, 10), 64)
