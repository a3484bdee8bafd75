"""Measured cases of a decoder step's operators between the quantized products and the cache: the gated block and its
gradient, rotary positions, attention over a window of the 4-bit cache, log probabilities and their gradient.

``own`` False runs the operators in their plain form (elementary torch operations in 32 bits, angles in 64, one rounding
at the end); ``own`` True runs them through ``affine_quantized_gemm_amd``.

Quantized weights are [N, K*bits/32] int32 words, a little-endian bitstream of codes along K, with a scale and a bias per
group of gs codes: w = s q + b.  A gated block's are [2F, K], the gate's rows first.

The cache is an int32 pool [layers, pages, kv_heads, words]; one page of one layer and head holds PS tokens of D values as
4-bit codes, a scale and a bias per token and group of gs values (G = D / gs groups), in four parts:

  K codes  [PS][4][D/32] words       word (t, j, s): values d = 32 s + 8 j + e, value e in bits 4e..4e+3
  V codes  [PS/4][16][2][D/64] words word (u, i, p, c): token 4u + 2p in the low half and 4u + 2p + 1 in the
                                     high one, in each the values d = 64 c + 16 n + i, n = 0..3, in bits 4n..4n+3
  K scales [PS/4][G][2][4] 16-bit    (u, g): the scales of tokens 4u..4u+3, then their biases
  V scales as K's
"""

import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ----

def listed():
    return [
        # gated block.  Verify rows of a small decoder (the example's sizes): latency is all that counts.
        {"name": "gated 5 rows 1k", "op": "gated", "dt": "f16", "bits": 4, "gs": 64, "rows": 5, "hidden": 1024, "ffn": 2048,
         "act": "silu"},
        # verify step at full width: the weights' bytes
        {"name": "gated 6 rows 4k", "op": "gated", "dt": "bf16", "bits": 4, "gs": 64, "rows": 6, "hidden": 4096, "ffn": 14336,
         "act": "silu"},
        # the most rows a product takes, 64 users or a piece of a prompt, in 6 bits
        {"name": "gated 64 rows 4k 6-bit", "op": "gated", "dt": "f16", "bits": 6, "gs": 128, "rows": 64, "hidden": 4096,
         "ffn": 14336, "act": "gelu_tanh"},
        # its gradient, for tuning what lies before frozen weights (prompts, adapters): an odd number of rows
        {"name": "gated backward 37 rows 4k", "op": "gated_backward", "dt": "bf16", "bits": 4, "gs": 64, "rows": 37,
         "hidden": 4096, "ffn": 14336, "act": "silu"},
        # rotary positions.  Four users' draft trees of 7 rows, q and k heads together: latency.
        {"name": "rotary 28 rows", "op": "rotary", "dt": "bf16", "rows": 28, "heads": 40, "others": 8, "dim": 128, "turned": 128,
         "sections": "64", "far": 100000, "pairs": "halves", "inverse": False},
        # a prompt with images: time, height and width
        {"name": "rotary 8191 rows 3 axes", "op": "rotary", "dt": "f16", "rows": 8191, "heads": 40, "others": 8, "dim": 128,
         "turned": 128, "sections": "16 24 24", "far": 8191, "pairs": "halves", "inverse": False},
        # attention with a window.  One user's next token far into a document.
        {"name": "window one token 131071", "op": "window", "dt": "bf16", "batch": 1, "rows_lo": 1, "rows_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 128, "page": 128, "len_lo": 131071, "len_hi": 131071, "tree": False, "window": 4096,
         "sinks": 4},
        # verify rows of 16 users near 8k tokens, a window that begins inside a page
        {"name": "window verify 16 8k", "op": "window", "dt": "bf16", "batch": 16, "rows_lo": 4, "rows_hi": 6, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 7901, "len_hi": 8190, "tree": False, "window": 1023,
         "sinks": 4},
        # pieces of four prompts over what is cached before them
        {"name": "window 64 rows 16k", "op": "window", "dt": "f16", "batch": 4, "rows_lo": 64, "rows_hi": 64, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 15001, "len_hi": 16321, "tree": False, "window": 4096,
         "sinks": 64},
        # log probabilities.  A verify step's rows over a whole vocabulary, with the likeliest tokens.
        {"name": "log_probs 6 rows", "op": "log_probs", "dt": "bf16", "rows": 6, "vocab": 151936, "given": 1, "top": 8,
         "barred": False, "scale": 1.0},
        # prompts scored, some tokens barred by a grammar, a vocabulary whose rows begin anywhere
        {"name": "log_probs 1000 rows odd", "op": "log_probs", "dt": "f16", "rows": 1000, "vocab": 151941, "given": 1, "top": 20,
         "barred": True, "scale": 1.25},
        # the gradient of tokens' log probabilities and of the entropy, padding among the rows
        {"name": "log_probs backward 1000 rows", "op": "log_probs_backward", "dt": "bf16", "rows": 1000, "vocab": 151936,
         "given": 1, "top": 0, "barred": False, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "rotary", "rotary", "window", "window", "log_probs", "log_probs",
                     "log_probs_backward"])
    c = {"op": op, "dt": rng.choice(["f16", "bf16"])}
    if op in ("gated", "gated_backward"):
        c["bits"], c["gs"] = rng.choice([4, 4, 6, 8]), rng.choice([32, 64, 128])
        c["rows"] = rng.choice([1, rng.randint(1, 8), rng.randint(2, 64)])
        unit = max(64, c["gs"])
        c["hidden"] = unit * _log(rng, max(1, 256 // unit), 8192 // unit)
        c["ffn"] = _log(rng, 500, 2 ** 26 // c["hidden"] if c["hidden"] > 4096 else 14336)
        if op == "gated_backward":
            c["ffn"] = c["ffn"] // 16 * 16
        # at most the largest listed cases: 64 rows of 2 x 14336 x 4096, 37 of the gradient
        c["rows"] = max(1, min(c["rows"], (64 if op == "gated" else 37) * 14336 * 4096 // (c["hidden"] * c["ffn"])))
        c["act"] = rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"])
    elif op == "rotary":
        c["dim"] = rng.choice([64, 80, 128, 128, 256])
        c["turned"] = rng.choice([c["dim"], c["dim"], c["dim"] // 16 // 2 * 16])
        axes, half = rng.choice([1, 1, 2, 3]), c["turned"] // 2
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        c["sections"] = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half]))
        c["heads"], c["others"] = rng.randint(1, 48), rng.randint(0, 8)
        c["rows"] = _log(rng, 1, 8191 * 40 * 128 // (c["heads"] * c["dim"] * 2) + 1)
        c["far"] = _log(rng, 10, 1000000)
        c["pairs"], c["inverse"] = rng.choice(["halves", "halves", "adjacent"]), rng.random() < 0.3
    elif op == "window":
        c["dim"] = rng.choice([64, 128, 128, 256])
        c["gs"] = rng.choice([g for g in (32, 64, 128) if g <= c["dim"]])
        c["page"], c["kv_heads"] = rng.choice([32, 64, 64, 128, 256]), rng.choice([1, 2, 4, 5, 8, 16])
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        c["rows_hi"] = rng.choice([1, 1, rng.randint(2, 8), rng.randint(2, 64)])
        c["rows_lo"] = rng.randint(max(1, c["rows_hi"] // 2), c["rows_hi"])
        c["batch"] = _log(rng, 1, 32)
        c["sinks"] = rng.choice([0, 1, 4, 4, rng.randint(1, 200)])
        # at most the largest listed case: four windows of 4096 at 64 rows of 32 heads of 128
        most = int(min(4096, 4 * 4096 * 8 * 128 * 4 / (c["batch"] * c["kv_heads"] * c["dim"]),
                       4 * 4096 * 64 * 32 * 128 / (c["rows_hi"] * c["heads"] * c["dim"] * c["batch"])))
        c["window"] = _log(rng, 1, max(2, most - c["sinks"]))
        c["len_hi"] = max(c["rows_hi"], _log(rng, 16, max(17, min(131000, 260000 * 8 * 128 // (c["batch"] * c["kv_heads"] * c["dim"])))))
        c["len_lo"] = rng.randint(c["rows_hi"], c["len_hi"])
        c["tree"] = rng.random() < 0.3
    else:
        c["vocab"] = rng.choice([151936, _log(rng, 100, 200000), _log(rng, 1000, 200000)])
        c["rows"] = _log(rng, 1, 1000 * 151936 // max(c["vocab"], 16000))
        c["given"] = rng.choice([1, 1, rng.randint(2, 8)])
        c["top"] = 0 if op == "log_probs_backward" else rng.choice([0, 1, rng.randint(1, 20), rng.randint(1, 64)])
        c["barred"], c["scale"] = rng.random() < 0.3, rng.choice([1.0, 1.0, 0.5, 1.6])
    return c


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, both taken where n > 1, in a mixed order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    return [v[(i * step) % n] for i in range(n)] if math.gcd(step, n) == 1 else v


def _sections(c):
    """Pairs of each axis."""
    return [int(n) for n in c["sections"].split()]


def _rows_lens(c):
    """New tokens and lengths (the new ones counted in) of each sequence."""
    rows = _spread(c["rows_lo"], c["rows_hi"], c["batch"], 7)
    lens = [max(n, r) for n, r in zip(_spread(c["len_lo"], c["len_hi"], c["batch"], 5), rows)]
    return rows, lens


def work(case):
    c = case
    if c["op"] in ("gated", "gated_backward"):
        m, k, f = c["rows"], c["hidden"], c["ffn"]
        weights = 2 * f * (k * c["bits"] // 8 + 4 * k // c["gs"])
        product = 2 * m * 2 * f * k
        if c["op"] == "gated":
            return {"bytes": weights + 2 * m * (k + f), "flops": product}
        return {"bytes": weights + 2 * m * (k + f + k + 2 * f), "flops": 2 * product}
    if c["op"] == "rotary":
        return {"bytes": c["rows"] * (2 * 2 * c["heads"] * c["dim"] + 8 * len(_sections(c))),
                "flops": c["rows"] * c["heads"] * c["turned"] * 3}
    if c["op"] == "window":
        rows, lens = _rows_lens(c)
        held = [n - max(0, (n - r) - c["window"] + 1 - c["sinks"]) if n - r > c["window"] else n for r, n in zip(rows, lens)]
        kv = sum(held) * c["kv_heads"] * (c["dim"] + 8 * (c["dim"] // c["gs"]))
        pairs = sum(min(n - r + i + 1, c["window"] + c["sinks"]) for r, n in zip(rows, lens) for i in range(r))
        return {"bytes": kv + sum(rows) * c["heads"] * (4 * c["dim"] + 4), "flops": 4 * c["dim"] * c["heads"] * pairs}
    n = c["rows"] * c["vocab"]
    if c["op"] == "log_probs":
        return {"bytes": 2 * n + c["rows"] * (8 + 12 * (c["given"] + c["top"])), "flops": 4 * n}
    return {"bytes": 4 * n + c["rows"] * (12 + 12 * c["given"]), "flops": 6 * n}


# ---- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _words(g, *shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda").random_(-(1 << 31), (1 << 31) - 1, generator=g)


def _tree_masks(rows, g):
    """For each sequence a random draft tree: a row sees its own token and its ancestors'."""
    words = []
    r = np.random.RandomState(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    for n in rows:
        m = []
        for i in range(n):
            m.append((1 << i) | (m[r.randint(max(0, i - 4), i)] if i else 0))
        words += m
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def _prepare_gated(c, g, st):
    m, k, f, dt = c["rows"], c["hidden"], c["ffn"], DT[c["dt"]]
    st["wq"] = _words(g, 2 * f, k * c["bits"] // 32)
    # codes spread over their range: weights of deviation 1 / sqrt(hidden)
    step = math.sqrt(12 / k) / 2 ** c["bits"]
    st["scales"] = (step * (0.7 + 0.6 * torch.rand(2 * f, k // c["gs"], device="cuda", generator=g))).to(dt)
    middle = (2 ** c["bits"] - 1) / 2
    noise = 0.1 * torch.randn(st["scales"].shape, device="cuda", generator=g)
    st["biases"] = (-st["scales"].float() * middle + noise * k ** -0.5).to(dt)
    st["x"] = torch.randn(m, k, device="cuda", generator=g).to(dt)
    if c["op"] == "gated_backward":
        st["grad"] = (0.1 * torch.randn(m, f, device="cuda", generator=g)).to(dt)


def _prepare_rotary(c, g, st):
    rows, dt, axes = c["rows"], DT[c["dt"]], len(_sections(c))
    # q and k as the projection leaves them, v behind them
    st["sections"] = _sections(c)
    whole = torch.randn(rows, c["heads"] + c["others"], c["dim"], device="cuda", generator=g).to(dt)
    st["x"] = whole[:, :c["heads"]]
    st["freq"] = 10000.0 ** (-torch.arange(0, c["turned"], 2, device="cuda", dtype=torch.float32) / c["turned"])
    if axes == 1:
        st["pos"] = torch.randint(0, c["far"], (rows,), device="cuda", generator=g)
    else:  # rows of pictures between runs of text: time grows, the others go over a grid
        t = torch.arange(rows, device="cuda")
        side = max(2, int(math.sqrt(rows)) // 2)
        start = int(torch.randint(0, c["far"], (1,), device="cuda", generator=g))
        st["pos"] = torch.stack([start + t // (side * side), start + t // side % side, start + t % side][:axes])


def _prepare_window(c, g, st):
    rows, lens = _rows_lens(c)
    dim, h, hk, dt, ps, gs = c["dim"], c["heads"], c["kv_heads"], DT[c["dt"]], c["page"], c["gs"]
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)  # pages lie anywhere in the pool
    width = max(need)
    col = torch.arange(width, device="cuda")
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")[:, None]
    held = col < torch.tensor(need, device="cuda")[:, None]
    st["tables"] = torch.where(held, order[(first + col).clamp(max=pages - 1)], -1).int().contiguous()
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    st["ragged"], st["rows_hi"], st["len_hi"] = len(set(rows)) > 1, max(rows), max(lens)
    st["q"] = torch.randn(sum(rows), h + 2 * hk, dim, device="cuda", generator=g).to(dt)[:, :h]
    st["mask"] = _tree_masks(rows, g) if c["tree"] else None
    # codes spread over their range; K with offsets of its channels, V without
    code, sb = ps * dim // 8, ps * (dim // gs)
    pool = _words(g, 1, pages, hk, 2 * code + 2 * sb)
    off = 1.5 * torch.randn(hk, 1, dim // gs, 1, device="cuda", generator=g)
    for part in (0, 1):
        scale = 0.2 + 0.1 * torch.rand(pages, hk, ps // 4, dim // gs, 4, device="cuda", generator=g)
        bias = -7.5 * scale + (off if part == 0 else 0.0)
        both = torch.stack((scale, bias), -2).to(dt).contiguous()
        at = 2 * code + part * sb
        pool[0, :, :, at:at + sb] = both.view(torch.int32).flatten(2)
    st["pool"] = pool


def _prepare_log_probs(c, g, st):
    rows, vocab, dt = c["rows"], c["vocab"], DT[c["dt"]]
    logits = torch.empty(rows, vocab, dtype=dt, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for at in range(0, rows, step):  # (32-bit values of some rows at a time)
        part = 2.0 * torch.randn(min(step, rows - at), vocab, device="cuda", generator=g)
        # a few tokens stand out, as after a context
        ids = torch.randint(0, vocab, (part.shape[0], 8), device="cuda", generator=g)
        part.scatter_add_(1, ids, 4 + 8 * torch.rand(ids.shape, device="cuda", generator=g))
        if c["barred"]:
            part.masked_fill_(torch.rand(part.shape, device="cuda", generator=g) < 0.5, -torch.inf)
        logits[at:at + step] = part.to(dt)
    st["logits"] = logits
    tokens = torch.randint(0, vocab, (rows, c["given"]), device="cuda", generator=g)
    tokens[torch.rand(rows, device="cuda", generator=g) < 0.1] = -100  # padding
    st["tokens"] = tokens[:, 0].contiguous() if c["given"] == 1 else tokens
    if c["op"] == "log_probs_backward":
        z = c["scale"] * logits.double()
        st["lse"] = torch.logsumexp(z, -1)
        p = torch.exp(z - st["lse"][:, None])
        st["entropy"] = (st["lse"] - (p * z.clamp(min=-1e30)).sum(-1)).float()
        st["lse"] = st["lse"].float()
        st["g_tokens"] = -torch.rand(st["tokens"].shape, device="cuda", generator=g)
        st["g_entropy"] = 0.01 * torch.randn(rows, device="cuda", generator=g)


def prepare(case, seed):
    c = dict(case)
    st = {"c": c}
    makes = {"gated": _prepare_gated, "gated_backward": _prepare_gated, "rotary": _prepare_rotary, "window": _prepare_window,
             "log_probs": _prepare_log_probs, "log_probs_backward": _prepare_log_probs}
    makes[c["op"]](c, _gen(seed), st)
    if own and c["op"] == "window":
        from affine_quantized_gemm_amd import KVCache
        st["cache"] = KVCache(st["pool"], c["dim"], c["gs"], c["page"], DT[c["dt"]])
    return st


# ---- plain forms ----

def _weights(st):
    """[2F, K] in 32 bits."""
    c = st["c"]
    bits, gs = c["bits"], c["gs"]
    at = bits * torch.arange(c["hidden"], device="cuda")
    words = st["wq"].long() & 0xFFFFFFFF
    low, high = at // 32, (at // 32 + 1).clamp(max=words.shape[1] - 1)
    codes = ((words[:, low] >> at % 32) | (words[:, high] << (32 - at % 32))) & (2 ** bits - 1)
    w = codes.float().unflatten(-1, (-1, gs)) * st["scales"].float()[..., None] + st["biases"].float()[..., None]
    return w.flatten(-2)


def _act(a, name):
    """act(a) and act'(a)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-a))
        return a * s, s * (1 + a * (1 - s))
    if name == "relu":
        return torch.where(a > 0, a, 0.0), (a > 0).to(a.dtype)
    if name == "gelu":
        half = 0.5 * (1 + torch.erf(a * 0.5 ** 0.5))
        return a * half, half + a * torch.exp(-0.5 * a * a) * (2 * math.pi) ** -0.5
    t = torch.tanh((2 / math.pi) ** 0.5 * (a + 0.044715 * a * a * a))
    slope = (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * a * a)
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * slope


def _plain_gated(st):
    c, dt = st["c"], DT[st["c"]["dt"]]
    w, f = _weights(st), c["ffn"]
    both = torch.matmul(st["x"].float(), w.t())
    act, slope = _act(both[:, :f], c["act"])
    up = both[:, f:]
    if c["op"] == "gated":
        return {"h": (act * up).to(dt)}
    grad = st["grad"].float()
    both = torch.cat((grad * up * slope, grad * act), 1)
    return {"dx": torch.matmul(both, w).to(dt), "dgu": both.to(dt)}


def _plain_rotary(st):
    c, x = st["c"], st["x"].float()
    half, sections = c["turned"] // 2, st["sections"]
    axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), torch.tensor(sections, device="cuda"))
    pos = st["pos"].view(len(sections), -1)
    angle = pos[axis].t().double() * st["freq"].double()  # [rows, half]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["inverse"]:
        sin = -sin
    if c["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return {"y": torch.cat((turned, x[..., 2 * half:]), -1).to(DT[c["dt"]])}


def _tokens_of(c, pool, page, slot):
    """K and V [B, T, kv_heads, D] in 32 bits of the tokens at slots of pages [B, T]."""
    dim, ps, gs, dt = c["dim"], c["page"], c["gs"], DT[c["dt"]]
    code, sb = ps * dim // 8, ps * (dim // gs)
    page, slot = page[..., None, None], slot[..., None, None]
    head = torch.arange(c["kv_heads"], device="cuda")[:, None]
    nibble = torch.arange(8, device="cuda", dtype=torch.int32) * 4
    k = pool[page, head, slot * (dim // 8) + torch.arange(dim // 8, device="cuda")]  # (j, s)
    k = ((k[..., None] >> nibble) & 15).unflatten(-2, (4, dim // 32)).transpose(-3, -2).flatten(-3)
    c64 = dim // 64
    at = torch.arange(16 * c64, device="cuda")  # (i, c)
    v = pool[page, head, code + ((slot // 4 * 16 + at // c64) * 2 + slot % 4 // 2) * c64 + at % c64]
    v = v >> (16 * (slot % 2)).int()
    v = ((v[..., None] >> nibble[:4]) & 15).unflatten(-2, (16, c64)).permute(0, 1, 2, 4, 5, 3).flatten(-3)  # c, n, i
    halves = pool.view(dt)
    group = torch.arange(dim // gs, device="cuda")

    def values(codes, first):
        place = 2 * first + (slot // 4 * (dim // gs) + group) * 8 + slot % 4
        s, b = halves[page, head, place].float(), halves[page, head, place + 4].float()
        return (codes.float().unflatten(-1, (-1, gs)) * s[..., None] + b[..., None]).flatten(-2)

    return values(k, 2 * code), values(v, 2 * code + sb)


def _plain_window(st):
    c = st["c"]
    dim, h, hk, window, sinks, m = c["dim"], c["heads"], c["kv_heads"], c["window"], c["sinks"], st["rows_hi"]
    batch, lens, starts = c["batch"], st["lens"].long(), st["starts"].long()
    new = starts[1:] - starts[:-1]
    before = lens - new
    # the tokens that some row may see: the sinks, and from the first window's begin to the end
    low = (before - window).clamp(min=0)
    t = torch.arange(sinks + min(window + m, st["len_hi"]), device="cuda")
    pos = torch.where(t < sinks, t, low[:, None].clamp(min=sinks) + t - sinks)
    there = pos < lens[:, None]
    pos = torch.where(there, pos, 0)
    page = st["tables"].gather(1, pos // c["page"]).long()
    k, v = _tokens_of(c, st["pool"][0], page, pos % c["page"])
    row = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(starts, row, right=True) - 1
    i = row - starts[b]
    q = torch.zeros(batch, m, h, dim, device="cuda")
    q[b, i] = st["q"].float()
    q = q.view(batch, m, hk, h // hk, dim).permute(0, 2, 1, 3, 4).reshape(batch, hk, -1, dim)
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) / math.sqrt(dim)
    # what the rows see of the new tokens; a row's window ends with the last of them
    bits = torch.zeros(batch, m, dtype=torch.int64, device="cuda")
    bits[b, i] = st["mask"] if st["mask"] is not None else torch.where(i == 63, -1, (2 << i.clamp(max=62)) - 1)
    sees = ((bits[..., None] >> torch.arange(64, device="cuda")) & 1 == 1)  # [B, m, 64]
    after = sees.flip(-1).cumsum(-1).flip(-1)  # seen ones from here on
    sees_new = sees & (after <= window)
    j = pos - before[:, None]  # place among the new tokens
    jj = j.clamp(0, 63)[:, None].expand(batch, m, -1)
    cached = (j < 0)[:, None] & (pos[:, None] >= (before[:, None] - window + after[..., 0])[..., None])
    fresh = (j >= 0)[:, None] & sees_new.gather(2, jj)
    first = (pos < sinks)[:, None] & ((j < 0)[:, None] | sees.gather(2, jj))
    allowed = (cached | fresh | first) & there[:, None]
    allowed = allowed[:, None, :, None].expand(batch, hk, m, h // hk, -1).reshape(batch, hk, m * (h // hk), -1)
    s = torch.where(allowed, s, -torch.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(p, v.transpose(1, 2).contiguous()) / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.view(batch, hk, m, h // hk, dim).permute(0, 2, 1, 3, 4).reshape(batch, m, h, dim)
    lse = lse.view(batch, hk, m, h // hk).permute(0, 2, 1, 3).reshape(batch, m, h)
    return {"out": o[b, i].to(DT[c["dt"]]), "lse": lse[b, i]}


def _plain_log_probs(st):
    c, logits = st["c"], st["logits"]
    vocab = c["vocab"]
    z = c["scale"] * logits.float()
    top = z.amax(-1, keepdim=True)
    z -= top
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    entropy = (log_total - (e * z.clamp(min=-1e30)).sum(-1, keepdim=True) / total)[:, 0]
    tokens = st["tokens"].view(c["rows"], -1)
    given = tokens >= 0
    lp = torch.where(given, z.gather(1, tokens.clamp(min=0)) - log_total, 0.0).view(st["tokens"].shape)
    out = {"lse": (top + log_total)[:, 0], "entropy": entropy, "tokens": lp}
    if c["top"]:
        # a value's order in the high half of a key, the lowest id first in the low one
        bits = (logits + 0.0).view(torch.int16).long()
        keys = torch.where(bits < 0, ~bits & 0x7FFF | -0x8000, bits) << 32
        keys = keys | (vocab - 1 - torch.arange(vocab, device="cuda"))
        keys = torch.topk(keys, min(c["top"], vocab), sorted=True).values
        ids = vocab - 1 - (keys & 0xFFFFFFFF)
        out["top_values"], out["top_ids"] = z.gather(1, ids) - log_total, ids
    return out


def _plain_log_probs_backward(st):
    c = st["c"]
    lp = c["scale"] * st["logits"].float() - st["lse"][:, None]
    p = torch.exp(lp)
    tokens = st["tokens"].view(c["rows"], -1)
    g = torch.where(tokens >= 0, st["g_tokens"].view(tokens.shape), 0.0)
    d = -p * (g.sum(-1, keepdim=True) + st["g_entropy"][:, None] * (lp.clamp(min=-1e30) + st["entropy"][:, None]))
    d.scatter_add_(1, tokens.clamp(min=0), g)
    return {"d": (c["scale"] * d).to(DT[c["dt"]])}


def run(state):
    st = state
    c = st["c"]
    op = c["op"]
    if not own:
        if op in ("gated", "gated_backward"):
            return _plain_gated(st)
        if op == "rotary":
            return _plain_rotary(st)
        if op == "window":
            return _plain_window(st)
        return _plain_log_probs(st) if op == "log_probs" else _plain_log_probs_backward(st)
    import affine_quantized_gemm_amd as Q
    if op == "gated":
        return {"h": Q.gated(st["x"], st["wq"], st["scales"], st["biases"], c["bits"], c["gs"], act=c["act"])}
    if op == "gated_backward":
        dx, dgu = Q.gated_backward(st["x"], st["wq"], st["scales"], st["biases"], c["bits"], c["gs"], st["grad"], act=c["act"])
        return {"dx": dx, "dgu": dgu}
    if op == "rotary":
        return {"y": Q.rotary(st["x"], st["pos"], st["freq"], sections=st["sections"], pairs=c["pairs"], inverse=c["inverse"])}
    if op == "window":
        ragged = {"starts": st["starts"], "max_new": st["rows_hi"]} if st["ragged"] else {}
        out, lse = st["cache"].attend(0, st["q"], st["tables"], st["lens"], mask=st["mask"], max_len=st["len_hi"], lse=True,
                                      window=c["window"], sinks=c["sinks"], **ragged)
        return {"out": out, "lse": lse}
    if op == "log_probs":
        r = Q.log_probs(st["logits"], st["tokens"], top=min(c["top"], c["vocab"]), scale=c["scale"])
        out = {"lse": r.lse, "entropy": r.entropy, "tokens": r.tokens}
        if c["top"]:
            out["top_values"], out["top_ids"] = r.top_values, r.top_ids
        return out
    return {"d": Q.log_probs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"], st["g_tokens"],
                                      grad_entropy=st["g_entropy"], scale=c["scale"])}


# ---- in 64 bits ----

def _exact_weights(st):
    c = st["c"]
    n, k, bits = 2 * c["ffn"], c["hidden"], c["bits"]
    byte = st["wq"].view(torch.uint8)
    if bits == 8:
        q = byte
    elif bits == 4:
        q = torch.stack((byte % 16, byte // 16), -1)
    else:  # four codes in three bytes
        a, b, d = byte.view(n, -1, 3).int().unbind(-1)
        q = torch.stack((a % 64, a // 64 + b % 16 * 4, b // 16 + d % 4 * 16, d // 4), -1)
    q = q.reshape(n, k).double()
    wide = lambda t: t.double().repeat_interleave(c["gs"], 1)
    return q * wide(st["scales"]) + wide(st["biases"])


def _exact_gated(st):
    c, f = st["c"], st["c"]["ffn"]
    w, x = _exact_weights(st), st["x"].double()
    gate, up = x @ w[:f].t(), x @ w[f:].t()
    if c["act"] == "silu":
        act = gate * torch.sigmoid(gate)
        slope = torch.sigmoid(gate) + act * torch.sigmoid(-gate)
    elif c["act"] == "relu":
        act, slope = gate.clamp(min=0), torch.heaviside(gate, torch.zeros_like(gate))
    elif c["act"] == "gelu":
        phi = torch.special.ndtr(gate)
        act, slope = gate * phi, phi + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
    else:  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
        r = math.sqrt(8 / math.pi)
        s = torch.sigmoid(r * (gate + 0.044715 * gate ** 3))
        act, slope = gate * s, s + gate * s * (1 - s) * r * (1 + 0.134145 * gate ** 2)
    if c["op"] == "gated":
        return {"h": act * up}
    d = st["grad"].double()
    dg, du = d * up * slope, d * act
    return {"dx": dg @ w[:f] + du @ w[f:], "dgu": torch.cat((dg, du), 1)}


def _exact_rotary(st):
    c = st["c"]
    x = st["x"].double().cpu().numpy()
    half = c["turned"] // 2
    pos = st["pos"].cpu().numpy().reshape(len(_sections(c)), -1).astype(np.float64)
    freq = st["freq"].cpu().numpy().astype(np.float64)
    angle = np.empty((x.shape[0], half))
    at = 0
    for axis, n in enumerate(_sections(c)):
        angle[:, at:at + n] = pos[axis][:, None] * freq[at:at + n]
        at += n
    turn = np.exp((-1j if c["inverse"] else 1j) * angle)[:, None]
    y = x.copy()
    if c["pairs"] == "halves":
        z = (x[..., :half] + 1j * x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    else:
        z = (x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    return {"y": torch.from_numpy(y)}


def _exact_window(st):
    c = st["c"]
    dim, gs, ps, hk, dt = c["dim"], c["gs"], c["page"], c["kv_heads"], DT[c["dt"]]
    share, code, sb = c["heads"] // hk, ps * dim // 8, ps * (dim // gs)
    d = torch.arange(dim, device="cuda")
    outs, sums = [], []
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    masks = None if st["mask"] is None else st["mask"].tolist()
    for b in range(c["batch"]):
        n, r0, r1 = lens[b], starts[b], starts[b + 1]
        before = n - (r1 - r0)
        t = torch.arange(n, device="cuda")
        t = t[(t < c["sinks"]) | (t >= before - c["window"])]
        rec, slot = st["pool"][0][st["tables"][b].long()[t // ps]], t % ps  # [T, hk, words]
        at = torch.arange(t.numel(), device="cuda")[:, None]
        kw = rec[at, :, (slot[:, None] * 4 + d % 32 // 8) * (dim // 32) + d // 32].long()  # [T, D, hk]
        vw = rec[at, :, code + ((slot[:, None] // 4 * 16 + d % 16) * 2 + slot[:, None] % 4 // 2) * (dim // 64) + d // 64].long()
        kq = (kw >> (4 * (d % 8))[:, None]) % 16
        vq = (vw >> (16 * (slot % 2)[:, None] + 4 * (d % 64 // 16))[..., None]) % 16
        halves = rec.view(dt)
        place = (slot[:, None] // 4 * (dim // gs) + d // gs) * 8 + slot[:, None] % 4
        get = lambda first, more: halves[at, :, 2 * first + place + more].double()
        k = kq * get(2 * code, 0) + get(2 * code, 4)
        v = vq * get(2 * code + sb, 0) + get(2 * code + sb, 4)
        for r in range(r0, r1):
            word = (1 << (r - r0 + 1)) - 1 if masks is None else masks[r]
            seen = [before + j for j in range(r1 - r0) if word >> j & 1]
            last = seen[-c["window"]:]
            low = before - (c["window"] - len(last))
            ok = ((t < before) & ((t >= low) | (t < c["sinks"])))
            ok |= torch.isin(t, torch.tensor(last + [p for p in seen if p < c["sinks"]], device="cuda"))
            q = st["q"][r].double().view(hk, share, dim)
            s = torch.matmul(q, k[ok].permute(2, 1, 0)) / math.sqrt(dim)
            outs.append(torch.matmul(torch.softmax(s, -1), v[ok].permute(2, 0, 1)).reshape(c["heads"], dim))
            sums.append(torch.logsumexp(s, -1).reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(sums)}


def _exact_log_probs(st):
    c = st["c"]
    rows, back = c["rows"], c["op"] == "log_probs_backward"
    found = []
    step = max(1, (1 << 27) // c["vocab"])
    for at in range(0, rows, step):
        logits = st["logits"][at:at + step]
        tokens = st["tokens"][at:at + step].view(logits.shape[0], -1)
        pad = tokens < 0
        lp = torch.log_softmax(c["scale"] * logits.double(), -1)
        if back:
            # d/dz of sum_n g_n lp[t_n] + g_H H, with the given logarithms of sums and entropies
            lp = c["scale"] * logits.double() - st["lse"][at:at + step, None].double()
            p = torch.exp(lp)
            g = st["g_tokens"][at:at + step].view(tokens.shape).double().masked_fill(pad, 0)
            d = torch.zeros_like(p).scatter_add_(1, tokens.masked_fill(pad, 0), g) - p * g.sum(1, keepdim=True)
            h = st["entropy"][at:at + step, None].double()
            d -= st["g_entropy"][at:at + step, None].double() * torch.where(p > 0, p * (lp + h), 0.0)
            found.append({"d": (c["scale"] * d).cpu()})
            continue
        r = {"lse": torch.logsumexp(c["scale"] * logits.double(), -1), "entropy": torch.special.entr(torch.exp(lp)).sum(-1),
             "tokens": lp.gather(1, tokens.masked_fill(pad, 0)).masked_fill(pad, 0).view(st["tokens"][at:at + step].shape)}
        if c["top"]:
            order = torch.sort(logits.double(), dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            r["top_values"], r["top_ids"] = lp.gather(1, order), order
        found.append({k: v.cpu() for k, v in r.items()})
    return {k: torch.cat([f[k] for f in found]) for k in found[0]}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "gated_backward"):
        return _exact_gated(st)
    if op == "rotary":
        return _exact_rotary(st)
    return _exact_window(st) if op == "window" else _exact_log_probs(st)
