"""Measured cases of the 4-bit paged K/V cache: appending to it, attending over it, moving its pages.

``own`` False runs the operators in their plain form (elementary torch operations in 32 bits, one rounding at
the end); ``own`` True runs them through ``affine_quantized_gemm_amd.KVCache``.

The cache is an int32 pool [layers, pages, kv_heads, words].  One page of one layer and head holds PS tokens of
D values as 4-bit affine codes, one scale and one bias per token and group of gs consecutive values
(G = D / gs groups), in four parts:

  K codes  [PS][4][D/32] words       word (t, j, s): values d = 32 s + 8 j + e, value e in bits 4e..4e+3
  V codes  [PS/4][16][2][D/64] words word (u, i, p, c): token 4u + 2p in the low half and 4u + 2p + 1 in the
                                     high one, in each the values d = 64 c + 16 n + i, n = 0..3, in bits 4n..4n+3
  K scales [PS/4][G][2][4] 16-bit    (u, g): the scales of tokens 4u..4u+3, then their biases
  V scales as K's

Quantization is the weights': lo = min, hi = max of a group, s = fp32 (hi - lo) / 15 rounded up to the type,
b = lo, q = clamp(rint(fp32 (x - b) / s), 0, 15), 0 where s is 0.
"""

import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ----

def listed():
    return [
        # attention.  One user's next token, short context: latency is all that counts.
        {"name": "attend one token 777", "op": "attend", "dt": "bf16", "batch": 1, "rows_lo": 1, "rows_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 777, "len_hi": 777, "tree": False},
        # batched decode: 32 users between 1k and 4k tokens, one row each
        {"name": "attend 32 tokens 1k-4k", "op": "attend", "dt": "f16", "batch": 32, "rows_lo": 1, "rows_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 1021, "len_hi": 4093, "tree": False},
        # verify step of speculative decoding: 4 to 6 rows for each of 16 users near 8k tokens
        {"name": "attend verify 16 8k", "op": "attend", "dt": "bf16", "batch": 16, "rows_lo": 4, "rows_hi": 6, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 7901, "len_hi": 8190, "tree": False},
        # verify of a draft tree, no shared heads, narrow heads and fine groups, some users just started
        {"name": "attend tree 8 to 2k", "op": "attend", "dt": "f16", "batch": 8, "rows_lo": 13, "rows_hi": 13, "heads": 16,
         "kv_heads": 16, "dim": 64, "gs": 32, "page": 32, "len_lo": 13, "len_hi": 2003, "tree": True},
        # one user with a long document: the work has to be split over the tokens
        {"name": "attend one token 131071", "op": "attend", "dt": "bf16", "batch": 1, "rows_lo": 1, "rows_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 128, "page": 128, "len_lo": 131071, "len_hi": 131071, "tree": False},
        # 64 rows a user, the most the products take: a piece of a prompt over what is cached before it
        {"name": "attend 64 rows 16k", "op": "attend", "dt": "f16", "batch": 4, "rows_lo": 64, "rows_hi": 64, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 15001, "len_hi": 16321, "tree": False},
        # appending.  One token for each of 64 users.
        {"name": "append 64 tokens", "op": "append", "dt": "bf16", "batch": 64, "rows_lo": 1, "rows_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 512, "len_hi": 1500},
        # verify rows of wide heads, ragged, ends inside pages
        {"name": "append verify 16 wide", "op": "append", "dt": "bf16", "batch": 16, "rows_lo": 4, "rows_hi": 6, "heads": 16,
         "kv_heads": 4, "dim": 256, "gs": 128, "page": 32, "len_lo": 61, "len_hi": 999},
        # four prompts of about 2k tokens
        {"name": "append prompts 4 2k", "op": "append", "dt": "f16", "batch": 4, "rows_lo": 1801, "rows_hi": 2047, "heads": 32,
         "kv_heads": 8, "dim": 128, "gs": 64, "page": 64, "len_lo": 1801, "len_hi": 2501},
        # pages.  Three pages of a one-layer cache (a draft head's): latency.
        {"name": "copy 3 pages", "op": "copy", "dt": "f16", "layers": 1, "pages": 64, "kv_heads": 8, "dim": 128, "gs": 64,
         "page": 64, "moves": 3},
        # 16 users forked into 4 branches each over 8 layers, last round's branches freed first
        {"name": "fork 16 into 64", "op": "fork", "dt": "f16", "layers": 8, "pages": 1500, "kv_heads": 8, "dim": 128, "gs": 64,
         "page": 64, "sources": 16, "branches": 4, "len_lo": 301, "len_hi": 4000, "width": 64},
        # a pool with every third page live, packed into its lower part
        {"name": "compact 2k pages", "op": "compact", "dt": "bf16", "layers": 8, "pages": 2049, "kv_heads": 8, "dim": 128,
         "gs": 64, "page": 64, "live": 700, "width": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "copy", "fork", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    c = {"op": op, "dt": rng.choice(["f16", "bf16"]), "kv_heads": rng.choice([1, 2, 4, 5, 8, 16]), "dim": dim,
         "gs": rng.choice([g for g in (32, 64, 128) if g <= dim]), "page": rng.choice([32, 64, 64, 128, 256])}
    if op == "attend":
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        c["rows_hi"] = rng.choice([1, 1, rng.randint(2, 8), rng.randint(2, 64)])
        c["rows_lo"] = rng.randint(max(1, c["rows_hi"] // 2), c["rows_hi"])
        c["batch"] = _log(rng, 1, 64)
        # at most the largest listed case: 70k cached tokens of 32 heads of 128 at 64 rows
        most = int(min(131000, 64000 * 8 * 128 / (c["kv_heads"] * dim) / c["batch"],
                       64000 * 64 * 32 * 128 / (c["rows_hi"] * c["heads"] * dim) / c["batch"]))
        c["len_hi"] = _log(rng, max(1, c["rows_hi"]), max(most, c["rows_hi"] + 64))
        c["len_lo"] = rng.randint(min(c["rows_hi"], c["len_hi"]), c["len_hi"])
        c["tree"] = rng.random() < 0.3
    elif op == "append":
        c["heads"] = c["kv_heads"] * rng.choice([1, 4])
        c["batch"] = _log(rng, 1, 64)
        most = max(1, int(8000 * 8 * 128 / (c["kv_heads"] * dim) / c["batch"]))
        c["rows_hi"] = _log(rng, 1, most)
        c["rows_lo"] = rng.randint(1, c["rows_hi"])
        c["len_hi"] = c["rows_hi"] + _log(rng, 1, 2000)
        c["len_lo"] = rng.randint(c["rows_hi"], c["len_hi"])
    else:
        c["layers"] = rng.choice([1, 2, 4, 8])
        size = c["layers"] * c["kv_heads"] * c["page"] * (dim + 8 * (dim // c["gs"]))  # bytes of a page in all layers
        c["pages"] = min(4000, max(40, int(2 ** rng.uniform(18, 30) / size)))
        if op == "copy":
            c["moves"] = _log(rng, 1, max(1, c["pages"] // 3))
        elif op == "fork":
            c["width"] = rng.choice([4, 16, 63])
            c["branches"] = rng.randint(1, 5)
            c["sources"] = max(1, min(32, c["pages"] // (c["width"] + c["branches"])))
            c["len_hi"] = rng.randint(1, min(c["width"], c["pages"] - c["branches"]) * c["page"])
            c["len_lo"] = rng.randint(1, c["len_hi"])
        else:
            c["live"] = rng.randint(1, c["pages"])
            c["width"] = rng.choice([4, 16, 63])
    return c


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, both taken where n > 1, in a mixed order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    return [v[(i * step) % n] for i in range(n)] if math.gcd(step, n) == 1 else v


def _rows_lens(c):
    """New tokens and lengths (the new ones counted in) of each sequence."""
    rows = _spread(c["rows_lo"], c["rows_hi"], c["batch"], 7)
    lens = [max(n, r) for n, r in zip(_spread(c["len_lo"], c["len_hi"], c["batch"], 5), rows)]
    return rows, lens


def _token_bytes(c):
    return c["dim"] + 8 * (c["dim"] // c["gs"])  # K and V of one token and kv head


def work(case):
    c = case
    if c["op"] == "attend":
        rows, lens = _rows_lens(c)
        kv = sum(lens) * c["kv_heads"] * _token_bytes(c)
        io = sum(rows) * c["heads"] * (c["dim"] * 2 * 2 + 4)
        pairs = sum(r * (n - r) + r * (r + 1) // 2 for r, n in zip(rows, lens))
        return {"bytes": kv + io, "flops": 4 * c["dim"] * c["heads"] * pairs}
    if c["op"] == "append":
        # the new rows in, their codes stored, the values they stand for out
        t = sum(_rows_lens(c)[0]) * c["kv_heads"]
        return {"bytes": t * (2 * c["dim"] * 2 * 2 + _token_bytes(c)), "flops": 0}
    page = c["layers"] * c["kv_heads"] * c["page"] * _token_bytes(c)
    if c["op"] == "copy":
        return {"bytes": 2 * page * c["moves"], "flops": 0}
    if c["op"] == "fork":
        n = c["sources"] * c["branches"]
        tails = sum(1 for v in _spread(c["len_lo"], c["len_hi"], c["sources"], 5) if v % c["page"]) * c["branches"]
        return {"bytes": 2 * page * tails + 2 * 4 * n * c["width"] + 8 * c["pages"], "flops": 0}
    # pages live at or above the live count: the live ones are spread evenly
    moved = sum(1 for i in range(c["live"]) if i * c["pages"] // c["live"] >= c["live"])
    return {"bytes": 2 * page * moved + 16 * c["pages"], "flops": 0}


# ---- the format, plain ----

def _quantize(x, gs, dt):
    """x [..., D] of the type -> codes [..., D] int32, scales and biases [..., G] of the type."""
    g = x.float().unflatten(-1, (x.shape[-1] // gs, gs))
    lo = g.amin(-1) + 0.0
    s32 = (g.amax(-1) - lo) / torch.full_like(lo, 15)  # by a number, torch multiplies with its reciprocal
    s = s32.to(dt)
    up = (s.view(torch.int16) + 1).view(dt)
    s = torch.where(s.float() < s32, up, s)
    sf = s.float()[..., None]
    q = torch.where(sf == 0, 0.0, ((g - lo[..., None]) / torch.where(sf == 0, 1.0, sf)).round().clamp(0, 15))
    return q.flatten(-2).to(torch.int32), s, lo.to(dt)


def _pack_k(q):
    """codes [..., D] -> words [..., D/8] in the K order."""
    w = q.unflatten(-1, (q.shape[-1] // 32, 4, 8))
    w = (w << (4 * torch.arange(8, device=q.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    return w.transpose(-1, -2).flatten(-2)


def _pack_v(q):
    """codes [..., D] -> 16-bit halves [..., 16, D/64] in the V order."""
    h = q.unflatten(-1, (q.shape[-1] // 64, 4, 16)).transpose(-1, -2)  # [..., c, i, n]
    h = (h << (4 * torch.arange(4, device=q.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    return h.transpose(-1, -2).to(torch.int16)


def _parts(c):
    """First word of each of the four parts, and the words in all."""
    code, sb = c["page"] * c["dim"] // 8, c["page"] * (c["dim"] // c["gs"])
    return 0, code, 2 * code, 2 * code + sb, 2 * code + 2 * sb


def _values(words, c):
    """Records [..., words] -> K and V values in 32 bits, [..., page, D] each."""
    a, b, s, t, e = _parts(c)
    dim, gs, dt = c["dim"], c["gs"], DT[c["dt"]]
    four = 4 * torch.arange(8, device=words.device, dtype=torch.int32)
    k = words[..., a:b].unflatten(-1, (c["page"], 4, dim // 32))
    k = ((k[..., None] >> four) & 15).transpose(-3, -2).flatten(-3)
    v = words[..., b:s].unflatten(-1, (c["page"] // 4, 16, 2, dim // 64))
    v = ((v[..., None] >> four) & 15).unflatten(-1, (2, 4))  # [..., u, i, p, c, half, n]
    n = v.dim()
    v = v.permute(*range(n - 6), n - 6, n - 4, n - 2, n - 3, n - 1, n - 5).flatten(-3).flatten(-4, -2)

    def values(code, sb):
        sb = sb.contiguous().view(dt).unflatten(-1, (c["page"] // 4, dim // gs, 2, 4)).float()
        sb = sb.movedim(-1, -3).flatten(-4, -3)  # [..., page, G, 2]
        return (code.float().unflatten(-1, (dim // gs, gs)) * sb[..., 0, None] + sb[..., 1, None]).flatten(-2)

    return values(k, words[..., s:t]), values(v, words[..., t:e])


# ---- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pool_of(c, pages, g):
    """A one-layer pool whose pages hold quantized values as a model leaves them: K with offsets of its channels, V without."""
    dt, h, ps, dim = DT[c["dt"]], c["kv_heads"], c["page"], c["dim"]
    words = _parts(c)[-1]
    pool = torch.empty(1, pages, h, words, dtype=torch.int32, device="cuda")
    offs = 1.5 * torch.randn(h, 1, dim, device="cuda", generator=g)
    step = max(1, (1 << 25) // (h * ps * dim))  # pages made at a time
    for at in range(0, pages, step):
        n = min(step, pages - at)
        rec = pool[0, at:at + n]
        for part, off in ((0, offs), (1, 0.0)):
            x = (torch.randn(n, h, ps, dim, device="cuda", generator=g) + off).to(dt)
            q, s, b = _quantize(x, c["gs"], dt)
            first, sb = _parts(c)[part], _parts(c)[2 + part]
            if part == 0:
                w = _pack_k(q).flatten(-2)
            else:  # tokens 2p and 2p + 1 share a word
                v = _pack_v(q).unflatten(-3, (ps // 4, 2, 2)).permute(0, 1, 2, 5, 3, 6, 4).contiguous()
                w = v.view(torch.int32).flatten(-5)
            rec[..., first:first + ps * dim // 8] = w
            both = torch.stack((s, b), -1).unflatten(-3, (ps // 4, 4)).permute(0, 1, 2, 4, 5, 3).contiguous()
            rec[..., sb:sb + ps * (dim // c["gs"])] = both.view(torch.int32).flatten(-4)
    return pool


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


def _cache(c, pool):
    from affine_quantized_gemm_amd import KVCache
    return KVCache(pool, c["dim"], c["gs"], c["page"], DT[c["dt"]])


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    st = {"c": c}
    if c["op"] in ("attend", "append"):
        rows, lens = _rows_lens(c)
        need = [-(-n // c["page"]) for n in lens]
        width, pages = max(need), sum(need) + 3
        order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)  # pages lie anywhere in the pool
        tables = torch.full((c["batch"], width), -1, dtype=torch.int32)
        at = 0
        order = order.cpu()
        for b, n in enumerate(need):
            tables[b, :n] = order[at:at + n]
            at += n
        st["tables"], st["lens"] = tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = np.concatenate([[0], np.cumsum(rows)])
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["ragged"], st["rows_hi"], st["len_hi"] = len(set(rows)) > 1, max(rows), max(lens)
        total = int(starts[-1])
        # q, k and v as the projection of a layer leaves them: one row of all heads a token
        dim, h, hk, dt = c["dim"], c["heads"], c["kv_heads"], DT[c["dt"]]
        qkv = torch.randn(total, (h + 2 * hk) * dim, device="cuda", generator=g).to(dt)
        st["q"] = qkv[:, :h * dim].view(total, h, dim)
        st["k"] = qkv[:, h * dim:(h + hk) * dim].view(total, hk, dim)
        st["v"] = qkv[:, (h + hk) * dim:].view(total, hk, dim)
        if c["op"] == "attend":
            st["pool"] = _pool_of(c, pages, g)
            # what lies past a sequence's end was never written: scales there are NaN
            sb = st["pool"][0, :, :, _parts(c)[2]:].view(torch.int16)
            sb = sb.unflatten(-1, (2, c["page"] // 4, dim // c["gs"], 2, 4))
            ends = torch.tensor([n - 1 for n in need], device="cuda")
            last = st["tables"][torch.arange(c["batch"], device="cuda"), ends].long()
            used = (st["lens"] - ends * c["page"])[:, None] > torch.arange(c["page"], device="cuda")
            used = used.view(c["batch"], 1, 1, c["page"] // 4, 1, 1, 4)
            sb[last] = torch.where(used, sb[last], torch.tensor(0x7fff, dtype=torch.int16, device="cuda"))
            st["mask"] = _tree_masks(rows, g) if c["tree"] else None
        else:
            st["pool"] = torch.zeros(1, pages, hk, _parts(c)[-1], dtype=torch.int32, device="cuda")
    else:
        words = _parts(c)[-1]
        pool = torch.empty(c["layers"], c["pages"], c["kv_heads"], words, dtype=torch.int32, device="cuda")
        pool.random_(-(1 << 31), (1 << 31) - 1, generator=g)
        st["pool"] = pool
        ids = torch.randperm(c["pages"], device="cuda", generator=g, dtype=torch.int32)
        if c["op"] == "copy":
            st["src"], st["dst"] = ids[:c["moves"]].contiguous(), ids[c["moves"]:2 * c["moves"]].contiguous()
        elif c["op"] == "fork":
            n, k, ps = c["sources"], c["branches"], c["page"]
            lens = _spread(c["len_lo"], c["len_hi"], n, 5)
            tables = torch.full((n + n * k, c["width"]), -1, dtype=torch.int32)
            refs = torch.zeros(c["pages"], dtype=torch.int32)
            at, host = 0, ids.cpu()
            for i, v in enumerate(lens):
                m = -(-v // ps)
                tables[i, :m] = host[at:at + m]
                at += m
            refs[host[:at].long()] = 1
            st["tables"], st["refs"] = tables.cuda(), refs.cuda()
            st["lens"] = torch.tensor(lens + [0] * (n * k), dtype=torch.int32, device="cuda")
            st["src"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(k)
            st["dst"] = n + torch.randperm(n * k, device="cuda", generator=g, dtype=torch.int32)
        else:
            # evenly spread live pages, named by the tables in any order, some by two sequences
            live = (torch.arange(c["live"], device="cuda") * c["pages"] // c["live"]).int()
            rows = -(-c["live"] // c["width"])
            full = torch.full((rows * c["width"],), -1, dtype=torch.int32, device="cuda")
            full[:c["live"]] = live[torch.randperm(c["live"], device="cuda", generator=g)]
            tables = full.view(rows, c["width"])
            st["tables"] = torch.cat((tables, tables[:1]))
            st["refs"] = torch.bincount(st["tables"][st["tables"] >= 0], minlength=c["pages"]).int()
    if own:
        st["cache"] = _cache(c, st["pool"])
    return st


# ---- plain forms ----

def _place(st):
    """Sequence, place in it and position of every new token."""
    starts, lens = st["starts"], st["lens"]
    row = torch.arange(st["k"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(starts, row, right=True) - 1
    i = row - starts[b]
    return b, i, lens[b] - (starts[b + 1] - starts[b]) + i


def _plain_attend(st):
    c = st["c"]
    dim, h, hk, dt = c["dim"], c["heads"], c["kv_heads"], DT[c["dt"]]
    tables, lens, starts = st["tables"], st["lens"], st["starts"]
    batch, n = tables.shape[0], tables.shape[1] * c["page"]
    k, v = _values(st["pool"][0][tables.clamp(min=0)], c)  # [B, W, hk, page, D]
    k = k.transpose(1, 2).reshape(batch, hk, n, dim)
    v = v.transpose(1, 2).reshape(batch, hk, n, dim)
    b, i, _ = _place(st)
    m = st["rows_hi"]
    q = torch.zeros(batch, m, h, dim, device="cuda")
    q[b, i] = st["q"].float()
    q = q.view(batch, m, hk, h // hk, dim).permute(0, 2, 1, 3, 4).reshape(batch, hk, m * (h // hk), dim)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(dim)
    bits = torch.zeros(batch, m, dtype=torch.int64, device="cuda")
    bits[b, i] = st["mask"] if st["mask"] is not None else (2 << i.long()) - 1
    new = starts[1:] - starts[:-1]
    j = torch.arange(n, device="cuda")[None] - (lens - new)[:, None]  # place among the new tokens
    allowed = (j[:, None] < 0) | ((bits[:, :, None] >> j.clamp(0, 63)[:, None]) & 1 == 1)
    allowed &= (torch.arange(n, device="cuda")[None] < lens[:, None])[:, None]
    allowed = allowed[:, None, :, None].expand(batch, hk, m, h // hk, n).reshape(batch, hk, -1, n)
    s = torch.where(allowed, s, -torch.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(n, device="cuda")[None] < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.view(batch, hk, m, h // hk, dim).permute(0, 2, 1, 3, 4).reshape(batch, m, h, dim)
    lse = lse.view(batch, hk, m, h // hk).permute(0, 2, 1, 3).reshape(batch, m, h)
    return {"out": o[b, i].to(dt), "lse": lse[b, i]}


def _plain_append(st):
    c = st["c"]
    dim, gs, ps, dt = c["dim"], c["gs"], c["page"], DT[c["dt"]]
    b, _, pos = _place(st)
    page, slot = st["tables"][b, pos // ps].long()[:, None], (pos % ps).long()[:, None]
    head = torch.arange(c["kv_heads"], device="cuda")[None]
    pool, half = st["pool"][0], st["pool"][0].view(torch.int16)
    got = []
    for part, x in ((0, st["k"]), (1, st["v"])):
        q, s, z = _quantize(x, gs, dt)
        first, sb = _parts(c)[part], _parts(c)[2 + part]
        if part == 0:
            at = first + slot * (dim // 8)
            at = at[..., None] + torch.arange(dim // 8, device="cuda")
            pool[page[..., None], head[..., None], at] = _pack_k(q)
        else:  # half-word (u, i, p, c, token & 1)
            i = torch.arange(16, device="cuda")[:, None]
            quad = torch.arange(dim // 64, device="cuda")[None]
            at = (((slot // 4)[..., None, None] * 16 + i) * 2 + (slot % 4 // 2)[..., None, None]) * (dim // 64) + quad
            at = 2 * (first + at) + (slot % 2)[..., None, None]
            half[page[..., None, None], head[..., None, None], at] = _pack_v(q)
        at = 2 * sb + ((slot // 4)[..., None] * (dim // gs) + torch.arange(dim // gs, device="cuda")) * 8 + (slot % 4)[..., None]
        half[page[..., None], head[..., None], at] = s.view(torch.int16)
        half[page[..., None], head[..., None], at + 4] = z.view(torch.int16)
        got.append((q.unflatten(-1, (dim // gs, gs)).float() * s.float()[..., None] + z.float()[..., None]).flatten(-2).to(dt))
    return {"k": got[0], "v": got[1]}


def _plain_free(st, seqs, ps):
    tables, lens, refs = st["tables"], st["lens"], st["refs"]
    rows, seqs = tables[seqs.long()], seqs.long()
    held = torch.arange(tables.shape[1], device="cuda")[None] < (-(-lens[seqs] // ps))[:, None]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -held.flatten().int())
    tables[seqs] = -1
    lens[seqs] = 0


def _plain_fork(st):
    c = st["c"]
    ps, pool, tables, lens, refs = c["page"], st["pool"], st["tables"], st["lens"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    _plain_free(st, st["dst"], ps)
    n = lens[src]
    whole, part = n // ps, n % ps > 0
    free = torch.sort((refs > 0).int(), stable=True).indices  # free pages first, ascending
    rank = torch.cumsum(part.int(), 0) - 1
    ok = ~part | (rank < (refs == 0).sum())
    fresh = free[rank.clamp(0, refs.shape[0] - 1)].int()
    col = torch.arange(tables.shape[1], device="cuda")[None]
    old = tables[src]
    row = torch.where(col < whole[:, None], old, torch.where((col == whole[:, None]) & part[:, None], fresh[:, None], -1))
    tables[dst] = torch.where(ok[:, None], row, -1)
    lens[dst] = torch.where(ok, n, 0)
    shared = (col < whole[:, None]) & ok[:, None]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), shared.flatten().int())
    take = part & ok
    to, come = fresh[take].long(), old.gather(1, whole[:, None].long().clamp(max=tables.shape[1] - 1))[take, 0].long()
    refs[to] = 1
    pool[:, to] = pool[:, come]
    return {"tables": tables, "lens": lens, "refs": refs, "ok": ok.int(), "pool": pool}


def _plain_compact(st):
    pool, tables, refs = st["pool"], st["tables"], st["refs"]
    live, ids = refs > 0, torch.arange(refs.shape[0], device="cuda")
    n = live.sum()
    moves, holes = live & (ids >= n), ~live & (ids < n)
    src, dst = ids[moves], ids[holes]
    to = ids.clone()
    to[src] = dst
    out = torch.where(tables >= 0, to[tables.clamp(min=0).long()].int(), -1)
    counts = torch.where(ids < n, refs, 0)
    counts[dst] = refs[src]
    pool[:, dst] = pool[:, src]
    return {"tables": out, "refs": counts, "pool": pool}


def run(state):
    st = state
    c = st["c"]
    op = c["op"]
    if not own:
        if op == "attend":
            return _plain_attend(st)
        if op == "append":
            return _plain_append(st)
        if op == "copy":
            st["pool"][:, st["dst"].long()] = st["pool"][:, st["src"].long()]
            return {"pool": st["pool"]}
        return _plain_fork(st) if op == "fork" else _plain_compact(st)
    cache = st["cache"]
    if op == "attend":
        ragged = {"starts": st["starts"], "max_new": st["rows_hi"]} if st["ragged"] else {}
        out, lse = cache.attend(0, st["q"], st["tables"], st["lens"], mask=st["mask"], max_len=st["len_hi"], lse=True, **ragged)
        return {"out": out, "lse": lse}
    if op == "append":
        ragged = {"starts": st["starts"], "max_new": st["rows_hi"]} if st["ragged"] else {}
        cache.append(0, st["k"], st["v"], st["tables"], st["lens"], **ragged)
        k, v = cache.read(0, st["k"].shape[0], st["tables"], st["lens"], **ragged)
        return {"k": k, "v": v}
    if op == "copy":
        cache.copy_pages(st["src"], st["dst"])
        return {"pool": st["pool"]}
    if op == "fork":
        cache.free(st["tables"], st["lens"], st["refs"], st["dst"])
        ok = cache.fork(st["tables"], st["lens"], st["refs"], st["src"], st["dst"])
        return {"tables": st["tables"], "lens": st["lens"], "refs": st["refs"], "ok": ok, "pool": st["pool"]}
    tables, refs = cache.compact(st["tables"], st["refs"])
    return {"tables": tables, "refs": refs, "pool": st["pool"]}


# ---- from the definition, in 64 bits ----

def _exact_values(rec, c, part, n):
    """The first n tokens' values of records [W, words] of one head, code by code."""
    dim, gs, ps = c["dim"], c["gs"], c["page"]
    t, d = torch.arange(n, device="cuda")[:, None], torch.arange(dim, device="cuda")[None]
    page, slot = t // ps, t % ps
    if part == 0:
        word, shift = slot * (dim // 8) + (d % 32 // 8) * (dim // 32) + d // 32, 4 * (d % 8) + 0 * slot
    else:
        word = ps * dim // 8 + ((slot // 4 * 16 + d % 16) * 2 + slot % 4 // 2) * (dim // 64) + d // 64
        shift = 4 * (d % 64 // 16) + 16 * (slot % 2)
    code = (rec[page, word].long() >> shift) & 15
    groups = dim // gs
    first = 2 * (2 * (ps * dim // 8) + part * ps * groups)
    at = first + (slot // 4 * groups + d // gs) * 8 + slot % 4
    half = rec.view(DT[c["dt"]])
    return half[page, at].double() * code + half[page, at + 4].double()


def _exact_attend(c, seed):
    st = prepare(c, seed)
    rows, lens = _rows_lens(c)
    h, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(sum(rows), h, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(rows), h), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (r, n) in enumerate(zip(rows, lens)):
        rec = st["pool"][0][st["tables"][b, :-(-n // c["page"])].long()]
        see = torch.ones(r, n, dtype=torch.bool, device="cuda")
        for i in range(r):
            if st["mask"] is None:
                see[i, n - r + i + 1:] = False
            else:
                w = int(st["mask"][at + i])
                see[i, n - r:] = torch.tensor([w >> j & 1 == 1 for j in range(r)], device="cuda")
        for kh in range(hk):
            one = rec[:, kh].contiguous()
            k, v = _exact_values(one, c, 0, n), _exact_values(one, c, 1, n)
            for x in range(kh * (h // hk), (kh + 1) * (h // hk)):
                s = (st["q"][at:at + r, x].double() @ k.t()) / math.sqrt(dim)
                s = s.masked_fill(~see, -math.inf)
                lse[at:at + r, x] = torch.logsumexp(s, -1)
                out[at:at + r, x] = torch.softmax(s, -1) @ v
        at += r
    return {"out": out, "lse": lse}


def _exact_append(c, seed):
    st = prepare(c, seed)
    got = {}
    for name in ("k", "v"):
        x = st[name].cpu().double().numpy()
        t, h, dim = x.shape
        g = x.reshape(t, h, dim // c["gs"], c["gs"]).astype(np.float32)  # exact: the values are of 16 bits
        lo, hi = g.min(-1), g.max(-1)
        step = (hi - lo) / np.float32(15)
        near = torch.from_numpy(step).to(DT[c["dt"]])
        wide = near.double().numpy()
        up = (near.view(torch.int16) + 1).view(DT[c["dt"]]).double().numpy()
        s = np.where(wide < step.astype(np.float64), up, wide)[..., None]
        s32 = s.astype(np.float32)
        q = np.zeros_like(g)
        np.divide(g - lo[..., None], s32, out=q, where=s32 != 0)
        q = np.clip(np.rint(q), 0, 15).astype(np.float64)
        got[name] = (s * q + lo[..., None].astype(np.float64)).reshape(t, h, dim)
    return got


def exact(case, seed):
    c = dict(case)
    if c["op"] == "attend":
        return _exact_attend(c, seed)
    if c["op"] == "append":
        return _exact_append(c, seed)
    return None  # pages and tables: whole numbers
