"""Plain CPU oracle of the paged 4-bit K/V cache.

TEST INFRASTRUCTURE ONLY (as ``qmm_oracle``, whose quantizer it uses).  A
cache is a dict: ``pool`` uint32 [layers, pages, kv_heads, words] and the
geometry.  Positions are written and read one value at a time through index
arithmetic; attention is computed in fp64 from the dequantized values s*q + b.
"""

from __future__ import annotations

import numpy as np

from . import qmm_oracle as O


def record_words(dim, gs, page):
    return page * dim // 4 + 2 * page * (dim // gs)


def new_cache(layers, pages, kv_heads, dim, gs, page, dt, fill=0):
    pool = np.full((layers, pages, kv_heads, record_words(dim, gs, page)), fill, dtype=np.uint32)
    return {"pool": pool, "dim": dim, "gs": gs, "page": page, "dt": dt}


def _code_at(c, part, slot):
    """(word, shift) [dim] of one token's codes."""
    dim, d = c["dim"], np.arange(c["dim"])
    if part == 0:
        return slot * (dim // 8) + (d // 8 % 4) * (dim // 32) + d // 32, 4 * (d % 8)
    unit = (slot // 4) * 16 + d % 16
    word = c["page"] * dim // 8 + (unit * 2 + slot % 4 // 2) * (dim // 64) + d // 64
    return word, 4 * (d % 64 // 16) + 16 * (slot % 2)


def _half_at(c, part, slot):
    """Half-word [groups] of one token's scales (biases: 4 further)."""
    groups = c["dim"] // c["gs"]
    first = c["page"] * c["dim"] // 4 + part * c["page"] * groups
    return 2 * first + ((slot // 4) * groups + np.arange(groups)) * 8 + slot % 4


def store(c, layer, page, head, slot, part, x):
    """Quantize one token's values x [dim] (oracle dtype) into its slot."""
    wq, s, b = O.quantize(x.reshape(1, -1), c["dt"], 4, c["gs"])
    codes = O.unpack(wq, 4, c["dim"])[0].astype(np.uint32)
    rec = c["pool"][layer, page, head]
    word, shift = _code_at(c, part, slot)
    np.bitwise_and.at(rec, word, ~(np.uint32(15) << shift.astype(np.uint32)))
    np.bitwise_or.at(rec, word, codes << shift.astype(np.uint32))
    half = rec.view(np.uint16)
    at = _half_at(c, part, slot)
    half[at] = s.reshape(-1).view(np.uint16)
    half[at + 4] = b.reshape(-1).view(np.uint16)


def load(c, layer, page, head, slot, part):
    """(codes int, scales, biases) [dim], fp64, of one token."""
    rec = c["pool"][layer, page, head]
    word, shift = _code_at(c, part, slot)
    codes = (rec[word].astype(np.int64) >> shift) & 15
    half = rec.view(np.uint16)
    at = _half_at(c, part, slot)
    tod = (lambda a: a.view(np.float16).astype(np.float64)) if c["dt"] == "f16" else (lambda a: O.to_f64(a, "bf16"))
    return codes, np.repeat(tod(half[at].copy()), c["gs"]), np.repeat(tod(half[at + 4].copy()), c["gs"])


def places(starts, lens):
    """(sequence, row in it, position) of every new token."""
    out = []
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        out += [(b, i, int(lens[b]) - n + i) for i in range(n)]
    return out


def page_of(c, tables, b, pos):
    if pos < 0 or pos // c["page"] >= tables.shape[1]:
        return -1
    p = int(tables[b, pos // c["page"]])
    return p if 0 <= p < c["pool"].shape[1] else -1


def append(c, layer, k, v, tables, lens, starts):
    for row, (b, _, pos) in enumerate(places(starts, lens)):
        page = page_of(c, tables, b, pos)
        if page < 0:
            continue
        for h in range(k.shape[1]):
            store(c, layer, page, h, pos % c["page"], 0, k[row, h])
            store(c, layer, page, h, pos % c["page"], 1, v[row, h])


def read(c, layer, tables, lens, starts, kv_heads):
    """fp64 values s*q + b of the new tokens: k, v [rows, kv_heads, dim] (zeros where there is no page)."""
    where = places(starts, lens)
    out = np.zeros((2, len(where), kv_heads, c["dim"]))
    for row, (b, _, pos) in enumerate(where):
        page = page_of(c, tables, b, pos)
        if page < 0:
            continue
        for h in range(kv_heads):
            for part in (0, 1):
                q, s, z = load(c, layer, page, h, pos % c["page"], part)
                out[part, row, h] = s * q + z
    return out[0], out[1]


def attend(c, layer, q, tables, lens, starts, scale, mask=None):
    """q [rows, heads, dim] fp64 -> out, lse, and per element a coarse bound of how far a kernel may be off.

    The bound is that of a plainer kernel, which rounds more, and over many
    tokens it is as large as the output (``attend_bound`` follows the
    roundings that there are).  u: half a unit in the last place of the type,
    relative:
      * out is rounded once: u |out|;
      * p s is rounded to the type before the second product, whose codes are
        taken about their middle (|code - 8| <= 8): 8 u sum p s, twice that
        where the codes' offset is removed by a second sum of the same
        rounded p s;  an fp16 p s below 2^-14 is off by up to 2^-25 instead;
      * the score of a token is off by E = 2^-21 scale (sum_g s_g 160 sum_{d in g} |q_d| + sum_d |q_d k_d|):
        fp32 sums of at most 256 products with codes that carry an offset of
        at most 144 (and 2^-24 a step); p is then off by 2 E + 2^-21 of
        itself, and so is every term of out, and of the sum that divides it;
      * sums of n terms in fp32, of magnitude at most sum p (|v| + 24 s):
        2^-24 n / 32 of that (32 terms a step).
    """
    rows, heads, dim = q.shape
    hk = c["pool"].shape[2]
    u = 2.0 ** -11 if c["dt"] == "f16" else 2.0 ** -8
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    cap = tables.shape[1] * c["page"]
    row = 0
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        length = min(max(int(lens[b]), 0), cap)
        pages = [page_of(c, tables, b, t) for t in range(length)]
        got = [t for t in range(length) if pages[t] >= 0]
        for h in range(hk):
            data = [[load(c, layer, pages[t], h, t % c["page"], part) for t in got] for part in (0, 1)]
            ks, kz, kc = (np.array([d[j] for d in data[0]]).reshape(len(got), dim) for j in (1, 2, 0))
            vs, vz, vc = (np.array([d[j] for d in data[1]]).reshape(len(got), dim) for j in (1, 2, 0))
            kk, vv = ks * kc + kz, vs * vc + vz
            for i in range(n):
                new = np.array(got, dtype=np.int64) - (int(lens[b]) - n)
                word = int(mask[row + i]) if mask is not None else (2 << i) - 1
                see = np.array([j < 0 or (j < 64 and word >> int(j) & 1) for j in new], dtype=bool)
                if not see.any():
                    continue
                for x in range(h * (heads // hk), (h + 1) * (heads // hk)):
                    qq = q[row + i, x]
                    sc = scale * (kk[see] @ qq)
                    e = abs(scale) * (160 * (ks[see] @ np.abs(qq)) + np.abs(kk[see]) @ np.abs(qq)).max() * 2.0 ** -21
                    top = sc.max()
                    p = np.exp(sc - top)
                    total = p.sum()
                    o = p @ vv[see] / total
                    ps = p[:, None] * vs[see]
                    small = (ps < 2.0 ** -14).sum(0) * 2.0 ** -22 if c["dt"] == "f16" else 0.0
                    size = p @ (np.abs(vv[see]) + 24 * vs[see]) / total
                    rel = 2 * (2 * e + 2.0 ** -21) + 2.0 ** -24 * (1 + len(p) / 32)
                    out[row + i, x] = o
                    tol[row + i, x] = u * np.abs(o) + (16 * u * ps.sum(0) + small) / total + rel * size + 2.0 ** -25
                    lse[row + i, x] = top + np.log(total)
                    ltol[row + i, x] = 2 * e + 2.0 ** -20 * (1 + abs(top) + len(p) / 4096)
        row += n
    return out, lse, tol, ltol


def attend_bound(c, layer, q, tables, lens, starts, scale, mask=None):
    """As ``attend``, with a bound that follows the kernel rounding by rounding: out, lse, tol, ltol.

    With weights w_t = p_t / l of the tokens that a row sees, p <= 1, out = sum w (s (code - 7.5) + m), m = b + 7.5 s.
    N: tokens of the sequence.  u: 2^-11 (fp16) or 2^-8 (bf16), a rounding to the type.

      * out is rounded once, after all that follows: half a unit in its last place (fp16: at least 2^-25);
      * p s is an fp16 operand, for either type: 2^-11 |code - 7.5| w s;  the largest p s of a row and group counts
        for at least 2^-4, so one below 2^-10 of it (a subnormal) is off by up to 2^-21 of that largest instead;
      * the matrix core cuts each product with a code off at 2^-18 of a code times the largest p s of the 32 of one
        product, in the sum and in what centres it: 2 * 32 * 2^-18 w s;
      * p is rounded to the type for the middles m, and so is the sum that they are divided by: only what m differs
        from its mean counts, 2 u w |m - mean| (a mean per part of the sequence, hence 2);  fp16: the row's largest p
        counts for at least 4, one below 2^-16 of it is off by up to 2^-27 of that;
      * the score of a token is off by E = |scale| (2 * 32 * 2^-18 sum_g s_g sum_(32 d in g) max |q| [the same cut]
        + 2^-21 sum_g (15 s_g + |b_g|) sum_(d in g) |q_d|) + 2^-21 (|score| + |top| + 8), the last for the argument and the
        value of the exponential: w E |v - out|;
      * fp32 sums: of n = N / 32 + 4 steps, 2^-22 n of the 30 w s that the codes and their centre add up to and of
        w (|b| + 7.5 s), and the N / 4 of l, 2^-24 each, of out.
    """
    rows, heads, dim = q.shape
    hk, gs = c["pool"].shape[2], c["gs"]
    G = dim // gs
    half = c["dt"] == "f16"
    u = 2.0 ** -11 if half else 2.0 ** -8
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    cap = tables.shape[1] * c["page"]
    row = 0
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        length = min(max(int(lens[b]), 0), cap)
        pages = [page_of(c, tables, b, t) for t in range(length)]
        got = [t for t in range(length) if pages[t] >= 0]
        new = np.array(got, dtype=np.int64) - (int(lens[b]) - n)
        for h in range(hk if n else 0):
            data = [[load(c, layer, pages[t], h, t % c["page"], part) for t in got] for part in (0, 1)]
            kc, ks, kb, vc, vs, vb = (np.array([d[j] for d in data[i]]).reshape(len(got), dim)
                                      for i in (0, 1) for j in (0, 1, 2))
            kk, vv = ks * kc + kb, vs * vc + vb
            for i in range(n):
                word = int(mask[row + i]) if mask is not None else (2 << i) - 1
                see = np.array([j < 0 or (j < 64 and word >> int(j) & 1) for j in new], dtype=bool)
                if not see.any():
                    continue
                s, v, m, off = vs[see], vv[see], vb[see] + 7.5 * vs[see], np.abs(vc[see] - 7.5)
                for x in range(h * (heads // hk), (h + 1) * (heads // hk)):
                    qq = q[row + i, x]
                    a = np.abs(qq)
                    sc = scale * (kk[see] @ qq)
                    top = sc.max()
                    p = np.exp(sc - top)
                    total = p.sum()
                    w = (p / total)[:, None]
                    o = (w * v).sum(0)
                    chunks = a.reshape(dim // 32, 32).max(1).repeat(32) / 32
                    e = abs(scale) * (2.0 ** -12 * (ks[see] @ chunks) + 2.0 ** -21 * ((15 * ks[see] + np.abs(kb[see])) @ a))
                    e = (e + 2.0 ** -21 * (np.abs(sc) + abs(top) + 8))[:, None]
                    steps, ws, ps = length / 32 + 4, w * s, p[:, None] * s
                    mean = (w * m).sum(0)
                    t = 2.0 ** -11 * (ws * off).sum(0)
                    t += 2.0 ** -21 * ps.max(0) / total * (off * (ps < 2.0 ** -9 * ps.max(0))).sum(0)
                    t += 2.0 ** -12 * ws.sum(0)
                    t += 2 * u * (w * np.abs(m - mean)).sum(0)
                    if half:
                        t += 2.0 ** -27 / total * (np.abs(m - mean) * (p < 2.0 ** -15)[:, None]).sum(0)
                    t += 1.01 * (w * e * np.abs(v - o)).sum(0)
                    t += 2.0 ** -22 * steps * (30 * ws + w * (np.abs(vb[see]) + 7.5 * s)).sum(0)
                    t += 2.0 ** -24 * (length / 4 + 64) * np.abs(o)
                    t += np.maximum(u * 2.0 ** (np.frexp(np.abs(o) + t)[1] - 1), 2.0 ** -25 if half else 0.0)
                    out[row + i, x], tol[row + i, x] = o, t
                    lse[row + i, x] = top + np.log(total)
                    ltol[row + i, x] = 1.01 * (w * e).sum() + 2.0 ** -20 * (1 + abs(top)) + 2.0 ** -24 * length / 4
        row += n
    return out, lse, tol, ltol


# ---- pages ----

def reserve(tables, lens, refs, add, page):
    ok = np.zeros(len(lens), dtype=np.int32)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    before = 0
    for s in range(len(lens)):
        if lens[s] < 0 or add[s] < 0 or int(lens[s]) + int(add[s]) > tables.shape[1] * page:
            continue
        want = -(-(int(lens[s]) + int(add[s])) // page)
        c = -(-int(lens[s]) // page)
        while c < want and tables[s, c] >= 0:
            c += 1
        need = want - c
        before += need
        if need and before > len(free):
            continue
        for x in range(need):
            tables[s, c + x] = free[before - need + x]
            refs[free[before - need + x]] = 1
        lens[s] += add[s]
        ok[s] = 1
    return ok


def fork(pool, tables, lens, refs, src, dst, page):
    ok = np.zeros(len(src), dtype=np.int32)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    used = 0
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (0 <= s < len(lens) and 0 <= d < len(lens)) or s == d:
            continue
        tables[d], lens[d] = -1, 0
        n = int(lens[s])
        if not 0 <= n <= tables.shape[1] * page:
            continue
        whole, part = n // page, n % page > 0
        if part:
            last = tables[s, whole]
            if not 0 <= last < len(refs):
                continue
            used += 1
            if used > len(free):
                continue
        tables[d, :whole] = tables[s, :whole]
        for p in tables[s, :whole]:
            refs[p] += 1
        if part:
            tables[d, whole] = free[used - 1]
            refs[free[used - 1]] = 1
            pool[:, free[used - 1]] = pool[:, last]
        lens[d] = n
        ok[i] = 1
    return ok


def free(tables, lens, refs, which):
    for s in which:
        if 0 <= s < len(lens):
            for p in tables[s]:
                if 0 <= p < len(refs):
                    refs[p] -= 1
            tables[s], lens[s] = -1, 0


def compact(pool, tables, refs):
    live = int((refs > 0).sum())
    movers = [p for p in range(len(refs)) if p >= live and refs[p] > 0]
    holes = [p for p in range(live) if refs[p] <= 0]
    to = {p: p for p in range(len(refs))}
    out_refs = np.where(np.arange(len(refs)) < live, refs, 0).astype(np.int32)
    for m, h in zip(movers, holes):
        to[m] = h
        out_refs[h] = refs[m]
        pool[:, h] = pool[:, m]
    out = np.array([[to.get(int(p), -1) for p in row] for row in tables], dtype=np.int32).reshape(tables.shape)
    return out, out_refs, live
