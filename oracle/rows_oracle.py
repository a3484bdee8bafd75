"""Plain 64-bit forms of the gated block, rotary positions and log probabilities, with bounds for the kernels' results.

Test infrastructure: numpy, no code shared with the HIP path.  Each function
returns values and tolerances that follow the kernels rounding by rounding;
UNIT is half a step of a type, relative.
"""

from __future__ import annotations

import math

import numpy as np

from . import qmm_oracle as O

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def rounding(y, tol, dt):
    """Half a step of the type at |y| + tol (fp16: not below its smallest step)."""
    size = np.abs(y) + tol
    return UNIT[dt] * 2.0 ** np.frexp(size)[1] * 0.5 * (size > 0) + (2.0 ** -25 if dt == "f16" else 0.0)


# ---- gated block ----

def act(name, a):
    """act(a), act'(a) and a bound of |act''|."""
    if name == "silu":
        s = np.where(a >= 0, 1 / (1 + np.exp(-np.abs(a))), np.exp(-np.abs(a)) / (1 + np.exp(-np.abs(a))))
        return a * s, s * (1 + a * (1 - s)), 0.5
    if name == "relu":
        return np.maximum(a, 0), (a > 0).astype(np.float64), 0.0
    if name == "gelu":
        phi = 0.5 * _erfc(-a / math.sqrt(2))
        return a * phi, phi + a * np.exp(-a * a / 2) / math.sqrt(2 * math.pi), 0.8
    r = math.sqrt(2 / math.pi)
    t = r * (a + 0.044715 * a ** 3)
    s = np.where(t >= 0, 1 / (1 + np.exp(-2 * np.abs(t))), np.exp(-2 * np.abs(t)) / (1 + np.exp(-2 * np.abs(t))))
    return a * s, s + 2 * a * s * (1 - s) * r * (1 + 3 * 0.044715 * a * a), 1.2


def _codes(wq, scales, biases, dt, bits, gs):
    q = O.unpack(wq, bits, scales.shape[1] * gs).astype(np.float64)
    s = O.to_f64(scales, dt).repeat(gs, 1)
    b = O.to_f64(biases, dt).repeat(gs, 1)
    return q, s, b


def product(x, wq, scales, biases, dt, bits, gs):
    """x . W^T in 64 bits, and how far fp32 sums of the factored form may be off.

    A group's sum of x (q + off) takes GS/32 + 2 additions of at most A = sum |x| (q + off) (2^-23 each: the matrix core
    does not say how it rounds), the groups' sums and the terms of the biases U + 8 of at most sum |x w| + 4 max s A."""
    q, s, b = _codes(wq, scales, biases, dt, bits, gs)
    off = 1024.0 if dt == "f16" else 0.0 if bits == 8 else 128.0
    y = x @ (s * q + b).T
    a = np.abs(x)
    groups = q.shape[1] // gs
    parts = np.stack([(a[:, g * gs:(g + 1) * gs] @ (s * (q + off))[:, g * gs:(g + 1) * gs].T) for g in range(groups)])
    size = a @ np.abs(s * q + b).T
    e = 2.0 ** -23 * ((gs / 32 + 2) * parts.sum(0) + (groups + 8) * (size + 4 * parts.max(0)))
    return y, e


def gated(x, wq, scales, biases, dt, bits, gs, name, grad=None):
    """h and its tolerance; with grad: (grad_x, grad_gate_up) and theirs.

    act and act' are evaluated to 2^-21 (4 + |a|) of max(1, |a|) (the exponential's argument is off by 2^-23 of itself);
    |act'| <= 1.2."""
    f = scales.shape[0] // 2
    y, e = product(x, wq, scales, biases, dt, bits, gs)
    g, u, eg, eu = y[:, :f], y[:, f:], e[:, :f], e[:, f:]
    v, slope, bend = act(name, g)
    ev = 2.0 ** -21 * (4 + np.minimum(np.abs(g), 30)) * np.minimum(np.abs(v) + 2.0 ** -60, 1e30)
    et = 2.0 ** -21 * (4 + np.minimum(np.abs(g), 30)) * (np.abs(slope) + 1)
    if name == "relu":
        kink = np.abs(g) <= eg
        et = et + kink
    tv = 1.2 * eg + ev
    if grad is None:
        h = v * u
        tol = tv * (np.abs(u) + eu) + np.abs(v) * eu + 2.0 ** -22 * np.abs(h)
        return h, tol + rounding(h, tol, dt)
    ts = bend * eg + et
    dg, du = grad * u * slope, grad * v
    tg = np.abs(grad) * ((np.abs(u) + eu) * ts + np.abs(slope) * eu) + 2.0 ** -22 * np.abs(dg)
    tu = np.abs(grad) * tv + 2.0 ** -22 * np.abs(du)
    d, t = np.concatenate([dg, du], 1), np.concatenate([tg, tu], 1)
    return d, t


def gated_backward(x, wq, scales, biases, dt, bits, gs, name, grad):
    """(grad_x, its tolerance, grad_gate_up, its tolerance).

    grad_x is formed from the fp32 gradients: d times a scale in two bf16 pieces, within 2^-16 of it, times q + off (off 16,
    64 or 0 for 4, 6, 8 bits), plus d (b - off s) in fp32; sums of 2F terms over 2F/32 + 40 additions, 2^-23 each."""
    d, t = gated(x, wq, scales, biases, dt, bits, gs, name, grad)
    q, s, b = _codes(wq, scales, biases, dt, bits, gs)
    w = s * q + b
    y = d @ w
    a = np.abs(d) + t
    off = {4: 16.0, 6: 64.0, 8: 0.0}[bits]
    size = s * (q + off)
    tol = t @ np.abs(w) + 2.0 ** -16 * (a @ size) + 2.0 ** -23 * (d.shape[1] / 32 + 40) * (a @ (size + np.abs(b - off * s)))
    return y, tol + rounding(y, tol, dt), d, t + rounding(d, t, dt)


# ---- rotary positions ----

def rotary(x, positions, freq, sections, pairs, inverse, scale, dt):
    """positions [axes][rows].  An angle is off by 2^-22 (what is left of the revolutions, in fp32), cos and sin by 2^-22,
    the products and sums by 2^-23 each.  In fp64 a position times a frequency, and the kernel's product of a position with
    freq / (2 pi), which is rounded too, are off by 2^-53 and 2 * 2^-53 of the angle, so that there is no more to compare for
    positions of 10^12 (2^-51 of the angle)."""
    half = len(freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = (positions.astype(np.float64)[axis] * freq.astype(np.float64)[:, None]).T[:, None]
    c, s = np.cos(angle) * scale, np.sin(angle) * (-scale if inverse else scale)
    y, tol = x.copy(), np.zeros_like(x)
    a, b = (slice(0, half), slice(half, 2 * half)) if pairs == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    t = (2.0 ** -20 + 2.0 ** -51 * np.abs(angle)) * abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a] = t + rounding(y[..., a], t, dt)
    tol[..., b] = t + rounding(y[..., b], t, dt)
    return y, tol


# ---- log probabilities ----

def _safe(p, x):
    return np.where(p > 0, p * np.where(p > 0, x, 0), 0)


def log_probs(logits, tokens, top, scale):
    """logits in 64 bits (finite or -infinity): dict of lse, entropy, tokens, top_values, top_ids and a tolerance of each
    but the ids.

    With t = z - max, a 2^t is off by r = 2^-23 (8 + |t|) of itself, and sums of n terms in one lane and of the lanes by
    2^-24 (n + 64): sums of 2^t by E = sum p r + that, of t 2^t by sum p |t| r + that of sum p |t|."""
    rows, vocab = logits.shape
    z = scale * logits
    m = z.max(1, keepdims=True)
    none = np.isneginf(m)
    t = np.where(none, -np.inf, z - np.where(none, 0, m))
    with np.errstate(divide="ignore", invalid="ignore"):
        total = np.exp(t).sum(1, keepdims=True)
        lse = np.where(none, -np.inf, m + np.log(total))
        p = np.where(none, 0, np.exp(t) / np.where(none, 1, total))
        # (not z - lse: beside logits of 10^37 the logarithm of the sum is below a step of 64 bits)
        lp = np.where(none, -np.inf, t - np.log(total))
    size = np.where(np.isfinite(t), np.abs(t), 0)
    adds = 2.0 ** -24 * (vocab / 256 + 64)
    e = (p * 2.0 ** -23 * (8 + size)).sum(1) + adds
    mean = (p * size).sum(1)
    entropy = -_safe(p, lp).sum(1)
    tol_lse = e + 2.0 ** -22 * (np.abs(np.where(none, 0, lse)[:, 0]) + np.abs(np.where(none, 0, m)[:, 0]) + 2)
    tol_h = 2 * e + (p * size * 2.0 ** -23 * (8 + size)).sum(1) + (e + adds + 2.0 ** -22) * mean + 2.0 ** -22 * (entropy + 1)
    out = {"lse": lse[:, 0], "entropy": entropy, "tol_lse": tol_lse, "tol_entropy": tol_h}

    def at(ids):
        v = np.take_along_axis(lp, ids, 1)
        tt = np.take_along_axis(size, ids, 1)
        return v, e[:, None] + 2.0 ** -22 * (tt + np.abs(np.where(np.isfinite(v), v, 0)) + 2)

    if tokens is not None:
        ids = tokens.reshape(rows, -1)
        bad = (ids < 0) | (ids >= vocab)
        v, tol = at(np.where(bad, 0, ids))
        out["tokens"], out["tol_tokens"] = (np.where(bad, x, y).reshape(tokens.shape) for x, y in ((0, v), (0, tol)))
    if top:
        ids = np.argsort(-logits, axis=1, kind="stable")[:, :top]
        out["top_ids"] = ids
        out["top_values"], out["tol_top_values"] = at(ids)
    return out


def log_probs_backward(logits, tokens, lse, entropy, g_tokens, g_entropy, g_lse, scale, dt):
    """The gradient from lse and entropy as given, and its tolerance: ln p is off by 2^-23 (|scale z| + |lse|), p by 2^-22
    (2 + |ln p|) of itself more, the sums and products by a few 2^-24 of their terms."""
    rows, vocab = logits.shape
    none = np.isneginf(lse)
    base = np.where(none, 0, lse)[:, None]
    lp = np.where(none[:, None], -np.inf, scale * logits - base)
    p = np.exp(lp)
    live = np.isfinite(lp)
    size = np.where(live, np.abs(lp), 0)
    elp = 2.0 ** -23 * (np.where(live, np.abs(scale * logits), 0) + np.abs(base))
    g = np.zeros(rows)
    d, t = np.zeros_like(p), np.zeros_like(p)
    if g_tokens is not None:
        ids = tokens.reshape(rows, -1)
        good = (ids >= 0) & (ids < vocab) & ~none[:, None]
        gt = np.where(good, g_tokens.reshape(ids.shape), 0)
        r = np.arange(rows)[:, None].repeat(ids.shape[1], 1)
        np.add.at(d, (r, np.where(good, ids, 0)), gt)
        np.add.at(t, (r, np.where(good, ids, 0)), 2.0 ** -22 * ids.shape[1] * np.abs(gt))
        g = gt.sum(1)
        spread = np.abs(gt).sum(1) * ids.shape[1]
    else:
        spread = np.zeros(rows)
    gh = np.zeros(rows) if g_entropy is None else g_entropy
    h = np.zeros(rows) if g_entropy is None else entropy
    gl = np.zeros(rows) if g_lse is None else g_lse
    inner = (gl - g - gh * h)[:, None] - gh[:, None] * np.where(live, lp, 0)
    most = (np.abs(gl) + np.abs(g) + spread + np.abs(gh * h))[:, None] + np.abs(gh)[:, None] * size
    d = scale * (d + p * inner)
    t = scale * (t + p * (np.abs(inner) * (elp + 2.0 ** -22 * (2 + size)) + np.abs(gh)[:, None] * elp + 2.0 ** -22 * most))
    t += 2.0 ** -23 * np.abs(d)
    return d, t + rounding(d, t, dt)
