"""The attention oracle's bound without a GPU: planted mistakes of the size of one group's codes fall outside it."""

import numpy as np
import pytest
import torch

import synth
from oracle import kv_oracle as KO
from oracle import qmm_oracle as O

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def case(dt, n, dim=128, gs=64, heads=2, seed=7):
    k = (synth.normal((n, 1, dim), 1.0, dt, seed).float() + synth.normal((1, 1, dim), 1.5, "f16", seed + 1).float()).to(DT[dt])
    v, q = synth.normal((n, 1, dim), 1.0, dt, seed + 2), synth.normal((1, heads, dim), 1.0, dt, seed + 3)
    page = 64
    pages = -(-n // page)
    c = KO.new_cache(1, pages, 1, dim, gs, page, dt)
    tables = np.arange(pages, dtype=np.int32)[None]
    KO.append(c, 0, synth.to_oracle(k), synth.to_oracle(v), tables, [n], [0, n])
    return c, tables, O.to_f64(synth.to_oracle(q), dt), dim ** -0.5


def flat(c, tables, n, groups, tokens):
    """Codes of V of the given groups and tokens set to 0."""
    c = {**c, "pool": c["pool"].copy()}
    d = np.arange(c["dim"])
    d = d[np.isin(d // c["gs"], groups)]
    for t in tokens:
        word, shift = KO._code_at(c, 1, t % c["page"])
        np.bitwise_and.at(c["pool"][0, tables[0, t // c["page"]], 0], word[d], ~(np.uint32(15) << shift[d].astype(np.uint32)))
    return c


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n", [60, 700, 2000])
def test_mistakes_fall_outside_the_bound(dt, n):
    c, tables, q, scale = case(dt, n)
    out, lse, tol, ltol = KO.attend_bound(c, 0, q, tables, [n], [0, 1], scale)
    plain = KO.attend(c, 0, q, tables, [n], [0, 1], scale)
    assert np.allclose(out, plain[0], rtol=1e-12, atol=0) and np.allclose(lse, plain[1], rtol=1e-12)
    assert np.mean(np.abs(out) > tol) > 0.7                       # zeros for the output
    wrong = KO.attend(flat(c, tables, n, [1], range(n)), 0, q, tables, [n], [0, 1], scale)[0]
    far = np.abs(wrong - out) > tol
    assert far[..., 64:].mean() > 0.95 and not far[..., :64].any()  # one group's codes
    wrong = KO.attend(flat(c, tables, n, [0, 1], range(32)), 0, q, tables, [n], [0, 1], scale)[0]
    assert np.mean(np.abs(wrong - out) > tol) > 0.5               # one step's codes
    shifted = KO.attend(c, 0, q * 1.01, tables, [n], [0, 1], scale)
    assert (np.abs(shifted[1] - lse) > ltol).all()                # scores 1 % off


def test_bound_holds_for_the_roundings():
    """Against an emulation of the kernel's roundings (p s to fp16, p to the type, one rounding at the end)."""
    for dt in ("f16", "bf16"):
        n, dim, gs = 700, 128, 64
        c, tables, q, scale = case(dt, n)
        out, _, tol, _ = KO.attend_bound(c, 0, q, tables, [n], [0, 1], scale)
        data = [[np.array(x) for x in zip(*(KO.load(c, 0, tables[0, t // 64], 0, t % 64, part) for t in range(n)))]
                for part in (0, 1)]
        (kc, ks, kb), (vc, vs, vb) = data
        for x in range(2):
            sc = scale * ((ks * kc + kb) @ q[0, x])
            p = np.exp(sc - sc.max())
            p16 = torch.from_numpy(p).to(DT[dt]).double().numpy()
            ps = (p[:, None] * vs).astype(np.float16).astype(np.float64)
            o = (ps * (vc - 7.5)).sum(0) / p.sum() + (p16[:, None] * (vb + 7.5 * vs)).sum(0) / p16.sum()
            o = torch.from_numpy(o).to(DT[dt]).double().numpy()
            assert (np.abs(o - out[0, x]) <= tol[0, x]).all()
