"""64-bit attention under a causal mask, a sliding window and sinks, and how far a kernel's output may be off.

Plain numpy; nothing here looks at the library.

Tolerance of an output o = sum p v / sum p, S = sum p |v| / sum p:
  half a step of the output type at |o|, and S times what the weights p are off by, relatively:
  * scores: a sum of D products in fp32, D 2^-24 of sum |q||k| scale, twice in a weight (its own and the maximum's
    part in the denominator);
  * exp2, the sums and the quotient: 2^-18 (ex2.approx 2^-22, sums of up to a few thousand rounded terms in blocks);
  * weights enter the second product as fp16 (2^-11), as a bf16 pair (2^-16), or in fp32 or an fp16 pair (2^-22); as
    fp16 a weight below
    2^-14 of the base is held to 2^-25, which a row of L tokens meets at most L times (the base's own weight is at
    least 1): L 2^-25 max |v|;
  * grouped heads over an E4M3 cache at D = 128, single tokens: q goes in as three E4M3 terms, each to 2^-4 of what
    the ones before left: 2^-12 |q|, or 2^-17 of the largest |q| where that is more;
  * 4-bit caches: a score sums step times code and the offset apart, at most 3 times sum |q||k|, by matrix instructions
    of 16 products, each to two units of 2^-23 of what is summed: 3 * 16 * 2^-23; a code meets q to 2^-17 of a
    step times the largest |q| (half the elements; 2^-21 the other half); of V a product of 16 tokens keeps a code
    to 2^-17 of a step each at the largest weight, 2^-13 of a step per unit of weight."""
import math

import numpy as np

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def seen(length, pos, window, sinks):
    """[rows, length]: whether the query at pos[r] sees the key at t."""
    t, p = np.arange(length), np.asarray(pos)[:, None]
    m = t <= p
    return m & ((t > p - window) | (t < sinks)) if window else m


def attend(q, k, v, scale, pos, window=0, sinks=0):
    """q [n, Hq, D], k and v [L, Hkv, D] (float64) -> dict of out [n, Hq, D] and what the tolerance needs."""
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out, size = np.zeros_like(q), np.zeros_like(q)
    big, many, qk = np.zeros((n, hq, 1)), np.zeros((n, 1, 1)), np.zeros((n, hq, 1))
    m = seen(length, pos, window, sinks)
    many[:, 0, 0] = m.sum(1)
    alone = np.abs(q).max(2, keepdims=True) * scale if q.size else np.zeros((n, hq, 1))
    top = np.zeros((n, hq, 1))
    for h in range(hq):
        g = h // (hq // hkv)
        use = m.any(0)
        if not use.any():
            continue
        kk, vv, mm = k[use, g], v[use, g], m[:, use]
        z = np.where(mm, q[:, h] @ kk.T * scale, -np.inf)
        live = mm.any(1)
        with np.errstate(invalid="ignore"):
            p = np.exp(z - np.where(live, z.max(1), 0)[:, None])
        p = np.where(live[:, None], p / np.where(live, p.sum(1), 1)[:, None], 0)
        out[:, h], size[:, h] = p @ vv, p @ np.abs(vv)
        big[:, h, 0] = (np.abs(q[:, h]) @ np.abs(kk).T * scale * mm).max(1)
        qk[:, h, 0] = (np.abs(q[:, h]).max(1)[:, None] * np.abs(kk).sum(1) * scale * mm).max(1)
        top[:, h, 0] = (mm[:, :, None] * np.abs(vv)[None]).max((1, 2)) if n * use.sum() < 1 << 16 else np.abs(vv).max()
    return dict(out=out, size=size, big=big, many=many, qk=qk, top=top, d=d, alone=alone)


def tolerance(r, model, p="f32", terms=False, steps=None):
    """p: how the weights enter the second product ("f32", "f16", "pair"); terms: q as E4M3 terms; steps: the largest
    steps of K and V in a 4-bit cache."""
    score = r["d"] * 2.0 ** -24 * r["big"]
    if terms:
        score = score + 2.0 ** -12 * r["big"] + 2.0 ** -17 * r["qk"]
    if steps:
        score = 3 * 16 * 2.0 ** -23 * r["big"] + r["d"] * r["alone"] * steps[0] * (2.0 ** -18 + 2.0 ** -22)
    weight = 2 * score + 2.0 ** -18 + {"f32": 0.0, "f16": 2.0 ** -11, "pair": 2.0 ** -16}[p]
    lost = weight * r["size"] + (r["many"] * 2.0 ** -25 * r["top"] if p == "f16" else 0.0)
    if steps:
        lost = lost + 2.0 ** -13 * steps[1]
    return HALF[model] * (np.abs(r["out"]) + lost) + lost + 2.0 ** -25


def check(got, r, model, p="f32", terms=False, steps=None):
    err = np.abs(np.asarray(got, np.float64) - r["out"])
    tol = tolerance(r, model, p, terms, steps)
    assert np.isfinite(got).all()
    worst = float((err / tol).max()) if err.size else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} times the tolerance, at most {err.max():.3e}"


def scale_of(d):
    return 1.0 / math.sqrt(d)
