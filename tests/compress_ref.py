"""64-bit references of the cache-compression calls, straight from their definitions: 4-bit rows, attention with its
mass, eviction.  Plain numpy; nothing here looks at the library."""
import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def to64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def round_model(x, model: str) -> np.ndarray:
    """float64 (holding fp32 values) -> the model type's nearest value, as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().to(TORCH[model]).double().numpy()


def quantise4(rows: np.ndarray, model: str):
    """rows float64 [..., D] of model-type values -> codes uint8, step, low (float64), as the append stores them.

    The differences and quotients are rounded to fp32 as the definition says; np.rint ties to even."""
    with np.errstate(over="ignore", invalid="ignore"):
        low, high = rows.min(-1), rows.max(-1)
        span = (high - low).astype(np.float32)
        step = round_model((span / np.float32(15)).astype(np.float64), model)
        bad = ~np.isfinite(span)
    step = np.where(step < 2.0 ** -126, 0.0, step)
    step, low = np.where(bad, np.nan, step), np.where(bad, np.nan, low)
    ok = (step > 0)[..., None]
    with np.errstate(invalid="ignore"):
        d = (rows - low[..., None]).astype(np.float32)
        y = d / np.where(ok, step[..., None], 1.0).astype(np.float32)
        codes = np.where(ok, np.minimum(np.rint(y), 15), 0).astype(np.uint8)
    return codes, step, low


def values4(codes, step, low):
    return codes * step[..., None] + low[..., None]


def attention(q, k, v, scale):
    """q [Hq, D], k and v [L, Hkv, D], float64 -> (out [Hq, D], p [Hq, L], sum p|v| [Hq, D], largest sum |q||k| scale)."""
    hq, hkv, L = q.shape[0], k.shape[1], k.shape[0]
    if L == 0:
        z = np.zeros_like(q)
        return z, np.zeros((hq, 0)), z, 0.0
    g = hq // hkv
    kk, vv = np.repeat(k, g, axis=1), np.repeat(v, g, axis=1)
    x = np.einsum("hd,thd->ht", q, kk) * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    big = float(np.einsum("hd,thd->ht", np.abs(q), np.abs(kk)).max() * scale)
    return np.einsum("ht,thd->hd", p, vv), p, np.einsum("ht,thd->hd", p, np.abs(vv)), big


def code_alignment(d, q, step, scale):
    """What the 4-bit products lose: a code enters as a subnormal number, whose product with q is kept to 2^-17 of a code
    step times the head's largest |q| (half the elements; 2^-21 the other half).  Bound of a score's error, for a
    softmax weight twice that; q [Hq, D], step [L, Hkv] float64."""
    if step.size == 0:
        return 0.0
    return 2 * scale * float(np.abs(q).max() * step.max()) * d * (2.0 ** -18 + 2.0 ** -22)


def relative_weight_error(big):
    """Bound on a softmax weight's relative error.

    A score sums at most 8 matrix instructions of 16 products each, in fp32; each may lose a unit of 2^-23 of the
    largest partial sum on the way in and out: 16 * 2^-23 of sum |q||k| scale.  The 4-bit form sums |step c| and
    |offset| parts instead of their difference, at most 3 times as much for codes centred in the row's range.  A
    weight's exponent takes the error of its score and of the maximum's: twice that.  2^-19 is for exp2 (2^-22), the
    hi + lo 16-bit weights (2^-16 for bf16 pairs, counted apart) and fp32 sums over the splits."""
    return 2 * 3 * 16 * 2.0 ** -23 * big + 2.0 ** -19


def evict(mass, length, budget, recent):
    """mass [T] -> kept positions of one (sequence, head), by sorting (NaN last, ties to the lower position)."""
    if length <= budget:
        return list(range(length))
    n = length - recent
    def rank(t):
        m = float(mass[t])
        return (1, 0.0, t) if m != m else (0, -m, t)
    best = sorted(range(n), key=rank)[: budget - recent]
    return sorted(best) + list(range(n, length))
