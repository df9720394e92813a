"""Cases of the cache-compression operators: the 4-bit cache (append and read back, decode attention), the decode
attention that accumulates attention mass, and the eviction by that mass.

``own`` false: plain forms in elementary torch operations, 32 bits throughout, rounded once at the end.  ``own`` true:
the calls a user makes of paged_kv_cache_134_gb300.
"""
import math

import torch

own = False

DEV = "cuda"
MODEL = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the new token of a small batch written to a 4-bit cache and read back: a launch's latency
        dict(name="int4_append_step", op="append", tokens=32, hkv=8, d=128, bs=16, model="bf16"),
        # the packed prompts of the prefill configuration (5256 tokens, 32 heads) quantised into the cache and read
        # back, as when a finished prompt's cache is handed on at the model's precision
        dict(name="int4_append_prompt", op="append", tokens=5256, hkv=32, d=128, bs=16, model="f16"),
        # four short sequences at the smallest head size: the smallest decode call
        dict(name="int4_decode_tiny", op="decode", kv="int4", seqs=4, max_len=37, law="uniform", hq=8, hkv=8, d=64,
             bs=16, model="f16"),
        # the 7B layer shape, 32 sequences of 1..4096 tokens, one query head per KV head
        dict(name="int4_decode_7b", op="decode", kv="int4", seqs=32, max_len=4096, law="uniform", hq=32, hkv=32, d=128,
             bs=16, model="f16"),
        # a large batch of log-normal lengths (median 500), four query heads per KV head
        dict(name="int4_decode_stress", op="decode", kv="int4", seqs=256, max_len=8192, law="lognormal", hq=32, hkv=8,
             d=128, bs=16, model="bf16"),
        # one long conversation: few rows, the work has to be split along the sequence
        dict(name="int4_decode_long", op="decode", kv="int4", seqs=1, max_len=131071, law="full", hq=32, hkv=8, d=128,
             bs=32, model="bf16"),
        # a cache under eviction at the 7B shape: every step accumulates the mass of each token
        dict(name="mass_f16_7b", op="mass", kv="f16", seqs=32, max_len=4096, law="uniform", hq=32, hkv=32, d=128,
             bs=16, model="f16", decay=1.0),
        # the same with a 4-bit cache and grouped heads, old mass fading
        dict(name="mass_int4_stress", op="mass", kv="int4", seqs=256, max_len=8192, law="lognormal", hq=32, hkv=8,
             d=128, bs=16, model="bf16", decay=0.99),
        # one sequence in an E4M3 cache, eight query heads per KV head, small blocks
        dict(name="mass_fp8_one", op="mass", kv="fp8", seqs=1, max_len=2047, law="full", hq=64, hkv=8, d=128, bs=8,
             model="bf16", decay=1.0),
        # four short sequences cut to 16 tokens: the smallest eviction
        dict(name="evict_tiny", op="evict", seqs=4, max_len=37, law="uniform", hkv=8, d=64, bs=16, model="f16",
             budget=16, recent=4),
        # a full batch at the 7B shape cut to 1024 tokens a sequence
        dict(name="evict_7b", op="evict", seqs=32, max_len=4096, law="uniform", hkv=32, d=128, bs=16, model="f16",
             budget=1024, recent=256),
        # two long prompts cut to a sixteenth before decoding goes on
        dict(name="evict_long", op="evict", seqs=2, max_len=131071, law="full", hkv=8, d=128, bs=32, model="bf16",
             budget=8191, recent=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "mass", "mass", "evict"])
    d, bs, model = rng.choice([64, 128, 128]), rng.choice([8, 16, 32]), rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 5256), hkv=hkv, d=d, bs=bs, model=model)
    # tokens of the whole batch times KV heads: at most what the listed 7B cases hold
    seqs = _log(rng, 1, 256)
    most = min(131071, 32 * 1900 * 32 // (seqs * hkv))
    max_len = _log(rng, 1, max(1, most))
    law = rng.choice(["uniform", "lognormal", "full"])
    case = dict(op=op, seqs=seqs, max_len=max_len, law=law, hkv=hkv, d=d, bs=bs, model=model)
    if op == "evict":
        budget = max(1, int(max_len * rng.uniform(0.05, 1.1)))
        return dict(case, budget=budget, recent=int(budget * rng.uniform(0.0, 1.0)))
    group = rng.choice([1, 2, 4, 8]) if hkv < 32 else 1
    case.update(kv="int4", hq=hkv * group)
    if op == "mass":
        case.update(kv=rng.choice(["int4", "fp8", model]), decay=rng.choice([1.0, 0.99]))
    return case


# ------------------------------------------------------------------------------------------------ inputs

def _lens(case):
    """Lengths of the batch: fixed by the case, so that work() knows them."""
    g = torch.Generator().manual_seed(case["seqs"] * 1000003 + case["max_len"])
    n, hi = case["seqs"], case["max_len"]
    if case["law"] == "full":
        return torch.full((n,), hi, dtype=torch.int32)
    if case["law"] == "uniform":
        return torch.randint(1, hi + 1, (n,), generator=g, dtype=torch.int32)
    x = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) + math.log(500.0))
    return x.round().clamp(1, hi).to(torch.int32)


def _tables(lens, bs, first, gen):
    """Tables over a shuffled run of blocks that starts at `first` (-1 behind a sequence's blocks), and their number."""
    need = (lens.long() + bs - 1) // bs
    total, widest = int(need.sum()), int(need.max())
    blocks = torch.randperm(total, generator=gen, device=DEV, dtype=torch.int32) + first
    ends = need.cumsum(0).to(DEV)
    at = (ends - need.to(DEV))[:, None] + torch.arange(widest, device=DEV)
    inside = at < ends[:, None]
    return torch.where(inside, blocks[at.clamp(max=total - 1)], -1).contiguous(), total


def _fp8_scales(x):
    return (x.float().abs().amax(dim=(0, 2)).clamp(min=1e-6) / torch.full((), 448.0, device=DEV)).contiguous()


def _inputs(case, seed):
    """Inputs from the seed alone: what both sides and the definition start from."""
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    md, hkv, d, bs = MODEL[case["model"]], case["hkv"], case["d"], case["bs"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(md)

    x = dict(case=case, md=md)
    # keys of a few channels are far larger than the rest, as models have them
    gain = torch.ones(hkv, d, device=DEV)
    gain[:, :: 32] = 4.0
    if case["op"] == "append":
        n = case["tokens"]
        blocks = (n + bs - 1) // bs + 3
        slots = torch.randperm(blocks * bs, generator=gen, device=DEV)[:n].contiguous()
        x.update(k=(normal(n, hkv, d) * gain).to(md), v=normal(n, hkv, d), slots=slots, blocks=blocks)
        return x
    lens = _lens(case)
    tables, total = _tables(lens, bs, 0, gen)
    n = int(lens.sum())
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), lens.to(DEV).long())
    start = (lens.long().cumsum(0) - lens.long()).to(DEV)
    pos = torch.arange(n, device=DEV) - start[seq]
    slots = tables[seq, pos // bs].long() * bs + pos % bs
    x.update(lens=lens.to(DEV), tables=tables, blocks=total, slots=slots, seq=seq, pos=pos, start=start,
             k=(normal(n, hkv, d) * gain).to(md), v=normal(n, hkv, d), scale=1.0 / math.sqrt(d))
    if case["op"] != "decode":
        # the mass that earlier steps left: a few heavy tokens, a long light tail
        x["mass"] = torch.rand(case["seqs"], hkv, case["max_len"], generator=gen, device=DEV).pow(8) * 4
    if case["op"] == "evict":
        kept = lens.clamp(max=case["budget"])
        x["dst"], more = _tables(kept, bs, total, gen)
        x["blocks"] = total + more
        return x
    x["q"] = normal(case["seqs"], case["hq"], d)
    if case["kv"] == "fp8":
        x.update(k_scale=_fp8_scales(x["k"]), v_scale=_fp8_scales(x["v"]))
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    kv = case.get("kv") or ("int4" if case["op"] == "append" else case["model"])
    nb, bs, hkv, d = x["blocks"], case["bs"], case["hkv"], case["d"]
    if own:
        import paged_kv_cache_134_gb300 as P
        x["cache"] = P.KVCache(nb, bs, hkv, d, kv_dtype=kv, model_dtype=case["model"])
        if kv == "fp8":
            x["cache"].set_scales(x["k_scale"], x["v_scale"])
        if case["op"] != "append":
            P.paged_kv_append(x["cache"], x.pop("k"), x.pop("v"), x["slots"])
        if case["op"] == "evict":
            x["pool"] = x["cache"].view()[0].view(x["md"]).view(nb, 2, hkv, bs, d)
        return x
    # the plain cache: [K|V][slot][head] rows, 4-bit codes two to a byte with their step and offset
    x["rows"] = None
    if kv == "int4":
        x["codes"] = torch.zeros(2, nb * bs, hkv, d // 2, dtype=torch.uint8, device=DEV)
        x["step"] = torch.zeros(2, nb * bs, hkv, dtype=x["md"], device=DEV)
        x["low"] = torch.zeros_like(x["step"])
        if case["op"] != "append":
            _write4(x, x.pop("k"), x.pop("v"))
    elif case["op"] == "evict":
        x["pool"] = torch.zeros(nb, 2, hkv, bs, d, dtype=x["md"], device=DEV)
        b, o = x["slots"] // bs, x["slots"] % bs
        x["pool"][b, 0, :, o] = x.pop("k")
        x["pool"][b, 1, :, o] = x.pop("v")
    else:
        t = torch.float8_e4m3fn if kv == "fp8" else x["md"]
        rows = torch.stack([x.pop("k"), x.pop("v")]).float()
        if kv == "fp8":
            rows = (rows / torch.stack([x["k_scale"], x["v_scale"]])[:, None, :, None]).clamp(-448, 448)
        x["rows"] = torch.zeros(2, nb * bs, hkv, d, device=DEV).to(t)
        x["rows"].view(torch.uint8 if kv == "fp8" else t)[:, x["slots"]] = \
            rows.to(t).view(torch.uint8 if kv == "fp8" else t)
    return x


# ------------------------------------------------------------------------------------------------ plain forms

def _write4(x, k, v):
    """4-bit rows: offset = the row's least value, step = a fifteenth of its range, both in the model's type."""
    rows = torch.stack([k, v]).float()
    low, high = rows.amin(-1), rows.amax(-1)
    step = ((high - low) / torch.full_like(low, 15.0)).to(x["md"]).float()
    step = torch.where(step < 2.0 ** -126, torch.zeros_like(step), step)
    div = torch.where(step == 0, torch.ones_like(step), step)
    code = ((rows - low[..., None]) / div[..., None]).round().clamp(0, 15) * (step > 0)[..., None]
    code = code.to(torch.uint8)
    x["codes"][:, x["slots"]] = code[..., 0::2] | (code[..., 1::2] << 4)
    x["step"][:, x["slots"]] = step.to(x["md"])
    x["low"][:, x["slots"]] = low.to(x["md"])


def _read4(x, slots):
    """Values of the rows at `slots` (any shape): fp32 [2, *slots, hkv, d]."""
    codes = x["codes"][:, slots]
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    return code * x["step"][:, slots].float()[..., None] + x["low"][:, slots].float()[..., None]


def _rows(x, slots):
    if x["case"]["kv"] == "int4":
        return _read4(x, slots)
    if x["case"]["kv"] == "fp8":
        r = x["rows"].view(torch.uint8)[:, slots].view(torch.float8_e4m3fn).float()
        scale = torch.stack([x["k_scale"], x["v_scale"]])
        return r * scale.view(2, *([1] * slots.dim()), -1, 1)
    return x["rows"][:, slots].float()


def _attend(x):
    """Softmax weights [S, hkv, group, T] and outputs over every sequence's slots, padded to the longest."""
    c = x["case"]
    t = torch.arange(c["max_len"], device=DEV)
    valid = t < x["lens"][:, None]
    wide = x["tables"].shape[1]
    slots = x["tables"][:, (t // c["bs"]).clamp(max=wide - 1)].long() * c["bs"] + t % c["bs"]
    k, v = _rows(x, torch.where(valid, slots, 0))
    q = x["q"].float().view(c["seqs"], c["hkv"], -1, c["d"])
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * x["scale"]
    s = torch.where(valid[:, None, None], s, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)).view(c["seqs"], c["hq"], c["d"])
    return p, out.to(x["md"]), valid


def _evict(x):
    c = x["case"]
    bs, budget = c["bs"], c["budget"]
    lens = x["lens"].long()
    t = torch.arange(c["max_len"], device=DEV)
    valid = (t < lens[:, None])[:, None]
    late = (t >= (lens - c["recent"])[:, None])[:, None]
    rank = torch.where(late, math.inf, x["mass"])
    rank = torch.where(valid, rank, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    new = lens.clamp(max=budget)
    j = torch.arange(budget, device=DEV)
    taken = (j < new[:, None])[:, None]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=c["max_len"])
    kept = torch.where(taken, order, c["max_len"]).sort(dim=-1).values
    at = kept.clamp(max=c["max_len"] - 1)
    mass = torch.zeros_like(x["mass"])
    n = min(budget, c["max_len"])
    mass[..., :n] = torch.where(taken, x["mass"].gather(-1, at), 0.0)[..., :n]
    s, h, j = taken.expand(kept.shape).nonzero(as_tuple=True)
    i = kept[s, h, j]
    x["pool"][x["dst"][s, j // bs], :, h, j % bs] = x["pool"][x["tables"][s, i // bs], :, h, i % bs]
    return torch.where(taken, kept, -1).to(torch.int32), new.to(torch.int32), mass, x["pool"]


def run(x):
    c = x["case"]
    if own:
        import paged_kv_cache_134_gb300 as P
        if c["op"] == "append":
            P.paged_kv_append(x["cache"], x["k"], x["v"], x["slots"])
            return P.paged_kv_gather(x["cache"], x["slots"])
        if c["op"] == "decode":
            return P.paged_decode_attention(x["q"], x["cache"], x["tables"], x["lens"], x["scale"])
        if c["op"] == "mass":
            out = P.paged_decode_attention_mass(x["q"], x["cache"], x["tables"], x["lens"], x["scale"], x["mass"],
                                                decay=c["decay"])
            return out, x["mass"]
        kept, lens, mass = P.paged_kv_evict(x["cache"], x["tables"], x["lens"], x["mass"], c["budget"], c["recent"],
                                            x["dst"])
        return kept, lens, mass, x["pool"]
    if c["op"] == "append":
        _write4(x, x["k"], x["v"])
        k, v = _read4(x, x["slots"])
        return k.to(x["md"]), v.to(x["md"])
    if c["op"] == "evict":
        return _evict(x)
    p, out, valid = _attend(x)
    if c["op"] == "decode":
        return out
    new = x["mass"] * c["decay"] + p.sum(2)
    x["mass"].copy_(torch.where(valid[:, None], new, x["mass"]))
    return out, x["mass"]


# ------------------------------------------------------------------------------------------------ work, definition

ROW_BYTES = {"f16": lambda d: 2 * d, "bf16": lambda d: 2 * d, "fp8": lambda d: d, "int4": lambda d: d // 2 + 4}


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "append":
        rows = 2 * case["tokens"] * hkv
        return {"bytes": rows * (2 * d + 2 * (d // 2 + 4) + 2 * d) + 16 * case["tokens"], "flops": 6 * rows * d}
    lens = _lens(case).long()
    n, blocks = int(lens.sum()), int(((lens + case["bs"] - 1) // case["bs"]).sum())
    if case["op"] == "evict":
        kept = int(lens.clamp(max=case["budget"]).sum())
        return {"bytes": 4 * n * hkv + 4 * case["seqs"] * hkv * (case["budget"] + case["max_len"])
                + 2 * kept * hkv * 4 * d, "flops": n * hkv}
    b = 2 * n * hkv * ROW_BYTES[case["kv"]](d) + 4 * blocks + 2 * 2 * case["seqs"] * case["hq"] * d
    if case["op"] == "mass":
        b += 8 * n * hkv
    return {"bytes": b, "flops": 4 * n * case["hq"] * d}


def _def4(r, md):
    """The 4-bit value of each element of rows r (float64), from the definition."""
    low, high = r.amin(-1, keepdim=True), r.amax(-1, keepdim=True)
    step = ((high - low) / 15).to(torch.float32).to(md).double()
    code = torch.where(step > 0, (r - low) / torch.where(step > 0, step, 1.0), 0.0)
    return low + step * torch.round(code).clamp(0, 15)


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "append":
        return _def4(x["k"].double(), x["md"]), _def4(x["v"].double(), x["md"])
    if case["op"] == "evict":
        return None  # whole numbers and moved bits
    lens = _lens(case).tolist()
    out = torch.empty(case["seqs"], case["hq"], case["d"], dtype=torch.float64, device=DEV)
    mass = x["mass"].double() if case["op"] == "mass" else None
    group = case["hq"] // case["hkv"]
    at = 0
    for s, n in enumerate(lens):
        rows = []
        for name in ("k", "v"):
            r = x[name][at:at + n].double()
            if case["kv"] == "int4":
                r = _def4(r, x["md"])
            elif case["kv"] == "fp8":
                f = x[name + "_scale"][:, None]
                r = (x[name][at:at + n].float() / f).clamp(-448, 448).to(torch.float8_e4m3fn).double() * f.double()
            rows.append(r.repeat_interleave(group, dim=1))
        k, v = rows
        z = torch.einsum("hd,thd->ht", x["q"][s].double(), k) * x["scale"]
        p = torch.softmax(z, dim=-1)
        out[s] = torch.einsum("ht,thd->hd", p, v)
        if mass is not None:
            mass[s, :, :n] = mass[s, :, :n] * case["decay"] + p.view(case["hkv"], group, n).sum(1)
        at += n
    return out if mass is None else (out, mass)
