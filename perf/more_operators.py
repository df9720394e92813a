"""Cases of the operators between a layer's projections: keys and values appended to the cache with the norms and the
position rotation on the way, decode attention with a sliding window and sinks, and the attention of a chunk of new
tokens over the cache.

``own`` false: plain forms in elementary torch operations, 32 bits (angles in 64), rounded once at the end.  ``own``
true: the calls a user makes of paged_kv_cache_134_gb300.
"""
import math

import torch

own = False

DEV = "cuda"
MODEL = {"f16": torch.float16, "bf16": torch.bfloat16}
FAR = 131072  # positions of a long context


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the new token of a 7B batch of 32: rotation and append in front of a decode, a launch's latency
        dict(name="rotary_step_7b", op="rotary", seqs=32, new=1, far=False, hq=32, hkv=32, d=128, bs=16, model="f16",
             rot=128, pairs="half", norm=False, scaled=False),
        # the packed prompts of the prefill configuration's size (5256 tokens of 8 sequences), one query head per KV head
        dict(name="rotary_prompt_7b", op="rotary", seqs=8, new=657, far=False, hq=32, hkv=32, d=128, bs=16,
             model="f16", rot=128, pairs="half", norm=False, scaled=False),
        # chunks of long conversations, grouped heads with normed queries and keys, half of the head rotated by
        # frequencies scaled for a long context
        dict(name="rotary_norm_chunks", op="rotary", seqs=4, new=2047, far=True, hq=32, hkv=8, d=128, bs=16,
             model="bf16", rot=64, pairs="interleaved", norm=True, scaled=True),
        # four short sequences at the smallest head size, less than two blocks each in sight
        dict(name="window_tiny", op="window", kv="f16", seqs=4, max_len=37, law="uniform", hq=8, hkv=8, d=64, bs=16,
             model="f16", window=16, sinks=4),
        # the 7B batch with a window of a quarter of its longest context
        dict(name="window_7b", op="window", kv="f16", seqs=32, max_len=4096, law="uniform", hq=32, hkv=32, d=128,
             bs=16, model="f16", window=1024, sinks=4),
        # many log-normal lengths in an E4M3 cache, grouped heads, odd window
        dict(name="window_fp8_stress", op="window", kv="fp8", seqs=256, max_len=8192, law="lognormal", hq=32, hkv=8,
             d=128, bs=16, model="bf16", window=511, sinks=1),
        # few long conversations: the window has to be split
        dict(name="window_long", op="window", kv="bf16", seqs=4, max_len=131071, law="full", hq=32, hkv=8, d=128,
             bs=32, model="bf16", window=8192, sinks=64),
        # one sequence, a handful of drafted tokens, small blocks: latency
        dict(name="chunk_one", op="chunk", kv="bf16", seqs=1, max_len=2047, law="full", new=7, ragged=False, hq=64,
             hkv=8, d=128, bs=8, model="bf16", window=0, sinks=0),
        # drafted tokens of the 7B batch, checked in one pass
        dict(name="chunk_draft_7b", op="chunk", kv="f16", seqs=32, max_len=4096, law="uniform", new=5, ragged=False,
             hq=32, hkv=32, d=128, bs=16, model="f16", window=0, sinks=0),
        # the same for many ragged sequences over an E4M3 cache
        dict(name="chunk_draft_fp8", op="chunk", kv="fp8", seqs=256, max_len=8192, law="lognormal", new=4,
             ragged=False, hq=32, hkv=8, d=128, bs=16, model="bf16", window=0, sinks=0),
        # a batch that mixes single tokens with pieces of prompts, under a window
        dict(name="chunk_mixed_window", op="chunk", kv="bf16", seqs=64, max_len=8192, law="uniform", new=512,
             ragged=True, hq=32, hkv=8, d=128, bs=16, model="bf16", window=1024, sinks=4),
        # a piece of a prompt at the end of a long conversation
        dict(name="chunk_long", op="chunk", kv="bf16", seqs=1, max_len=131071, law="full", new=512, ragged=False,
             hq=32, hkv=8, d=128, bs=32, model="bf16", window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rotary", "window", "window", "chunk", "chunk"])
    d, bs, model = rng.choice([64, 128, 128]), rng.choice([8, 16, 32]), rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    hq = hkv * (rng.choice([1, 2, 4, 8]) if hkv < 32 else 1)
    if op == "rotary":
        tokens = _log(rng, 1, 5256 * 96 * 128 // ((hq + 2 * hkv) * d) // 2)
        seqs = _log(rng, 1, min(64, tokens))
        return dict(op=op, seqs=seqs, new=max(1, min(tokens // seqs, 8192)), far=rng.random() < 0.5, hq=hq, hkv=hkv, d=d,
                    bs=bs, model=model, rot=rng.choice([d, d, d // 2, d // 4]), pairs=rng.choice(["half", "interleaved"]),
                    norm=rng.random() < 0.5, scaled=rng.random() < 0.5)
    kv = rng.choice(["fp8", model, model])
    law = rng.choice(["uniform", "lognormal", "full"])
    seqs = _log(rng, 1, 256)
    # tokens of the whole batch times KV heads: at most what the 7B batch holds
    max_len = _log(rng, 1, max(1, min(131071, 32 * 1900 * 32 // (seqs * hkv))))
    case = dict(op=op, kv=kv, seqs=seqs, max_len=max_len, law=law, hq=hq, hkv=hkv, d=d, bs=bs, model=model)
    window, sinks = _log(rng, 1, max_len), rng.choice([0, 1, 4, 64])
    if op == "window":
        return dict(case, window=window, sinks=sinks)
    # new tokens: never more than the context, and products of at most the long listed case
    new = min(max_len, _log(rng, 1, 512))
    while new > 1 and seqs * new * hq * max_len * d > 512 * 32 * 131071 * 128 // 4:
        new //= 2
    windowed = rng.random() < 0.5
    return dict(case, new=new, ragged=rng.random() < 0.5, window=window if windowed else 0,
                sinks=sinks if windowed else 0)


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


def _news(case, lens):
    """New tokens of each sequence, at most its length: all alike, or a few long pieces among short ones."""
    if not case["ragged"]:
        return torch.minimum(lens, torch.full_like(lens, case["new"]))
    g = torch.Generator().manual_seed(case["seqs"] * 7919 + case["new"])
    u = torch.rand(case["seqs"], generator=g, dtype=torch.float64).pow(3)
    n = torch.exp(u * math.log(case["new"])).round().to(torch.int32).clamp(1, case["new"])
    return torch.minimum(lens, n)


def _tables(need, gen, wide=0):
    """Tables over a shuffled run of blocks (-1 behind a sequence's blocks), and their number."""
    total, widest = int(need.sum()), max(int(need.max()), wide)
    blocks = torch.randperm(total, generator=gen, device=DEV, dtype=torch.int32)
    ends = need.cumsum(0).to(DEV)
    at = (ends - need.to(DEV))[:, None] + torch.arange(widest, device=DEV)
    return torch.where(at < ends[:, None], blocks[at.clamp(max=total - 1)], -1).contiguous(), total


def _starts(case):
    """First position of each sequence's new tokens."""
    g = torch.Generator().manual_seed(case["seqs"] * 31 + case["new"])
    if case["far"]:
        return torch.randint(0, FAR - case["new"] + 1, (case["seqs"],), generator=g)
    return torch.zeros(case["seqs"], dtype=torch.int64) if case["new"] > 1 else \
        torch.randint(0, 4096, (case["seqs"],), generator=g)


def _inputs(case, seed):
    """Inputs from the seed alone: what both sides and the definition start from."""
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    md, hq, hkv, d, bs = MODEL[case["model"]], case["hq"], case["hkv"], case["d"], case["bs"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(md)

    x = dict(case=case, md=md)
    if case["op"] == "rotary":
        s, n = case["seqs"], case["new"]
        start = _starts(case)
        first, last = start // bs, (start + n - 1) // bs
        # blocks of the new tokens only: what lies before them is not touched by the append
        some, total = _tables(last - first + 1, gen)
        tables = torch.full((s, int(last.max()) + 1), -1, dtype=torch.int32, device=DEV)
        at = first.to(DEV)[:, None] + torch.arange(some.shape[1], device=DEV)
        row = torch.arange(s, device=DEV)[:, None].expand(at.shape)
        tables[row[some >= 0], at[some >= 0]] = some[some >= 0]
        seq = torch.arange(s, device=DEV, dtype=torch.int32).repeat_interleave(n)
        pos = (start.to(DEV)[:, None] + torch.arange(n, device=DEV)).reshape(-1).to(torch.int32)
        qkv = normal(s * n, (hq + 2 * hkv) * d)  # one projection's output: rows of q, k and v side by side
        q, k, v = (t.view(s * n, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
        x.update(q=q, k=k, v=v, tables=tables, seq=seq, pos=pos, blocks=total)
        if case["norm"]:
            x.update(wq=(normal(d) * 0.1 + 1).to(md), wk=(normal(d) * 0.1 + 1).to(md))
        return x
    lens = _lens(case)
    tables, total = _tables((lens.long() + bs - 1) // bs, gen)
    n = int(lens.sum())
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), lens.to(DEV).long())
    start = (lens.long().cumsum(0) - lens.long()).to(DEV)
    pos = torch.arange(n, device=DEV) - start[seq]
    x.update(lens=lens.to(DEV), tables=tables, blocks=total, slots=tables[seq, pos // bs].long() * bs + pos % bs,
             k=normal(n, hkv, d), v=normal(n, hkv, d), scale=1.0 / math.sqrt(d), host_lens=lens.tolist())
    if case["op"] == "window":
        x["q"] = normal(case["seqs"], hq, d) * 2
    else:
        new = _news(case, lens)
        x["host_new"] = new.tolist()
        x["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.long().cumsum(0)]).to(torch.int32).to(DEV)
        x["q"] = normal(int(new.sum()), hq, d) * 2
        x["most"] = int(new.max())
    if case["kv"] == "fp8":
        for name in ("k", "v"):
            x[name + "_scale"] = (x[name].float().abs().amax(dim=(0, 2)).clamp(min=1e-6) / 448.0).contiguous()
    return x


# scaled frequencies: slow dimensions divided by the factor, fast ones kept, a ramp over those between, and the
# attention's temperature folded into the rotated values
LONG = dict(type="yarn", factor=32.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0)


def _frequencies(rot, scaled):
    """Radians a position and the factor of cos and sin, in 64 bits."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if not scaled:
        return f, 1.0

    def dim_of(turns):
        return rot * math.log(LONG["original_max_position"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))

    low = max(math.floor(dim_of(LONG["beta_fast"])), 0)
    high = min(math.ceil(dim_of(LONG["beta_slow"])), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / LONG["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(LONG["factor"]) + 1.0


def prepare(case, seed):
    x = _inputs(case, seed)
    nb, bs, hkv, d = x["blocks"], case["bs"], case["hkv"], case["d"]
    kv = case.get("kv", case["model"])
    if own:
        import paged_kv_cache_134_gb300 as P
        x["cache"] = P.KVCache(nb, bs, hkv, d, kv_dtype=kv, model_dtype=case["model"])
        if case["op"] == "rotary":
            x["rotary"] = P.Rotary(case["rot"], base=10000.0, interleaved=case["pairs"] == "interleaved",
                                   scaling=LONG if case["scaled"] else None)
            x["pool"] = x["cache"].view()[0].view(x["md"]).view(nb, 2, hkv, bs, d)
            return x
        if kv == "fp8":
            x["cache"].set_scales(x["k_scale"], x["v_scale"])
        P.paged_kv_append(x["cache"], x.pop("k"), x.pop("v"), x["slots"])
        return x
    if case["op"] == "rotary":
        x["freq"], x["gain"] = _frequencies(case["rot"], case["scaled"])
        x["freq"] = x["freq"].to(DEV)
        x["pool"] = torch.zeros(nb, 2, hkv, bs, d, dtype=x["md"], device=DEV)
        return x
    t = torch.float8_e4m3fn if kv == "fp8" else x["md"]
    rows = torch.stack([x.pop("k"), x.pop("v")]).float()
    if kv == "fp8":
        rows = (rows / torch.stack([x["k_scale"], x["v_scale"]])[:, None, :, None]).clamp(-448, 448)
    raw = torch.uint8 if kv == "fp8" else t
    x["rows"] = torch.zeros(2, nb * bs, hkv, d, device=DEV).to(t)
    x["rows"].view(raw)[:, x["slots"]] = rows.to(t).view(raw)
    return x


# ------------------------------------------------------------------------------------------------ plain forms

def _turned(r, angle, gain, rot, pairs):
    """Rows r [T, H, D] with their first `rot` elements rotated by angle [T, rot / 2]."""
    c, s = (angle.cos() * gain).to(r.dtype)[:, None], (angle.sin() * gain).to(r.dtype)[:, None]
    a, b = (r[..., :rot // 2], r[..., rot // 2:rot]) if pairs == "half" else (r[..., :rot:2], r[..., 1:rot:2])
    y, z = a * c - b * s, b * c + a * s
    turned = torch.cat([y, z], -1) if pairs == "half" else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([turned, r[..., rot:]], -1)


def _rotary(x):
    c = x["case"]
    angle = x["pos"].double()[:, None] * x["freq"]
    rows = []
    for t, w in ((x["q"], "wq"), (x["k"], "wk")):
        r = t.float()
        if c["norm"]:
            r = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6) * x[w].float()
        rows.append(_turned(r, angle, x["gain"], c["rot"], c["pairs"]).to(x["md"]))
    b = x["tables"][x["seq"].long(), x["pos"].long() // c["bs"]].long()
    o = x["pos"].long() % c["bs"]
    x["pool"][b, 0, :, o] = rows[1]
    x["pool"][b, 1, :, o] = x["v"]
    return rows[0], x["pool"]


def _rows(x, slots):
    """Values at `slots` (any shape): fp32 [2, *slots, hkv, d]."""
    if x["case"]["kv"] == "fp8":
        r = x["rows"].view(torch.uint8)[:, slots].view(torch.float8_e4m3fn).float()
        return r * torch.stack([x["k_scale"], x["v_scale"]]).view(2, *([1] * slots.dim()), -1, 1)
    return x["rows"][:, slots].float()


def _seen(t, p, window, sinks):
    """Whether the query at position p sees the key at t."""
    seen = t <= p
    return seen & ((t > p - window) | (t < sinks)) if window else seen


def _window(x):
    c = x["case"]
    last = x["lens"].long()[:, None] - 1
    # the sinks, then the window from its first token on, each token once
    t = torch.arange(min(c["sinks"], c["max_len"]), device=DEV).expand(c["seqs"], -1)
    w = torch.arange(min(c["window"], c["max_len"]), device=DEV)
    w = (last - c["window"] + 1).clamp(min=0) + w
    t = torch.cat([t, torch.where(w < c["sinks"], c["max_len"], w)], 1)
    seen = t <= last
    t = torch.where(seen, t, 0)
    slots = x["tables"].gather(1, t // c["bs"]).long() * c["bs"] + t % c["bs"]
    k, v = _rows(x, slots)
    q = x["q"].float().view(c["seqs"], c["hkv"], -1, c["d"])
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * x["scale"]
    s = torch.where(seen[:, None, None], s, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    out = torch.matmul(e / e.sum(-1, keepdim=True), v.permute(0, 2, 1, 3))
    return out.view(c["seqs"], c["hq"], c["d"]).to(x["md"])


def _chunk(x):
    c = x["case"]
    out = torch.empty_like(x["q"])
    at = 0
    for s, (length, n) in enumerate(zip(x["host_lens"], x["host_new"])):
        t = torch.arange(max(0, length - n - c["window"] + 1) if c["window"] else 0, length, device=DEV)
        if c["window"]:
            t = torch.cat([torch.arange(min(c["sinks"], int(length - t.numel())), device=DEV), t])
        slots = x["tables"][s, t // c["bs"]].long() * c["bs"] + t % c["bs"]
        seen = _seen(t, torch.arange(length - n, length, device=DEV)[:, None], c["window"], c["sinks"])
        k, v = _rows(x, slots)
        q = x["q"][at:at + n].float().view(n, c["hkv"], -1, c["d"]).permute(1, 2, 0, 3)  # [hkv, group, n, d]
        o = torch.empty(c["hkv"], q.shape[1], n, c["d"], device=DEV)
        step = max(1, (1 << 29) // max(1, q.shape[1] * n * t.numel()))  # KV heads at a time: scores of 2 GB
        for h in range(0, c["hkv"], step):
            z = torch.matmul(q[h:h + step], k[:, h:h + step].permute(1, 2, 0)[:, None]) * x["scale"]
            z = torch.where(seen, z, -math.inf)
            e = torch.exp(z - z.amax(-1, keepdim=True))
            o[h:h + step] = torch.matmul(e / e.sum(-1, keepdim=True), v[:, h:h + step].transpose(0, 1)[:, None])
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["hq"], c["d"]).to(x["md"])
        at += n
    return out


def run(x):
    c = x["case"]
    if not own:
        return {"rotary": _rotary, "window": _window, "chunk": _chunk}[c["op"]](x)
    import paged_kv_cache_134_gb300 as P
    if c["op"] == "rotary":
        q = P.paged_kv_append_rotary(x["cache"], x["q"], x["k"], x["v"], x["tables"], x["seq"], x["pos"], x["rotary"],
                                     q_weight=x.get("wq"), k_weight=x.get("wk"), eps=1e-6)
        return q, x["pool"]
    if c["op"] == "window":
        return P.paged_decode_attention_window(x["q"], x["cache"], x["tables"], x["lens"], x["scale"], c["window"],
                                               sinks=c["sinks"])
    return P.paged_chunk_attention(x["q"], x["cache"], x["tables"], x["lens"], x["cu"], x["most"], x["scale"],
                                   window=c["window"], sinks=c["sinks"])


# ------------------------------------------------------------------------------------------------ work, definition

def _visible(case):
    """(keys that some query of the batch sees, pairs of query and key), summed over the sequences."""
    lens = _lens(case).tolist()
    new = [1] * len(lens) if case["op"] == "window" else _news(case, _lens(case)).tolist()
    keys = pairs = 0
    for length, n in zip(lens, new):
        w, k = case["window"] or length, case["sinks"] if case["window"] else 0
        first = max(0, length - n - w + 1)
        keys += length - first + min(k, first)
        for p in range(length - n, length):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(k, lo)
    return keys, pairs


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        t = case["seqs"] * case["new"]
        return {"bytes": t * (4 * (hq + 2 * hkv) * d + 12),
                "flops": t * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    keys, pairs = _visible(case)
    rows = case["seqs"] if case["op"] == "window" else int(_news(case, _lens(case)).sum())
    elt = 1 if case["kv"] == "fp8" else 2
    return {"bytes": 2 * keys * hkv * d * elt + 4 * keys // case["bs"] + 4 * rows * hq * d, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    x = _inputs(case, seed)
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    if case["op"] == "rotary":
        f, gain = _frequencies(case["rot"], case["scaled"])
        rot, outs = case["rot"], []
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), x["pos"].double()[:, None] * f.to(DEV)) * gain
        for t, w in ((x["q"], "wq"), (x["k"], "wk")):
            r = t.double()
            if case["norm"]:
                r = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * x[w].double()
            # a pair of elements as one complex number
            if case["pairs"] == "half":
                y = torch.complex(r[..., :rot // 2].contiguous(), r[..., rot // 2:rot].contiguous()) * z[:, None]
                r[..., :rot // 2], r[..., rot // 2:rot] = y.real, y.imag
            else:
                y = torch.complex(r[..., 0:rot:2].contiguous(), r[..., 1:rot:2].contiguous()) * z[:, None]
                r[..., 0:rot:2], r[..., 1:rot:2] = y.real, y.imag
            outs.append(r)
        pool = torch.zeros(x["blocks"], 2, hkv, bs, d, dtype=torch.float64, device=DEV)
        for j, r in enumerate((outs[1], x["v"].double())):
            pool.select(1, j).transpose(1, 2)[x["tables"][x["seq"].long(), x["pos"].long() // bs].long(),
                                              x["pos"].long() % bs] = r
        return outs[0], pool
    lens = x["host_lens"]
    new = x.get("host_new", [1] * len(lens))
    out = torch.empty(x["q"].shape, dtype=torch.float64, device=DEV)
    group, at, row = case["hq"] // hkv, 0, 0
    for length, n in zip(lens, new):
        p = torch.arange(length - n, length, device=DEV)[:, None]
        # the keys that some row sees; of the rest, scores are not formed
        t = torch.arange(length, device=DEV)
        if case["window"]:
            t = t[(t >= length - n - case["window"] + 1) | (t < case["sinks"])]
        seen = _seen(t, p, case["window"], case["sinks"])
        for g in range(hkv):
            kv = []
            for name in ("k", "v"):
                r = x[name][at:at + length, g][t].double()
                if case["kv"] == "fp8":
                    f = x[name + "_scale"][g]
                    r = (x[name][at:at + length, g][t].float() / f).clamp(-448, 448).to(torch.float8_e4m3fn).double() * f.double()
                kv.append(r)
            for h in range(g * group, (g + 1) * group):
                z = (x["q"][row:row + n, h].double() @ kv[0].T * x["scale"]).masked_fill(~seen, -math.inf)
                out[row:row + n, h] = torch.softmax(z, -1) @ kv[1]
        at, row = at + length, row + n
    return out
