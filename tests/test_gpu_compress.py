"""GPU tests of the 4-bit cache (append, read back, decode), the decode with attention mass and the eviction, against
64-bit references.

Every pool is filled with 0xFF first: a read of a slot that no token owns shows as NaN.  Stored bytes, kept positions
and moved rows are compared exactly; attention within half a step of the output type plus what
compress_ref.relative_weight_error derives for the weights."""
import math
import threading

import numpy as np
import pytest
import torch

import compress_ref as R
import paged_kv_cache_134_gb300 as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

TORCH = R.TORCH


class Setup:
    """Sequences of given lengths in a cache of their own, with the stored values in 64 bits."""

    def __init__(self, lens, hq=4, hkv=4, d=128, bs=16, kv="int4", model="f16", seed=0, extra=8, spread=True,
                 num_blocks=None, first=0):
        self.lens, self.hq, self.hkv, self.d, self.bs, self.kv, self.model = list(lens), hq, hkv, d, bs, kv, model
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [(n + bs - 1) // bs for n in self.lens]
        total = sum(need)
        self.nb = num_blocks or total + extra
        order = torch.randperm(total, generator=g, device="cuda").cpu()  # drawn either way: the data stay alike
        order = order if spread else torch.arange(total)
        self.free = [b for b in range(self.nb) if not first <= b < first + total]
        width = max(1, max(need, default=1))
        t = torch.full((len(self.lens), width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            t[i, :n] = order[at:at + n].to(torch.int32) + first
            at += n
        self.tables = t.cuda()
        self.context = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        n = sum(self.lens)
        md = TORCH[model]
        gain = torch.ones(hkv, d, device="cuda")
        gain[:, ::32] = 3.0
        self.k = (torch.randn(n, hkv, d, generator=g, device="cuda") * gain).to(md)
        self.v = torch.randn(n, hkv, d, generator=g, device="cuda").to(md)
        self.q = torch.randn(len(self.lens), hq, d, generator=g, device="cuda").to(md)
        seq = torch.repeat_interleave(torch.arange(len(self.lens)), torch.tensor(self.lens, dtype=torch.long))
        pos = torch.cat([torch.arange(m) for m in self.lens] + [torch.zeros(0, dtype=torch.long)])
        self.slots = (t[seq, pos // bs].long() * bs + pos % bs).cuda() if n else torch.zeros(0, dtype=torch.long).cuda()
        self.scale = 1.0 / math.sqrt(d)
        self.cache = P.KVCache(self.nb, bs, hkv, d, kv_dtype=kv, model_dtype=model)
        self.cache.view()[0].fill_(255)
        if kv == "fp8":
            self.ks = (self.k.float().abs().amax(dim=(0, 2)) / 448).clamp(min=1e-6) if n else torch.ones(hkv).cuda()
            self.vs = (self.v.float().abs().amax(dim=(0, 2)) / 448).clamp(min=1e-6) if n else torch.ones(hkv).cuda()
            self.cache.set_scales(self.ks.contiguous(), self.vs.contiguous())
        if n:
            P.paged_kv_append(self.cache, self.k, self.v, self.slots)

    def stored(self):
        """K and V as the cache holds them, float64 [N, Hkv, D] each."""
        out = []
        for name in ("k", "v"):
            x = getattr(self, name)
            if self.kv == "int4":
                out.append(R.values4(*R.quantise4(R.to64(x), self.model)))
            elif self.kv == "fp8":
                s = (self.ks if name == "k" else self.vs)[:, None]
                out.append(R.to64((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).float()) * R.to64(s))
            else:
                out.append(R.to64(x))
        return out

    def bounds(self, s, big):
        """(relative error of sequence s's softmax weights, error of a unit-weight sum of its V rows)."""
        rel = R.relative_weight_error(big)
        if self.kv == "bf16":
            rel += 2.0 ** -14                              # weights as bf16 hi + lo, each cut off
        if self.kv != "int4" or not self.lens[s]:
            return rel, 0.0
        step = [R.quantise4(R.to64(x[self.rows(s)]), self.model)[1] for x in (self.k, self.v)]
        rel += R.code_alignment(self.d, R.to64(self.q[s]), step[0], self.scale)
        # V: in a product of 16 tokens each keeps its code to 2^-17 of a step at the largest weight: 16 of them
        # lose at most 2^-13 of a step per unit of weight
        return rel, 2.0 ** -13 * float(step[1].max())

    def rows(self, s):
        a = sum(self.lens[:s])
        return slice(a, a + self.lens[s])

    def close(self):
        err = self.cache.check_error()
        self.cache.close()
        return err


def check_attention(x, out, mass=None, old=None, decay=1.0):
    k, v = x.stored()
    q, got = R.to64(x.q), R.to64(out)
    for s, n in enumerate(x.lens):
        ref, p, pv, big = R.attention(q[s], k[x.rows(s)], v[x.rows(s)], x.scale)
        rel, cut = x.bounds(s, big)
        tol = R.HALF_STEP[x.model] * np.abs(ref) * 1.001 + rel * pv + cut + 2.0 ** -24
        err = np.abs(got[s] - ref)
        assert np.all(err <= tol), f"sequence {s} (L {n}): {err.max():.3e}, {(err / tol).max():.2f} of its bound"
        if mass is None:
            continue
        m, before = R.to64(mass[s]), R.to64(old[s])
        add = p.reshape(x.hkv, x.hq // x.hkv, n).sum(1)
        want = before[:, :n] * decay + add
        bound = rel * add + 2.0 ** -22 * np.abs(want)
        assert np.all(np.abs(m[:, :n] - want) <= bound), f"mass of sequence {s}"
        assert np.array_equal(m[:, n:], before[:, n:]), f"mass behind sequence {s} changed"


# ------------------------------------------------------------------------------------------ 4-bit rows

V_ORDER = [0, 2, 4, 6, 1, 3, 5, 7]   # V rows of an octet by place


def int4_rows(raw, hkv, bs, d):
    """Bytes [NB, ...] of a 4-bit pool -> (code bytes [NB, Hkv, 2, bs, D / 2], parameter bytes [NB, Hkv, 2, bs, 4])."""
    nb = raw.shape[0]
    o = raw.reshape(nb, hkv, bs // 8, 8 * (d + 8))
    k = o[..., :4 * d].reshape(nb, hkv, bs // 8, 8, d // 2)
    placed = o[..., 4 * d:8 * d].reshape(nb, hkv, bs // 8, 8, d // 2)
    v = np.empty_like(placed)
    for place, row in enumerate(V_ORDER):
        r = placed[:, :, :, place]
        v[:, :, :, row] = np.roll(r, 32, axis=-1) if d == 128 and place & 2 else r
    par = o[..., 8 * d:].reshape(nb, hkv, bs // 8, 2, 8, 4).transpose(0, 1, 3, 2, 4, 5).reshape(nb, hkv, 2, bs, 4)
    return np.stack([k, v], 2).reshape(nb, hkv, 2, bs, d // 2), par


def int4_parts(cache, model):
    """(codes [NB, Hkv, 2, bs, D], step, low [NB, Hkv, 2, bs] as raw int16) of a 4-bit pool."""
    c, par = int4_rows(cache.view()[0].cpu().numpy().reshape(cache.num_blocks, -1), cache.num_kv_heads,
                       cache.block_size, cache.head_dim)
    par = np.ascontiguousarray(par).view(np.int16)
    w = np.ascontiguousarray(c).view(np.uint16)             # four codes a word, rotated left by three bits
    w = (w >> 3) | (w << 13)
    codes = np.stack([(w >> (4 * i)) & 15 for i in range(4)], -1).astype(np.uint8)
    return codes.reshape(*c.shape[:-1], -1), par[..., 0], par[..., 1]


def model_bits(x, model):
    return torch.from_numpy(np.asarray(x, np.float64)).to(TORCH[model]).view(torch.int16).numpy()


def special_rows(n, hkv, d, model, seed):
    """Rows of every magnitude, constants, single spikes, ties, exact steps, subnormals, NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hkv, d, generator=g) * torch.exp(4 * torch.randn(n, hkv, 1, generator=g))
    x[0] = 1.5
    x[1] = 0.0
    x[1, :, 3] = 8.0
    x[2] = torch.arange(d) % 16 - 7.0
    x[3] = (torch.arange(d) % 31) * 0.5            # half steps: ties go to even
    x[4] = torch.randn(hkv, d, generator=g) * 1e-7  # fp16 subnormals
    x[5, :, 0] = float("nan")
    x[6, :, d - 1] = float("inf")
    x[7, :, 1] = float("-inf")
    x[8] = torch.where(torch.arange(d) % 2 == 0, 60000.0, -60000.0)
    if model == "bf16":
        x[9] = torch.where(torch.arange(d) % 2 == 0, 3e38, -3e38)  # the range overflows
        x[10] = torch.randn(hkv, d, generator=g) * 1e-38
        x[11] = torch.randn(hkv, d, generator=g) * 1e37
    return x.to(TORCH[model]).cuda()


@pytest.mark.parametrize("model", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (3, 128, 16), (8, 64, 32), (32, 128, 8), (40, 128, 16)])
def test_int4_append_stores_the_definition_bit_for_bit(model, hkv, d, bs):
    n = 37
    cache = P.KVCache(9 if bs == 8 else 5, bs, hkv, d, kv_dtype="int4", model_dtype=model)
    cache.view()[0].fill_(255)
    before = cache.view()[0].clone()
    k, v = special_rows(n, hkv, d, model, 1), special_rows(n, hkv, d, model, 2).flip(0)
    slots = torch.randperm(cache.num_blocks * bs, generator=torch.Generator().manual_seed(5))[:n].cuda()
    slots[20] = -1
    P.paged_kv_append(cache, k, v, slots)
    codes, step, low = int4_parts(cache, model)
    owned = np.zeros((cache.num_blocks, bs), bool)
    for j, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        b, o = divmod(slot, bs)
        owned[b, o] = True
        for kv, x in enumerate((k, v)):
            c, s, z = R.quantise4(R.to64(x[j]), model)
            nan = np.isnan(s)
            assert np.array_equal(codes[b, :, kv, o], c), (j, kv)
            assert np.array_equal(step[b, ~nan, kv, o], model_bits(s, model)[~nan])
            lowf = torch.from_numpy(low[b, :, kv, o].copy()).view(TORCH[model]).double().numpy()
            assert np.array_equal(lowf, z, equal_nan=True)
            assert np.array_equal(torch.from_numpy(step[b, :, kv, o].copy()).view(TORCH[model]).isnan().numpy(), nan)
    empty = ~owned
    assert np.all(codes.transpose(0, 3, 1, 2, 4)[empty] == 15) and np.all(step.transpose(0, 3, 1, 2)[empty] == -1)
    kk, vv = P.paged_kv_gather(cache, slots)
    for x, got in ((k, kk), (v, vv)):
        want = R.values4(*R.quantise4(R.to64(x), model)).astype(np.float32)
        want[20] = 0
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want).to(TORCH[model])
        assert torch.equal(torch.nan_to_num(got.cpu(), 7.0), torch.nan_to_num(want, 7.0))
        assert torch.equal(got.cpu().isnan(), want.isnan())
    # a slot past the pool is reported, and nothing moves
    saved = cache.view()[0].clone()
    far = torch.tensor([cache.num_blocks * bs], device="cuda")
    P.paged_kv_append(cache, k[:1], v[:1], far)
    z, _ = P.paged_kv_gather(cache, far)
    assert not z.any() and torch.equal(saved, cache.view()[0]) and not torch.equal(saved, before)
    assert cache.check_error() == 2
    cache.close()


@pytest.mark.parametrize("model", ["f16", "bf16"])
def test_int4_codes_are_those_of_divisions(model):
    """Codes next to and at ties, over every magnitude of the step: the quotients are not divisions in the kernel."""
    n, hkv, d = 512, 4, 128
    g = torch.Generator().manual_seed(9)
    lo, hi = (-20, 12) if model == "f16" else (-120, 120)
    scale = torch.exp2(torch.randint(lo, hi, (n, hkv, 1), generator=g).double())
    steps = torch.randint(1, 64, (n, hkv, 1), generator=g)           # quarter steps of a whole number
    x = torch.randint(0, 61, (n, hkv, d), generator=g) * steps / 256.0 * scale
    x[..., 0], x[..., 1] = 0.0, 15.0 * steps[..., 0] / 64.0 * scale[..., 0]
    x[n // 2:] += torch.randn(n // 2, hkv, 1, generator=g) * scale[n // 2:]   # rounded: next to the ties
    x = x.to(TORCH[model]).cuda()
    cache = P.KVCache(n // 16, 16, hkv, d, kv_dtype="int4", model_dtype=model)
    P.paged_kv_append(cache, x, x.flip(0), torch.arange(n, device="cuda"))
    codes, step, _ = int4_parts(cache, model)
    for kv, rows in enumerate((x, x.flip(0))):
        c, s, _ = R.quantise4(R.to64(rows), model)
        got = codes[:, :, kv].transpose(0, 2, 1, 3).reshape(n, hkv, d)
        assert np.array_equal(step[:, :, kv].transpose(0, 2, 1).reshape(n, hkv), model_bits(s, model))
        assert np.array_equal(got, c)
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("model,hkv,d,bs", [("f16", 2, 128, 16), ("bf16", 4, 64, 8)])
def test_int4_append_at_and_packed_prefill_write_the_same_bytes(model, hkv, d, bs):
    x = Setup([19, 1, 40], hkv=hkv, hq=hkv * 2, d=d, bs=bs, model=model)
    want = x.cache.view()[0].clone()
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(x.lens)).int().cuda()
    pos = torch.cat([torch.arange(n) for n in x.lens]).int().cuda()
    x.cache.view()[0].fill_(255)
    slots = torch.empty_like(x.slots)
    P.paged_kv_append_at(x.cache, x.k, x.v, x.tables, seq, pos, slots)
    assert torch.equal(slots, x.slots) and torch.equal(want, x.cache.view()[0])
    x.cache.view()[0].fill_(255)
    cu = torch.tensor([0, 19, 20, 60], dtype=torch.int32, device="cuda")
    q = torch.randn(60, hkv * 2, d, device="cuda").to(TORCH[model])
    out = P.packed_prefill_attention(q, x.k, x.v, cu, 40, x.tables, x.cache, x.scale)
    assert torch.equal(want, x.cache.view()[0])
    k, v = R.to64(x.k), R.to64(x.v)
    for s in range(3):
        a = int(cu[s])
        for r in (0, x.lens[s] // 2, x.lens[s] - 1):
            ref, _, pv, big = R.attention(R.to64(q[a + r]), k[a:a + r + 1], v[a:a + r + 1], x.scale)
            # the prefill's own accuracy: fp16 weights (2^-11), or bf16 hi + lo
            tol = R.HALF_STEP[model] * np.abs(ref) + (R.relative_weight_error(big) + 2.0 ** -11) * pv + 1e-6
            assert np.all(np.abs(R.to64(out[a + r]) - ref) <= tol)
    assert x.close() == 0


@pytest.mark.parametrize("kv", ["f16", "bf16", "fp8", "int4"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (5, 128, 8)])
def test_gather_reads_back_what_the_cache_holds(kv, hkv, d, bs):
    x = Setup([23, 9], hkv=hkv, hq=hkv, d=d, bs=bs, kv=kv, model=kv if kv in TORCH else "bf16")
    pick = torch.randperm(32, generator=torch.Generator().manual_seed(1)).cuda()
    k, v = P.paged_kv_gather(x.cache, x.slots[pick].contiguous())
    for got, ref in zip((k, v), x.stored()):
        want = torch.from_numpy(ref.astype(np.float32)).to(TORCH[x.model])[pick.cpu()]
        assert torch.equal(got.cpu(), want)
    e = P.paged_kv_gather(x.cache, x.slots[:0])
    assert e[0].shape == (0, hkv, d)
    assert x.close() == 0


@pytest.mark.parametrize("bs,d", [(8, 64), (16, 128), (32, 64)])
def test_int4_blocks_copy_and_swap_whole(bs, d):
    x = Setup([50, 20], hkv=3, hq=3, d=d, bs=bs, extra=6)
    used = x.tables[x.tables >= 0]
    dst = torch.tensor(x.free[: min(4, used.numel())], dtype=torch.int32, device="cuda")
    src = used[: dst.numel()].contiguous()
    P.paged_block_copy(x.cache, src, dst)
    pool = x.cache.view()[0].view(x.nb, -1)
    assert pool.shape[1] == x.cache.block_bytes and torch.equal(pool[src.long()], pool[dst.long()])
    want = pool[src.long()].clone()
    host = P.paged_block_swap_out(x.cache, src)
    torch.cuda.synchronize()
    pool[src.long()] = 255
    P.paged_block_swap_in(x.cache, src, host)
    assert torch.equal(pool[src.long()], want)
    assert x.close() == 0


# ------------------------------------------------------------------------------------------ decode

LENS = [0, 1, 7, 8, 9, 16, 17, 63, 64, 65, 130, 300]
SHAPES = [(1, 1, 64, 8, "f16"), (4, 2, 128, 16, "f16"), (8, 2, 64, 32, "bf16"), (16, 2, 128, 8, "bf16"),
          (3, 3, 128, 32, "bf16"), (8, 1, 128, 16, "f16")]


@pytest.mark.parametrize("hq,hkv,d,bs,model", SHAPES)
def test_int4_decode(hq, hkv, d, bs, model):
    x = Setup(LENS, hq=hq, hkv=hkv, d=d, bs=bs, model=model, seed=hq)
    out = torch.full_like(x.q, float("nan"))
    P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale, out=out)
    check_attention(x, out)
    again = P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale)
    assert torch.equal(out, again)
    fixed = torch.empty_like(out)
    P.paged_decode_attention_noalloc(x.q, x.cache, x.tables, x.context, x.scale, fixed)
    assert torch.equal(out, fixed)
    assert x.close() == 0


@pytest.mark.parametrize("hq,hkv,lens", [(8, 1, [5000]), (32, 8, [2500, 3, 1025]), (2, 2, [9001])])
def test_int4_decode_long_rows_in_many_splits(hq, hkv, lens):
    x = Setup(lens, hq=hq, hkv=hkv, model="bf16", bs=32, seed=7)
    check_attention(x, P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale))
    assert x.close() == 0


@pytest.mark.parametrize("hq,hkv,lens,pad", [(8, 8, [9001, 40], 0), (16, 2, [3000] * 5 + [0, 1], 0), (4, 4, [33, 7, 0, 64], 600)])
def test_int4_decode_without_allocation_captured(hq, hkv, lens, pad):
    """The fixed scratch: joined by a merge launch, by the last CTA, and single units under wide tables; twice in a graph."""
    x = Setup(lens, hq=hq, hkv=hkv, model="f16", seed=12)
    t = torch.nn.functional.pad(x.tables, (0, pad), value=-1).contiguous()
    want = P.paged_decode_attention(x.q, x.cache, t, x.context, x.scale)
    check_attention(x, want)
    outs = [torch.zeros_like(x.q) for _ in range(2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            P.paged_decode_attention_noalloc(x.q, x.cache, t, x.context, x.scale, o)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    assert x.close() == 0


def test_int4_decode_does_not_depend_on_placement_or_on_other_lengths():
    a = Setup([700, 45, 200], seed=3)
    b = Setup([700, 45, 200], seed=3, spread=False)
    oa = P.paged_decode_attention(a.q, a.cache, a.tables, a.context, a.scale)
    ob = P.paged_decode_attention(b.q, b.cache, b.tables, b.context, b.scale)
    assert torch.equal(oa, ob)
    short = a.context.clone()
    short[0] = 1
    oc = P.paged_decode_attention(a.q, a.cache, a.tables, short, a.scale)
    assert torch.equal(oa[1:], oc[1:])
    assert a.close() == 0 and b.close() == 0


@pytest.mark.parametrize("kv,model", [("int4", "f16"), ("int4", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("f16", "f16"),
                                      ("bf16", "bf16")])
@pytest.mark.parametrize("hq,hkv,d,bs", [(2, 2, 64, 8), (4, 2, 128, 16), (8, 2, 128, 32), (8, 1, 64, 16),
                                         (16, 2, 128, 8)])
def test_decode_with_attention_mass(kv, model, hq, hkv, d, bs):
    x = Setup(LENS, hq=hq, hkv=hkv, d=d, bs=bs, kv=kv, model=model, seed=hq + d)
    mass = torch.rand(len(LENS), hkv, 311, device="cuda")
    old = mass.clone()
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass)
    check_attention(x, out, mass, old)
    mid = mass.clone()
    out2 = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass, decay=0.5)
    check_attention(x, out2, mass, mid, 0.5)
    assert torch.equal(out, out2)
    m3 = mid.clone()
    P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, m3, decay=0.0)
    assert torch.allclose(m3[-1, :, :300].sum(-1), torch.full((hkv,), hq / hkv, device="cuda"), rtol=1e-4)
    assert x.close() == 0


SHORT = [0, 1, 2, 7, 8, 9, 16, 17, 31, 32, 32, 5]


@pytest.mark.parametrize("kv,model", [("int4", "f16"), ("int4", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("f16", "f16"),
                                      ("bf16", "bf16")])
@pytest.mark.parametrize("group,hkv,d,bs", [(1, 3, 128, 8), (2, 2, 64, 16), (4, 1, 128, 32), (4, 2, 64, 8), (8, 2, 128, 16)])
def test_mass_of_short_rows(kv, model, group, hkv, d, bs):
    """Tables of at most 32 tokens: a warp takes a row (of eight heads only where the rows are many)."""
    x = Setup(SHORT * (18 if group == 8 else 1), hq=group * hkv, hkv=hkv, d=d, bs=bs, kv=kv, model=model, seed=group)
    if group == 8 and kv != "f16":
        assert len(x.lens) * hkv < 608  # few rows here; many below
    mass = torch.rand(len(x.lens), hkv, 33, device="cuda")
    old = mass.clone()
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass, decay=0.5)
    check_attention(x, out, mass, old, 0.5)
    again = old.clone()
    assert torch.equal(out, P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, again, decay=0.5))
    assert torch.equal(mass, again)
    assert x.close() == 0


@pytest.mark.parametrize("group,d,bs", [(1, 128, 16), (4, 64, 8), (8, 128, 8)])
@pytest.mark.parametrize("kv", ["int4", "fp8", "f16"])
def test_many_short_rows(kv, group, d, bs):
    x = Setup([(7 * i) % 33 for i in range(170)], hq=4 * group, hkv=4, d=d, bs=bs, kv=kv, model="f16", seed=3)
    mass = torch.zeros(170, 4, 32, device="cuda")
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass)
    check_attention(x, out, mass, torch.zeros_like(mass))
    if kv == "int4":
        check_attention(x, P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale))
    # bad blocks and lengths: reported, their tokens left out
    t = x.tables.clone()
    t[32, 0] = -3
    t[19, 0] = x.nb
    far = x.context.clone()
    far[64] = 1000
    out = P.paged_decode_attention_mass(x.q, x.cache, t, far, x.scale, mass)
    assert x.cache.check_error() == 5
    k, v = x.stored()
    for s in (19, 32):
        stay = list(range(min(bs, x.lens[s]), x.lens[s]))
        ref, _, pv, big = R.attention(R.to64(x.q[s]), k[x.rows(s)][stay], v[x.rows(s)][stay], x.scale)
        rel, cut = x.bounds(s, big)
        assert np.all(np.abs(R.to64(out[s]) - ref) <= R.HALF_STEP["f16"] * np.abs(ref) * 1.001 + rel * pv + cut + 2.0 ** -24)
    x.cache.close()


@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_mass_of_long_rows(kv):
    x = Setup([4001, 5, 0, 1600], hq=8, hkv=2, kv=kv, model="bf16", seed=9)
    mass = torch.zeros(4, 2, 4001, device="cuda")
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass)
    check_attention(x, out, mass, torch.zeros_like(mass))
    assert x.close() == 0


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_a_batch_of_more_sequences_than_a_launch_takes(kv):
    lens = [(i * 37) % 90 for i in range(1500)]
    x = Setup(lens, hq=2, hkv=1, d=64, kv=kv, seed=4)
    mass = torch.zeros(1500, 1, 90, device="cuda")
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass)
    check_attention(x, out, mass, torch.zeros_like(mass))
    if kv == "int4":
        check_attention(x, P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale))
    assert x.close() == 0


def test_offsets_beyond_32_bits():
    bs, hkv, d = 32, 8, 128
    block = hkv * bs * (d + 8)
    nb = (5 << 30) // block
    x = Setup([70, 33], hq=8, hkv=hkv, d=d, bs=bs, num_blocks=nb, first=nb - 5)
    assert int(x.tables.max()) * block > 2 ** 32
    mass = torch.zeros(2, hkv, 70, device="cuda")
    check_attention(x, P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass), mass,
                    torch.zeros_like(mass))
    check_attention(x, P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale))
    dst = torch.arange(2, dtype=torch.int32, device="cuda")[:, None].contiguous()
    kept, lens, _ = P.paged_kv_evict(x.cache, x.tables, x.context, mass, 32, 4, dst)
    check_evicted(x, kept, lens, dst, mass, 32, 4)
    assert x.close() == 0


@pytest.mark.parametrize("step", [1e-5, 1.0, 1e4, 1e30])
def test_int4_values_of_any_magnitude(step):
    """V steps far from 1 (and mixed within a row of tokens) keep their precision."""
    model = "bf16"
    x = Setup([200, 90], hq=4, hkv=2, model=model, seed=2)
    x.v = (x.v.float() * step * torch.exp(torch.randn(x.v.shape[0], 1, 1, device="cuda"))).to(TORCH[model])
    P.paged_kv_append(x.cache, x.k, x.v, x.slots)
    out = P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale)
    k, v = x.stored()
    for s in range(2):
        ref, _, pv, big = R.attention(R.to64(x.q[s]), k[x.rows(s)], v[x.rows(s)], x.scale)
        rel, cut = x.bounds(s, big)
        tol = R.HALF_STEP[model] * np.abs(ref) * 1.001 + rel * pv + cut
        assert np.all(np.abs(R.to64(out[s]) - ref) <= tol)
    assert x.close() == 0


@pytest.mark.parametrize("gain", [1e-20, 1e-3, 1e3])
def test_int4_queries_of_any_magnitude(gain):
    """bf16 queries are scaled into fp16's range and back: scores do not lose by it."""
    x = Setup([130], hq=4, hkv=1, model="bf16", seed=6)
    x.q = (x.q.float() * gain).to(torch.bfloat16)
    x.scale /= gain
    check_attention(x, P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale))
    assert x.close() == 0


def test_nan_and_infinity_stay_in_their_sequence():
    x = Setup([40, 40], hq=2, hkv=2, seed=8)
    k = x.k.clone()
    k[50, 0, 3] = float("inf")
    P.paged_kv_append(x.cache, k, x.v, x.slots)
    out = P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1, 0]).all() and torch.isfinite(out[1, 1]).all()
    assert x.close() == 0


@pytest.mark.parametrize("kv", ["f16", "fp8", "int4"])
def test_bad_blocks_and_lengths_are_reported_and_their_tokens_left_out(kv):
    x = Setup([100, 64, 30], hq=4, hkv=2, kv=kv, seed=5)
    t = x.tables.clone()
    t[0, 2] = 10 ** 6
    t[1, 3] = -7
    mass = torch.zeros(3, 2, 100, device="cuda")
    out = P.paged_decode_attention_mass(x.q, x.cache, t, x.context, x.scale, mass)
    assert x.cache.check_error() == 1
    k, v = x.stored()
    for s, gone in ((0, range(32, 48)), (1, range(48, 64))):
        stay = [i for i in range(x.lens[s]) if i not in gone]
        ref, p, pv, big = R.attention(R.to64(x.q[s]), k[x.rows(s)][stay], v[x.rows(s)][stay], x.scale)
        rel, cut = x.bounds(s, big)
        tol = R.HALF_STEP[x.model] * np.abs(ref) * 1.001 + rel * pv + cut
        assert np.all(np.abs(R.to64(out[s]) - ref) <= tol)
        assert not mass[s][:, list(gone)].any()
    # a length past the tables or the mass rows is cut to them
    far = x.context.clone()
    far[2] = 10 ** 9
    P.paged_decode_attention_mass(x.q, x.cache, x.tables[:, :1].contiguous(), far, x.scale, mass)
    assert x.cache.check_error() == 4
    if kv == "int4":
        P.paged_decode_attention(x.q, x.cache, x.tables[:, :2].contiguous(), x.context, x.scale)
        assert x.cache.check_error() == 4
    x.cache.close()


# ------------------------------------------------------------------------------------------ eviction

def check_evicted(x, kept, new_lens, dst, mass, budget, recent, new_mass=None):
    """kept, lengths and mass against the sort; the rows' stored values against the source's."""
    k, v = x.stored()
    hk, m = kept.cpu().numpy(), mass.cpu().numpy()
    assert new_lens.tolist() == [min(n, budget) for n in x.lens]
    slots, want = [], []
    for s, n in enumerate(x.lens):
        for h in range(x.hkv):
            ref = R.evict(m[s, h], n, budget, recent)
            assert hk[s, h, :len(ref)].tolist() == ref and np.all(hk[s, h, len(ref):] == -1), (s, h)
            if new_mass is not None:
                nm = new_mass[s, h].cpu().numpy()
                assert np.array_equal(nm[:len(ref)], m[s, h, ref], equal_nan=True) and not nm[len(ref):].any()
        for j in range(min(n, budget)):
            slots.append(int(dst[s, j // x.bs]) * x.bs + j % x.bs)
            base = x.rows(s).start
            want.append([[a[base + hk[s, h, j], h] for h in range(x.hkv)] for a in (k, v)])
    if slots:
        got = P.paged_kv_gather(x.cache, torch.tensor(slots, device="cuda"))
        for i in range(2):
            ref = torch.from_numpy(np.array([w[i] for w in want]).astype(np.float32)).to(TORCH[x.model])
            assert torch.equal(got[i].cpu(), ref)
    return slots


def dst_tables(x, budget, spare=0):
    width = max(1, max((min(n, budget) + x.bs - 1) // x.bs for n in x.lens))
    t = torch.full((len(x.lens), width), -1, dtype=torch.int32)
    at = spare
    for s, n in enumerate(x.lens):
        need = (min(n, budget) + x.bs - 1) // x.bs
        t[s, :need] = torch.tensor(x.free[at:at + need], dtype=torch.int32)
        at += need
    return t.cuda()


EVICT = [("f16", "f16", 2, 64, 8), ("bf16", "bf16", 3, 128, 16), ("fp8", "bf16", 2, 128, 32), ("fp8", "f16", 1, 64, 8),
         ("int4", "f16", 2, 128, 16), ("int4", "bf16", 3, 64, 8), ("int4", "f16", 1, 64, 32), ("f16", "f16", 1, 128, 32)]


@pytest.mark.parametrize("kv,model,hkv,d,bs", EVICT)
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 5), (33, 33), (100, 0), (500, 7)])
def test_evict(kv, model, hkv, d, bs, budget, recent):
    x = Setup([0, 1, 16, 17, 100, 33, 300], hq=hkv, hkv=hkv, d=d, bs=bs, kv=kv, model=model, extra=80, seed=budget)
    g = torch.Generator(device="cuda").manual_seed(recent)
    mass = torch.rand(7, hkv, 307, generator=g, device="cuda")
    mass[4] = (mass[4] * 4).floor()                        # many ties
    mass[6, :, ::7] = float("nan")
    mass[6, :, 1::7] = -mass[6, :, 1::7]
    mass[6, :, 2::7] = 0.0
    mass[6, :, 3::7] = -0.0
    mass[6, :, 5] = float("inf")
    dst = dst_tables(x, budget)
    before = x.cache.view()[0].clone().view(x.nb, -1)
    kept, lens, new = P.paged_kv_evict(x.cache, x.tables, x.context, mass, budget, recent, dst)
    slots = check_evicted(x, kept, lens, dst, mass, budget, recent, new)
    after = x.cache.view()[0].view(x.nb, -1)
    used = set(dst[dst >= 0].tolist())
    same = [b for b in range(x.nb) if b not in used]
    assert torch.equal(before[same], after[same])          # the old blocks and the free ones
    # slots behind a new length hold what they held
    tail = [b * bs + o for b in used for o in range(bs) if b * bs + o not in set(slots)]
    if tail:
        raw = after.cpu().numpy()
        for slot in tail:
            b, o = divmod(slot, bs)
            if kv == "int4":
                codes, par = int4_rows(raw[b:b + 1], hkv, bs, d)
                assert (codes[:, :, :, o] == 255).all() and (par[:, :, :, o] == 255).all()
            else:
                assert (raw[b].reshape(2, hkv, bs, -1)[:, :, o] == 255).all()
    assert x.close() == 0


def test_evict_long_rows_and_given_outputs():
    x = Setup([20001, 9000], hq=1, hkv=1, d=64, kv="f16", extra=400, bs=32, seed=1)
    mass = torch.rand(2, 1, 20001, device="cuda").pow(9)
    mass[1] = 0.25                                         # every candidate ties
    dst = dst_tables(x, 5000)
    kept = torch.empty(2, 1, 5000, dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    new = torch.full((2, 1, 5003), 7.0, device="cuda")
    got = P.paged_kv_evict(x.cache, x.tables, x.context, mass, 5000, 1001, dst, kept=kept, new_lens=lens, new_mass=new)
    assert got[0] is kept and got[1] is lens and got[2] is new
    check_evicted(x, kept, lens, dst, mass, 5000, 1001, new)
    assert x.close() == 0


@pytest.mark.parametrize("kv,model,hkv,d,bs", EVICT)
@pytest.mark.parametrize("budget,recent", [(7, 0), (700, 64), (4999, 4999)])
def test_evict_few_rows_of_very_different_lengths(kv, model, hkv, d, bs, budget, recent):
    """Rows that several CTAs share: long, one behind the budget, at it, one token, none; masses with NaN, infinities,
    zeros of both signs and runs of ties."""
    x = Setup([9003, budget + 1, budget, 1, 0], hq=hkv, hkv=hkv, d=d, kv=kv, model=model, bs=bs, seed=21,
              extra=5 * ((5000 + bs) // bs + 1))
    g = torch.Generator(device="cuda").manual_seed(3)
    mass = torch.rand(5, hkv, 9003, generator=g, device="cuda").pow(6)
    mass[0, :, 100:4000:7] = float("nan")
    mass[0, :, 5000:5100] = float("inf")
    mass[0, :, 6000:6500] = 0.0
    mass[0, :, 6500:7000] = -0.0
    mass[0, :, 7000:8000] = 0.5
    dst = dst_tables(x, budget)
    kept, lens, new = P.paged_kv_evict(x.cache, x.tables, x.context, mass, budget, recent, dst)
    check_evicted(x, kept, lens, dst, mass, budget, recent, new)
    far = x.context.clone()
    far[0] = 9004
    kept, lens, new = P.paged_kv_evict(x.cache, x.tables, far, mass, budget, recent, dst)
    assert x.cache.check_error() == 4
    assert lens.tolist() == [0, budget, budget, 1, 0] and (kept[0] == -1).all() and not new[0].any()
    x.cache.close()


def test_evict_reports_bad_blocks_and_lengths():
    x = Setup([40, 40, 40], hq=1, hkv=1, d=64, extra=20, seed=1)
    mass = torch.rand(3, 1, 40, device="cuda")
    dst = dst_tables(x, 16)
    bad = dst.clone()
    bad[0, 0] = x.nb
    t = x.tables.clone()
    t[1, 0] = -5
    P.paged_kv_evict(x.cache, t, x.context, mass, 16, 2, bad)
    assert x.cache.check_error() == 1
    far = x.context.clone()
    far[1] = 41 + x.bs * 2
    far[2] = -3
    kept, lens, new = P.paged_kv_evict(x.cache, x.tables, far, mass, 16, 2, dst)
    assert x.cache.check_error() == 4
    assert lens.tolist() == [16, 0, 0] and (kept[1:] == -1).all() and not new[1:].any()
    x.cache.close()


# ------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("kv,model", [("int4", "bf16"), ("f16", "f16")])
def test_decode_evict_and_decode_on(kv, model):
    """Steps with mass, a cut to the budget, the old blocks reused, and decoding on over what stayed."""
    x = Setup([90, 37, 150], hq=4, hkv=2, kv=kv, model=model, extra=40, seed=11)
    mass = torch.zeros(3, 2, 160, device="cuda")
    for _ in range(3):
        old = mass.clone()
        out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass)
        check_attention(x, out, mass, old)
        x.q = torch.randn_like(x.q)
    budget, recent = 48, 16
    dst = dst_tables(x, budget + 16)
    k, v = x.stored()
    kept, lens, mass2 = P.paged_kv_evict(x.cache, x.tables, x.context, mass, budget, recent, dst)
    check_evicted(x, kept, lens, dst, mass, budget, recent, mass2)
    x.cache.view()[0].view(x.nb, -1)[x.tables[x.tables >= 0].long()] = 255   # the old blocks are anybody's now
    # the next token of each sequence, then attention over what stayed and it
    nk, nv = torch.randn(2, 3, 2, 128, device="cuda").to(TORCH[model])
    P.paged_kv_append_at(x.cache, nk, nv, dst, torch.arange(3, dtype=torch.int32, device="cuda"), lens)
    now = lens + 1
    out = P.paged_decode_attention_mass(x.q, x.cache, dst, now, x.scale, mass2)
    hk = kept.cpu().numpy()
    new = [R.values4(*R.quantise4(R.to64(t), model)) if kv == "int4" else R.to64(t) for t in (nk, nv)]
    for s in range(3):
        n, base = int(lens[s]), x.rows(s).start
        kk, vv = [np.concatenate([np.stack([a[base + hk[s, h, :n], h] for h in range(2)], 1), b[s:s + 1]])
                  for a, b in ((k, new[0]), (v, new[1]))]
        ref, p, pv, big = R.attention(R.to64(x.q[s]), kk, vv, x.scale)
        rel, cut = x.bounds(s, big)
        tol = R.HALF_STEP[model] * np.abs(ref) * 1.001 + 1.5 * (rel * pv + cut)  # (the new token's step besides)
        assert np.all(np.abs(R.to64(out[s]) - ref) <= tol)
        # the new token started from the zero behind the compacted mass
        got = R.to64(mass2[s, :, n])
        assert np.all(np.abs(got - p.reshape(2, 2, n + 1).sum(1)[:, n]) <= 1e-4)
    assert x.close() == 0


@pytest.mark.parametrize("kv", ["int4", "bf16"])
def test_captured_and_replayed(kv):
    """A step captured before any warm-up call (its workspace is allocated during the capture), replayed on new
    inputs while an eager call of another size runs on the same stream in between."""
    x = Setup([700, 300, 5], hq=8, hkv=2, kv=kv, model="bf16", extra=60, seed=13)
    big = Setup([3000], hq=8, hkv=2, kv=kv, model="bf16", seed=14)
    mass = torch.zeros(3, 2, 700, device="cuda")
    dst = dst_tables(x, 128)
    out = torch.empty_like(x.q)
    kept = torch.empty(3, 2, 128, dtype=torch.int32, device="cuda")
    lens = torch.empty(3, dtype=torch.int32, device="cuda")
    new = torch.empty(3, 2, 700, device="cuda")
    k2, v2 = torch.empty_like(x.k), torch.empty_like(x.v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.paged_kv_append(x.cache, x.k, x.v, x.slots)
        P.paged_kv_gather(x.cache, x.slots, k2, v2)
        P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, mass, out=out)
        P.paged_kv_evict(x.cache, x.tables, x.context, mass, 128, 32, dst, kept=kept, new_lens=lens, new_mass=new)
    for i in range(2):
        x.q.normal_()
        x.k.normal_()
        old = mass.clone()
        g.replay()
        other = torch.zeros(1, 2, 3000, device="cuda")
        P.paged_decode_attention_mass(big.q, big.cache, big.tables, big.context, big.scale, other)
        P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, old.clone())
        torch.cuda.synchronize()
        check_attention(x, out, mass, old)
        check_evicted(x, kept, lens, dst, mass, 128, 32, new)
    assert x.close() == 0 and big.close() == 0


@pytest.mark.parametrize("kv", ["int4", "f16"])
def test_two_streams_and_two_graphs_of_one_cache_at_once(kv):
    lens = [[2000, 1500], [1800, 900]]
    x = Setup(lens[0] + lens[1], hq=8, hkv=2, kv=kv, model="f16", seed=15)
    parts = []
    for i in range(2):
        sl = slice(2 * i, 2 * i + 2)
        parts.append(dict(q=x.q[sl].contiguous(), t=x.tables[sl].contiguous(), n=x.context[sl].contiguous(),
                          out=torch.empty_like(x.q[sl]), m=torch.zeros(2, 2, 2000, device="cuda"),
                          st=torch.cuda.Stream()))

    def call(p):
        P.paged_decode_attention_mass(p["q"], x.cache, p["t"], p["n"], x.scale, p["m"], decay=0.0, out=p["out"])

    for p in parts:
        call(p)
    torch.cuda.synchronize()
    want = [(p["out"].clone(), p["m"].clone()) for p in parts]
    for p in parts:
        p["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(p["g"]):
            call(p)
    for mode in ("streams", "graphs"):
        for p in parts:
            p["out"].fill_(float("nan"))
            p["m"].fill_(3.0)
        torch.cuda.synchronize()
        for _ in range(20):
            for p in parts:
                with torch.cuda.stream(p["st"]):
                    p["g"].replay() if mode == "graphs" else call(p)
        torch.cuda.synchronize()
        for p, (o, m) in zip(parts, want):
            assert torch.equal(p["out"], o) and torch.equal(p["m"][0, :, :int(p["n"][0])], m[0, :, :int(p["n"][0])])
    assert x.close() == 0


def test_two_host_threads_on_one_stream():
    """A call is two launches over the stream's workspace: another thread's do not come between them."""
    x = Setup([3000, 2000, 1500, 700], hq=8, hkv=2, kv="int4", model="f16", seed=18)
    parts = [dict(q=x.q[i:i + 2].contiguous(), t=x.tables[i:i + 2].contiguous(), n=x.context[i:i + 2].contiguous(),
                  m=torch.zeros(2, 2, 3000, device="cuda")) for i in (0, 2)]

    def call(p, out):
        P.paged_decode_attention_mass(p["q"], x.cache, p["t"], p["n"], x.scale, p["m"], decay=0.0, out=out)

    want = []
    for p in parts:
        out = torch.empty_like(p["q"])
        call(p, out)
        want.append((out, p["m"].clone()))
    torch.cuda.synchronize()
    outs = [[torch.empty_like(p["q"]) for _ in range(200)] for p in parts]
    threads = [threading.Thread(target=lambda p=p, o=o: [call(p, out) for out in o]) for p, o in zip(parts, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for p, o, (out, m) in zip(parts, outs, want):
        assert all(torch.equal(got, out) for got in o) and torch.equal(p["m"], m)
    assert x.close() == 0


def test_reserved_workspace_leaves_no_allocation_to_the_call():
    x = Setup([3000, 50], hq=8, hkv=2, model="bf16", seed=16)
    P.paged_decode_attention_noalloc(x.q, x.cache, x.tables, x.context, x.scale, torch.empty_like(x.q))  # loads code
    x.cache.reserve(2, 8, x.tables.shape[1])
    out = torch.empty_like(x.q)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    P.paged_decode_attention(x.q, x.cache, x.tables, x.context, x.scale, out=out)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    check_attention(x, out)
    assert x.close() == 0


def test_reserved_workspace_covers_smaller_calls():
    """No call of fewer sequences, heads or blocks than reserved asks for more than what was reserved."""
    width, seqs = 700, 160
    tables = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    q = torch.randn(seqs, 16, 128, device="cuda").bfloat16()

    def taken():  # device memory that torch does not hold
        torch.cuda.synchronize()
        return -torch.cuda.mem_get_info()[0] - torch.cuda.memory_reserved()

    for reserved in (False, True):  # (the first cache's calls load the code)
        x = Setup([1], hq=4, hkv=2, d=128, model="bf16", bs=8, extra=0)
        if reserved:
            x.cache.reserve(seqs, 16, width)
        before = taken()
        for n in (160, 1, 2, 3, 7, 20, 41, 80, 101):
            for w in (700, 5, 17, 33, 62, 130, 333, 512):
                for hq in (16, 2, 4):
                    P.paged_decode_attention(q[:n, :hq].contiguous(), x.cache, tables[:n, :w].contiguous(),
                                             lens[:n].contiguous(), 1.0)
        grown = taken() - before
        assert grown == 0 if reserved else grown > 0
        assert x.close() == 0


# ------------------------------------------------------------------------------------------ refusals

def test_refusals():
    x = Setup([20, 30], hq=4, hkv=2, extra=10, seed=1)
    c = x.cache
    mass = torch.zeros(2, 2, 32, device="cuda")
    dst = dst_tables(x, 16)
    ones = torch.ones(2, device="cuda")
    with pytest.raises(P.PagedKVError):
        c.set_scales(ones, ones)
    with pytest.raises(P.PagedKVError) as e:
        P.paged_decode_attention_cascade(x.q, c, x.tables, x.context, 16, x.scale)
    assert e.value.status == -4
    with pytest.raises(P.PagedKVError) as e:
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        P.paged_prefill_attention(x.q, x.k[:2], x.v[:2], cu, x.context, 1, x.tables, c, x.scale)
    assert e.value.status == -4
    bad = [
        lambda: P.paged_kv_gather(c, x.slots.int()),
        lambda: P.paged_kv_gather(c, x.slots, k=torch.empty(50, 2, 64, dtype=torch.float16, device="cuda")),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, x.scale, mass.half()),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, x.scale, mass[:1]),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, x.scale, mass, decay=1.5),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, x.scale, mass, decay=float("nan")),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, float("nan"), mass),
        lambda: P.paged_decode_attention_mass(x.q[:, :3].contiguous(), c, x.tables, x.context, x.scale, mass),
        lambda: P.paged_decode_attention_mass(x.q, c, x.tables, x.context, x.scale, mass[:, :, ::2]),
        lambda: P.paged_decode_attention_mass(x.q.bfloat16(), c, x.tables, x.context, x.scale, mass),
        lambda: P.paged_decode_attention_mass(x.q.cpu(), c, x.tables, x.context, x.scale, mass),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 0, 0, dst),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, 17, dst),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, -1, dst),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, (1 << 32) + 2, dst),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, (1 << 32) + 16, 2, dst),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 30, 2, dst),               # destination too narrow
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, 2, dst, new_mass=mass),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, 2, dst, new_lens=x.context),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, 2, dst[:1]),
        lambda: P.paged_kv_evict(c, x.tables, x.context, mass, 16, 2, dst, new_mass=torch.zeros(2, 2, 8).cuda()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, P.PagedKVError)):
            call()
            pytest.fail(f"call {i} went through")
    kept, lens, new = P.paged_kv_evict(c, x.tables, x.context, mass, 16, 2, dst)
    long = P.binding.lib().paged_kv_evict(c.handle, x.tables.data_ptr(), 1 << 30, x.context.data_ptr(), 2, mass.data_ptr(),
                                          1 << 31, 16, 2, dst.data_ptr(), dst.shape[1], kept.data_ptr(), lens.data_ptr(),
                                          new.data_ptr(), new.shape[2], None)
    assert long == -4
    # what a refused call leaves behind works
    check_attention(x, P.paged_decode_attention(x.q, c, x.tables, x.context, x.scale))
    assert x.close() == 0


def test_no_room_for_any_token():
    """Mass rows or tables of no tokens: every length is cut to 0 and reported, outputs are zero rows."""
    x = Setup([5, 0], hq=2, hkv=2, kv="f16", model="f16", seed=1)
    out = P.paged_decode_attention_mass(x.q, x.cache, x.tables, x.context, x.scale, torch.zeros(2, 2, 0, device="cuda"))
    assert not out.any() and x.cache.check_error() == 4
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    out = P.paged_decode_attention_mass(x.q, x.cache, none, x.context, x.scale, torch.zeros(2, 2, 9, device="cuda"))
    assert not out.any() and x.cache.check_error() == 4
    kept, lens, new = P.paged_kv_evict(x.cache, none, x.context, torch.zeros(2, 2, 9, device="cuda"), 3, 1, none)
    assert (kept == -1).all() and not lens.any() and not new.any() and x.cache.check_error() == 4
    x.cache.close()


def test_empty_batches():
    x = Setup([5], hq=2, hkv=2, seed=1)
    e = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    n = torch.zeros(0, dtype=torch.int32, device="cuda")
    m = torch.zeros(0, 2, 8, device="cuda")
    assert P.paged_decode_attention_mass(x.q[:0], x.cache, e, n, 1.0, m).shape == (0, 2, 128)
    kept, lens, new = P.paged_kv_evict(x.cache, e, n, m, 4, 1, e)
    assert kept.shape == (0, 2, 4) and lens.numel() == 0 and new.shape == (0, 2, 8)
    assert x.close() == 0
