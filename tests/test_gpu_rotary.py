"""GPU tests of paged_kv_append_rotary against the formula in 64 bits.

Tolerance: half a step of the model type (plus half its smallest subnormal), and what fp32 loses on the way, taken
relative to |y_a| + |y_b| of the pair: 2^-25 of a turn in the angle (1.9e-7), 2 ulp of sincospif, and for the norm a sum
of 128 squares in two levels (less than 20 roundings, halved by the root), rsqrtf's 2 ulp, two products and the
rotation's three roundings: less than 16 units of 2^-24 in all, 2^-20."""
import numpy as np
import pytest
import torch

import paged_kv_cache_134_gb300 as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

MODEL = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def formula(x, w, eps, pos, rotary):
    """(value, |y_a| + |y_b| of its pair) in 64 bits; x [T, H, D]."""
    x = x.double().cpu().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    r, d = rotary.rotary_dim, x.shape[-1]
    t = pos.double().cpu().numpy()[:, None] * np.array(rotary.inv_freq)
    c, s = (np.cos(t) * rotary.gain)[:, None], (np.sin(t) * rotary.gain)[:, None]
    a = slice(0, r, 2) if rotary.interleaved else slice(0, r // 2)
    b = slice(1, r, 2) if rotary.interleaved else slice(r // 2, r)
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(rotary.gain)
    return y, size


def check(got, want, model):
    y, size = want
    err = np.abs(got.double().cpu().numpy() - y)
    lost = size * 2.0 ** -20
    assert (err <= HALF[model] * (np.abs(y) + lost) + LEAST[model] + lost).all(), err.max()


class Case:
    def __init__(self, n, hq=4, hkv=2, d=128, bs=16, kv="f16", model="f16", far=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        md = MODEL[model]
        self.model, self.hq, self.hkv, self.d, self.n = model, hq, hkv, d, n
        self.qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).to(md).cuda()
        self.q, self.k, self.v = (t.view(n, h, d) for t, h in zip(self.qkv.split([hq * d, hkv * d, hkv * d], 1),
                                                                  (hq, hkv, hkv)))
        self.seqs = max(1, min(3, n))
        self.seq = (torch.arange(n) % self.seqs).to(torch.int32).cuda()
        first = torch.randint(0, 100000, (self.seqs,), generator=g) if far else torch.zeros(self.seqs, dtype=torch.long)
        pos = torch.arange(n) // self.seqs + first[torch.arange(n) % self.seqs]
        self.pos = pos.to(torch.int32).cuda()
        width = int(pos.max()) // bs + 1 if n else 1
        lo = first // bs
        used = [(s, b) for s in range(self.seqs) for b in range(int(lo[s]), int(first[s] + n // self.seqs) // bs + 1)]
        self.nb = len(used) + 2
        order = torch.randperm(self.nb, generator=g)
        t = torch.full((self.seqs, width), -1, dtype=torch.int32)
        for (s, b), i in zip(used, order):
            if b < width:
                t[s, b] = int(i)
        self.tables = t.cuda()
        self.wq = (torch.randn(d, generator=g) * 0.2 + 1).to(md).cuda()
        self.wk = (torch.randn(d, generator=g) * 0.2 + 1).to(md).cuda()
        self.args = (self.nb, bs, hkv, d, kv, model)
        self.ks = (torch.rand(hkv, generator=g) * 0.02 + 0.005).cuda()
        self.cache = self.new_cache()

    def new_cache(self):
        cache = P.KVCache(*self.args[:4], kv_dtype=self.args[4], model_dtype=self.args[5])
        if self.args[4] == "fp8":
            cache.set_scales(self.ks, self.ks)
        cache.view()[0].fill_(0xA5)
        return cache


CASES = [
    # n, hq, hkv, d, bs, kv, model, rot, interleaved, wq, wk, far
    (1, 1, 1, 64, 8, "f16", "f16", 64, False, 0, 0, 0),
    (1, 8, 1, 128, 16, "bf16", "bf16", 128, True, 1, 1, 1),
    (3, 32, 32, 128, 16, "f16", "f16", 128, False, 0, 0, 0),
    (7, 4, 2, 64, 16, "bf16", "bf16", 16, False, 1, 0, 0),
    (33, 32, 8, 128, 32, "bf16", "bf16", 64, True, 1, 1, 1),
    (33, 5, 5, 128, 8, "f16", "f16", 96, False, 0, 1, 0),
    (64, 2, 1, 64, 32, "f16", "f16", 32, True, 0, 0, 1),
    (257, 7, 7, 128, 16, "fp8", "f16", 128, False, 0, 0, 0),
    (130, 8, 2, 64, 16, "fp8", "bf16", 48, True, 1, 1, 0),
    (257, 8, 8, 128, 16, "int4", "f16", 128, False, 1, 1, 0),
    (130, 8, 2, 64, 8, "int4", "bf16", 64, True, 0, 0, 1),
    (1500, 64, 8, 128, 16, "bf16", "bf16", 32, False, 1, 1, 1),
    (2500, 3, 1, 128, 16, "f16", "f16", 112, True, 0, 1, 0),
    (5000, 2, 2, 64, 16, "bf16", "bf16", 64, False, 0, 0, 0),
    (0, 4, 2, 128, 16, "f16", "f16", 128, False, 0, 0, 0),
]


@pytest.mark.parametrize("n,hq,hkv,d,bs,kv,model,rot,inter,wq,wk,far", CASES)
def test_rotation_norm_and_append(n, hq, hkv, d, bs, kv, model, rot, inter, wq, wk, far):
    x = Case(n, hq, hkv, d, bs, kv, model, bool(far))
    r = P.Rotary(rot, interleaved=inter)
    wq, wk = (x.wq if wq else None), (x.wk if wk else None)
    before = x.qkv.clone()
    slots = torch.full((n,), -7, dtype=torch.int64, device="cuda")
    out = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r, q_weight=wq, k_weight=wk,
                                   eps=1e-5, slot_mapping=slots)
    assert x.cache.check_error() == 0
    assert torch.equal(x.qkv, before)  # the projection's output is left as it was
    assert out.shape == (n, hq, d)
    if n == 0:
        return
    check(out, formula(x.q, wq, 1e-5, x.pos, r), model)
    assert torch.equal(slots, P.paged_slot_mapping(x.tables, x.seq, x.pos, bs))
    # the pool, byte for byte: what an append of the rounded rows stores (the rows by the same call, as queries), and
    # nothing else
    rows = P.paged_kv_append_rotary(x.new_cache(), x.k, x.k, x.v, x.tables, x.seq, x.pos, r, q_weight=wk, k_weight=wk,
                                    eps=1e-5)
    check(rows, formula(x.k, wk, 1e-5, x.pos, r), model)
    other = x.new_cache()
    P.paged_kv_append(other, rows, x.v.contiguous(), slots)
    assert torch.equal(x.cache.view()[0], other.view()[0])


def test_in_place_and_contiguous_give_the_same_bits():
    x = Case(40, 8, 2)
    r = P.Rotary(128)
    out = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r, q_weight=x.wq)
    again = P.paged_kv_append_rotary(x.new_cache(), x.q.contiguous(), x.k.contiguous(), x.v.contiguous(), x.tables,
                                     x.seq, x.pos, r, q_weight=x.wq)
    assert torch.equal(out, again)
    kept = x.qkv.clone()
    got = P.paged_kv_append_rotary(x.new_cache(), x.q, x.k, x.v, x.tables, x.seq, x.pos, r, q_weight=x.wq, q_out=x.q)
    assert got is x.q and torch.equal(got, out)
    assert torch.equal(x.qkv[:, 8 * 128:], kept[:, 8 * 128:])  # k and v beside it are not touched


def test_keys_and_values_alone():
    x, r = Case(20), P.Rotary(64)
    assert P.paged_kv_append_rotary(x.cache, None, x.k, x.v, x.tables, x.seq, x.pos, r) is None
    other = x.new_cache()
    P.paged_kv_append_rotary(other, x.q, x.k, x.v, x.tables, x.seq, x.pos, r)
    assert torch.equal(x.cache.view()[0], other.view()[0])


def test_positions_of_the_rotation_and_tokens_without_a_slot():
    x, r = Case(12), P.Rotary(128)
    angles = torch.tensor([0, 1, -1, -4097, 2 ** 24 - 1, 131071, 99999, 5, 6, 7, -131072, 3], dtype=torch.int32).cuda()
    seq, pos = x.seq.clone(), x.pos.clone()
    seq[2], pos[5], seq[7], pos[9] = -1, -3, 99, 2 ** 31 - 1
    out = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, seq, pos, r, rotary_positions=angles)
    assert x.cache.check_error() == 0
    check(out, formula(x.q, None, 0, angles, r), "f16")
    slots = P.paged_slot_mapping(x.tables, seq, pos, 16)
    assert (slots < 0).sum() == 4
    rows = P.paged_kv_append_rotary(x.new_cache(), x.k, x.k, x.v, x.tables, seq, pos, r, rotary_positions=angles)
    other = x.new_cache()
    P.paged_kv_append(other, rows, x.v.contiguous(), slots)
    assert torch.equal(x.cache.view()[0], other.view()[0])


def test_a_table_entry_past_the_pool_is_reported():
    x, r = Case(4), P.Rotary(128)
    x.tables[0, 0] = x.nb
    before = x.cache.view()[0].clone()
    P.paged_kv_append_rotary(x.cache, x.q[:1], x.k[:1], x.v[:1], x.tables, x.seq[:1], x.pos[:1], r)
    assert torch.equal(x.cache.view()[0], before)
    assert x.cache.check_error() == 2


def test_the_largest_position():
    """The angle of position 2^31 - 1, whose product with a frequency 64-bit floats hold to 2^-22 of a turn."""
    x = Case(1, 2, 1)
    f = [k / 2.0 ** 30 * 2 * np.pi for k in range(1, 65)]  # p f = k (2 - 2^-30) turns: -k 2^-30 of one
    r = P.Rotary.from_frequencies(f)
    p = torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda()
    out = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r, rotary_positions=p)
    # sin of at most 64 2^-30 turns is below 4e-7, cos is 1: the rows come back to 2^-20 of their pair
    y = x.q.double().cpu().numpy()
    size = np.abs(y[..., :64]) + np.abs(y[..., 64:])
    check(out, (y, np.concatenate([size, size], -1)), "f16")


def test_zeros_infinities_and_nan_stay_in_their_rows():
    x, r = Case(6), P.Rotary(128)
    x.q[1] = 0
    x.q[2, 1, 5] = float("inf")
    x.k[3, 0, 7] = float("nan")
    out = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r, q_weight=x.wq, k_weight=x.wk,
                                   eps=0.0 + 1e-6)
    assert (out[1] == 0).all()
    bad = ~out.isfinite().all(-1)
    assert bad[2, 1] and bad.sum() == 1
    k, v = P.paged_kv_gather(x.cache, P.paged_slot_mapping(x.tables, x.seq, x.pos, 16))
    bad = ~k.isfinite().all(-1)
    assert bad[3, 0] and bad.sum() == 1 and torch.equal(v, x.v)


def test_graph_and_other_stream():
    x, r = Case(16), P.Rotary(128)
    want = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r)
    cache, out = x.new_cache(), torch.empty(16, 4, 128, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        P.paged_kv_append_rotary(cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r, q_out=out)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.view()[0], x.cache.view()[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.paged_kv_append_rotary(cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, P.Rotary(128), q_out=out)
    cache.view()[0].fill_(0xA5)
    out.zero_()
    x.pos += 1  # inputs are read when the graph runs
    g.replay()
    want = P.paged_kv_append_rotary(x.cache, x.q, x.k, x.v, x.tables, x.seq, x.pos, r)
    assert torch.equal(out, want)


def test_refusals():
    x, r = Case(4), P.Rotary(128)
    call = lambda **k: P.paged_kv_append_rotary(**{**dict(cache=x.cache, q=x.q, k=x.k, v=x.v, block_tables=x.tables,
                                                          seq_ids=x.seq, positions=x.pos, rotary=r), **k})
    wide = torch.zeros(4, 4, 2 * 128, dtype=torch.float16, device="cuda")
    for bad in (dict(k=x.k[:2]), dict(v=x.v[:, :1]), dict(q=x.q[:, :, :64]), dict(seq_ids=x.seq[:2]),
                dict(positions=x.pos[:1]), dict(rotary_positions=x.pos[:1]), dict(q=x.q.cpu()), dict(q=wide[:, :, ::2]),
                dict(q_weight=x.wq[:64]), dict(slot_mapping=torch.zeros(3, dtype=torch.int64, device="cuda")),
                dict(q=None, q_weight=x.wq), dict(q_out=wide), dict(q=wide[:, ::2, :128])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(k=x.k.float()), dict(seq_ids=x.seq.long()), dict(rotary=None), dict(k_weight=x.wk.float())):
        with pytest.raises(TypeError):
            call(**bad)
    odd = torch.zeros(4 * 4 * 128 + 64, dtype=torch.float16, device="cuda")
    for bad in (dict(q=odd[1:1 + 2048].view(4, 4, 128)), dict(eps=-1.0), dict(eps=float("nan")),
                dict(q=odd.as_strided((4, 4, 128), (516, 128, 1))), dict(q_out=odd.as_strided((4, 4, 128), (256, 128, 1)))):
        with pytest.raises(P.PagedKVError) as e:
            call(**bad)
        assert e.value.status == -1
    small = P.KVCache(4, 16, 2, 64, "f16")
    z = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(P.PagedKVError) as e:  # more rotated elements than the head has
        P.paged_kv_append_rotary(small, z, z, z, x.tables, x.seq, x.pos, r)
    assert e.value.status == -4


@pytest.mark.parametrize("n", [1, 5])
def test_outputs_over_the_inputs_are_refused_and_slices_of_one_matrix_are_not(n):
    x, r = Case(n, 4, 2), P.Rotary(128)
    wide = torch.zeros(n, 16, 128, dtype=torch.float16, device="cuda")  # q, k, v and the output side by side
    wide[:, :4], wide[:, 4:6], wide[:, 6:8] = x.q, x.k, x.v
    q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:8]
    call = lambda o, q=q: P.paged_kv_append_rotary(x.cache, q, k, v, x.tables, x.seq, x.pos, r, q_out=o)
    want = call(None).clone()
    for out in (wide[:, 2:6], wide[:, 3:7], wide[:, 5:9], wide[:, 1:5], wide.view(-1)[128:128 + n * 512].view(n, 4, 128)):
        with pytest.raises(P.PagedKVError) as e:
            call(out)
        assert e.value.status == -1
    assert torch.equal(call(wide[:, 8:12]), want) and torch.equal(call(wide[:, 12:]), want)
    assert torch.equal(call(q), want)  # in place
    assert x.cache.check_error() == 0
