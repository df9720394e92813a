"""GPU tests of paged_chunk_attention against 64 bits: drafted tokens, pieces of prompts and single tokens, with and
without a window, over 16-bit and E4M3 caches."""
import numpy as np
import pytest
import torch

import paged_kv_cache_134_gb300 as P
import seen_ref as R
from seen_setup import MODEL, Setup

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def weights(x, few=False):
    # (over an E4M3 cache the products run on fp16 whatever the model's type: codes and a scaled q are exact in it)
    if few and x.model == "f16":  # a pair of fp16: 2^-22, as good as fp32 here
        return dict(p="f32")
    return dict(p="pair" if x.kv == "bf16" else "f16")


def positions(length, n):
    return list(range(length - n, length))


def chunks(x, new):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    q, q64 = x.queries(int(sum(new)))
    return cu, q, q64


def run(x, new, window=0, sinks=0, most=None, hidden=True, few=False):
    """The call on sequences whose last new[i] tokens are the queries, checked row by row; what no row of a
    sequence sees is taken off the tables or spoilt first."""
    cu, q, q64 = chunks(x, new)
    for i, (n, m) in enumerate(zip(x.lens, new)):
        if not hidden or not window:
            break
        # (the first tile's rows see the most; later tiles' hidden blocks are in some row's sight)
        low = max(0, n - m - window + 1)
        out = [t for t in range(n) if t < low and t >= sinks]
        blocks = {t // x.bs for t in out if all(u in range(max(sinks, 0), low) for u in
                                                range(t // x.bs * x.bs, min(n, (t // x.bs + 1) * x.bs)))}
        for b in blocks:
            x.tables[i, b] = -1
        x.spoil(i, [t for t in out if t // x.bs not in blocks])
    got = P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, most or max(max(new), 1), R.scale_of(x.d),
                                  window=window, sinks=sinks)
    assert x.cache.check_error() == 0
    g = got.double().cpu().numpy()
    at = 0
    for i, (n, m) in enumerate(zip(x.lens, new)):
        r = R.attend(q64[at:at + m], *x.rows(i), R.scale_of(x.d), positions(n, m), window, sinks)
        R.check(g[at:at + m], r, x.model, **weights(x, few))
        at += m
    return got


SHORT = [(1, 1), (2, 1), (2, 2), (15, 3), (16, 4), (17, 5), (33, 1), (64, 7), (127, 4), (128, 8), (129, 2), (130, 16),
         (255, 3), (256, 5), (257, 1), (300, 12), (0, 0), (90, 0), (511, 9), (700, 16)]
CASES = [
    # hq, hkv, d, bs, kv, model, window, sinks
    (4, 4, 128, 16, "f16", "f16", 0, 0), (2, 2, 64, 8, "bf16", "bf16", 0, 0), (8, 2, 128, 16, "bf16", "bf16", 0, 0),
    (8, 1, 128, 32, "f16", "f16", 0, 0), (4, 2, 64, 32, "f16", "f16", 0, 0), (8, 2, 128, 8, "fp8", "bf16", 0, 0),
    (4, 4, 64, 16, "fp8", "f16", 0, 0), (8, 1, 128, 16, "bf16", "bf16", 0, 0),
    (4, 4, 128, 16, "f16", "f16", 16, 4), (8, 2, 128, 16, "bf16", "bf16", 1, 0), (8, 1, 128, 32, "f16", "f16", 33, 40),
    (4, 2, 64, 8, "bf16", "bf16", 100, 1), (8, 2, 128, 8, "fp8", "bf16", 20, 9), (2, 2, 64, 16, "fp8", "f16", 130, 130),
    (2, 1, 128, 16, "f16", "f16", 2, 0), (8, 2, 128, 32, "bf16", "bf16", 10 ** 9, 2 ** 31 - 1),
    (8, 4, 128, 16, "f16", "f16", 7, 200),
]


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks", CASES)
def test_few_rows(hq, hkv, d, bs, kv, model, window, sinks):
    """Drafted tokens: one tile of rows, two streams of keys."""
    lens, new = zip(*SHORT)
    run(Setup(lens, hq, hkv, d, bs, kv, model, seed=window % 91), new, window, sinks)


LONG = [(1, 1), (40, 40), (130, 128), (129, 129), (257, 255), (256, 256), (257, 257), (300, 1), (600, 400), (513, 20),
        (0, 0), (777, 31), (1000, 33), (64, 64), (500, 0), (140, 17)]


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks", CASES)
def test_many_rows(hq, hkv, d, bs, kv, model, window, sinks):
    """Pieces of prompts: tiles of rows in pairs, from single tokens to whole prompts."""
    lens, new = zip(*LONG)
    run(Setup(lens, hq, hkv, d, bs, kv, model, seed=window % 83), new, window, sinks)


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,lens,new,window,sinks", [
    (4, 4, 128, 16, "f16", "f16", [9000, 100, 5000], [3, 3, 1], 0, 0),
    (8, 1, 128, 8, "bf16", "bf16", [6001], [7], 0, 0),
    (8, 2, 128, 32, "fp8", "bf16", [12345, 8000], [16, 1], 0, 0),
    (2, 2, 64, 16, "bf16", "bf16", [20000], [130], 0, 0),
    (8, 1, 128, 16, "f16", "f16", [7000, 4100], [40, 200], 0, 0),
    (4, 1, 128, 16, "bf16", "bf16", [9000, 300], [5, 5], 5000, 100),
    (8, 2, 128, 16, "bf16", "bf16", [9000, 9000], [300, 1], 3333, 65),
    (2, 1, 64, 8, "fp8", "f16", [5000], [200], 2000, 8),
])
def test_keys_in_several_splits(hq, hkv, d, bs, kv, model, lens, new, window, sinks):
    run(Setup(lens, hq, hkv, d, bs, kv, model), new, window, sinks)


def test_rows_that_see_nothing_and_rows_that_are_not_the_calls():
    """Lengths below the chunk's, zero and negative: zero rows; rows behind the last sequence and of sequences with impossible
    numbers: left as they were."""
    for hq, hkv, most in ((4, 2, 9), (4, 2, 200), (8, 1, 9), (8, 1, 300)):
        x = Setup([20, 30, 40, 25, 50], hq, hkv)
        new = [5, 4, 9, 3, 6]
        cu, q, q64 = chunks(x, new)
        x.context[1], x.context[2], x.context[3] = 0, 4, -7
        out = torch.full((sum(new) + 3, hq, 128), 9.0, dtype=torch.float16, device="cuda")
        big = torch.cat([q, q[:3]])
        P.paged_chunk_attention(big, x.cache, x.tables, x.context, cu, most, R.scale_of(128), out=out)
        assert x.cache.check_error() == 0
        g = out.double().cpu().numpy()
        assert (g[5:9] == 0).all() and (g[9:14] == 0).all() and (g[18:21] == 0).all() and (g[27:] == 9).all()
        R.check(g[:5], R.attend(q64[:5], *x.rows(0), R.scale_of(128), positions(20, 5)), "f16", p="f16")
        R.check(g[21:27], R.attend(q64[21:27], *x.rows(4), R.scale_of(128), positions(50, 6)), "f16", p="f16")
        k, v = x.rows(2)
        R.check(g[14:18], R.attend(q64[14:18], k[:4], v[:4], R.scale_of(128), positions(4, 4)), "f16", p="f16")
        # a length above the tables', then row bounds that descend
        x.context[0] = 10000
        out.fill_(9.0)
        P.paged_chunk_attention(big, x.cache, x.tables, x.context, cu, most, R.scale_of(128), out=out)
        assert x.cache.check_error() == 4
        assert (out[:5] == 9).all() and (out[21:27] != 9).any()
        x.context[0] = 20
        bad = cu.clone()
        bad[1] = 27
        out.fill_(9.0)
        P.paged_chunk_attention(big, x.cache, x.tables, x.context, bad, most, R.scale_of(128), out=out)
        assert x.cache.check_error() & 8


def test_a_bad_block_id_is_reported():
    x = Setup([100, 60], 4, 2)
    cu, q, _ = chunks(x, [3, 3])
    x.tables[0, 2] = x.nb
    P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, 3, 0.1)
    assert x.cache.check_error() == 1


@pytest.mark.parametrize("kv,model", [("f16", "f16"), ("bf16", "bf16"), ("fp8", "bf16")])
def test_agrees_with_the_decode_and_the_prefill(kv, model):
    x = Setup([333, 1, 90, 700], 8, 2, 128, 16, kv, model)
    q, q64 = x.queries(4)
    cu = torch.arange(5, dtype=torch.int32).cuda()
    s = R.scale_of(128)
    for window, sinks in ((0, 0), (50, 3)):
        one = P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, 1, s, window=window, sinks=sinks)
        dec = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, s, window or 10 ** 6, sinks=sinks)
        for i, n in enumerate(x.lens):
            r = R.attend(q64[i:i + 1], *x.rows(i), s, [n - 1], window, sinks)
            tol = R.tolerance(r, model, "pair" if kv == "bf16" else "f16", kv == "fp8") + R.tolerance(r, model, **weights(x))
            assert (np.abs((one - dec)[i].double().cpu().numpy()) <= tol[0]).all()


@pytest.mark.parametrize("new,most", [([4, 7, 2], 16), ([300, 1, 40], 300)])
def test_equal_calls_and_other_sequences_give_equal_bits(new, most):
    lens = [4000, 900, 1500]
    x, y = Setup(lens, 8, 2), Setup(lens[:2] + [700], 8, 2, width=250)
    cu, q, _ = chunks(x, new)
    k, v = (torch.from_numpy(t[:4900]).to(torch.float16).cuda() for t in (x.k64, x.v64))
    P.paged_kv_append(y.cache, k, v, y.slots[:4900])
    call = lambda z: P.paged_chunk_attention(q, z.cache, z.tables, z.context, cu, most, 0.1)
    a, b = call(x), call(y)
    n = new[0] + new[1]
    assert torch.equal(a[:n], b[:n]) and all(torch.equal(a, call(x)) for _ in range(5))


def test_streams_graphs_and_reserved_workspaces():
    x = Setup([5000, 4000], 8, 2, 128, 16, "bf16", "bf16")
    x.cache.reserve_chunk(2, 600, 300, 8, x.tables.shape[1])
    sizes = [[4, 4], [300, 1], [16, 2], [100, 290]]
    calls = [chunks(x, new) for new in sizes]
    one = lambda i, out=None: P.paged_chunk_attention(calls[i][1], x.cache, x.tables, x.context, calls[i][0], max(sizes[i]),
                                                      0.1, window=4500, sinks=7, out=out)
    P.paged_chunk_attention(calls[0][1], x.cache, x.tables, x.context, calls[0][0], 4, 0.1)  # loads the kernels
    P.paged_chunk_attention(calls[1][1], x.cache, x.tables, x.context, calls[1][0], 300, 0.1)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    outs = [torch.empty_like(c[1]) for c in calls]
    for i in range(4):
        one(i, outs[i])
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] >= free - (1 << 21)  # (torch's own outputs come out of a pool of 2 MB pieces)
    want = [o.clone() for o in outs]
    graphs = []
    for i in (2, 3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one(i, outs[i])
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                one(i, outs[i]) if i < 2 else graphs[i - 2].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    x = Setup([20, 30])
    cu, q, _ = chunks(x, [3, 4])
    call = lambda **k: P.paged_chunk_attention(**{**dict(q=q, cache=x.cache, block_tables=x.tables, context_lens=x.context,
                                                         cu_seqlens=cu, max_seqlen=4, scale=0.1), **k})
    for bad in (dict(window=-1), dict(sinks=1), dict(window=4, sinks=-1), dict(cu_seqlens=cu[:2]),
                dict(context_lens=x.context[:1]), dict(block_tables=x.tables[:1]), dict(out=q[:3]), dict(q=q.cpu()),
                dict(q=q[:, :, :64].contiguous())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=q.float()), dict(cu_seqlens=cu.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad, status in ((dict(scale=float("nan")), -1), (dict(scale=0.0), -1), (dict(scale=-0.1), -1), (dict(max_seqlen=-1), -1),
                        (dict(out=q), -1), (dict(q=torch.zeros(7, 12, 128, dtype=torch.float16, device="cuda")), -4),
                        (dict(q=torch.zeros(7, 6, 128, dtype=torch.float16, device="cuda")), -1),
                        (dict(cache=P.KVCache(4, 16, 4, 128, "int4", "f16")), -4)):
        with pytest.raises(P.PagedKVError) as e:
            call(**bad)
        assert e.value.status == status
    with pytest.raises(P.PagedKVError):
        x.cache.reserve_chunk(1, 1, 1, 3, 10)
    assert call(q=q[:0]).shape == (0, 4, 128)
    assert MODEL["f16"] is torch.float16


@pytest.mark.parametrize("kv,model,norm", [("f16", "f16", False), ("fp8", "bf16", True), ("bf16", "bf16", True)])
def test_a_conversation_as_it_runs(kv, model, norm):
    """A prompt in pieces, then single tokens, then drafted ones: rotation and append, then the attention of each, against the
    whole sequence in 64 bits."""
    hq, hkv, d, bs, window, sinks = 8, 2, 128, 16, 150, 4
    g = torch.Generator().manual_seed(5)
    total = 400
    qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g).to(MODEL[model])
    cache = P.KVCache(40, bs, hkv, d, kv_dtype=kv, model_dtype=model)
    cache.view()[0].fill_(255)
    ks = torch.full((hkv,), 0.02).cuda()
    if kv == "fp8":
        cache.set_scales(ks, ks)
    r = P.Rotary(64, interleaved=True, scaling=dict(type="linear", factor=2.0))
    w = (torch.rand(d, generator=g) + 0.5).to(MODEL[model]).cuda() if norm else None
    tables = torch.randperm(40, generator=g)[:26].to(torch.int32)[None].contiguous().cuda()
    dev = qkv.cuda()
    q, k, v = (t.view(total, -1, d) for t in dev.split([hq * d, hkv * d, hkv * d], 1))
    pos = torch.arange(total, dtype=torch.int32).cuda()
    seq = torch.zeros(total, dtype=torch.int32).cuda()
    s = R.scale_of(d)
    # what the cache will hold, and the rotated queries, by the same call into another one
    other = P.KVCache(40, bs, hkv, d, kv_dtype=kv, model_dtype=model)
    if kv == "fp8":
        other.set_scales(ks, ks)
    q_all = P.paged_kv_append_rotary(other, q, k, v, tables, seq, pos, r, q_weight=w, k_weight=w)
    slots = P.paged_slot_mapping(tables, seq, pos, bs)
    pool = other.view()[0]
    if kv == "fp8":
        rows = pool.view(40, 2, hkv, bs, d)[slots // bs, :, :, slots % bs].view(torch.float8_e4m3fn).double() * float(ks[0])
    else:
        rows = pool.view(MODEL[model]).view(40, 2, hkv, bs, d)[slots // bs, :, :, slots % bs].double()
    k64, v64 = rows[:, 0].cpu().numpy(), rows[:, 1].cpu().numpy()
    at = 0
    for n in [200, 100, 57, 1, 1, 1, 5, 3, 1, 16, 1, 14]:
        e = at + n
        qr = P.paged_kv_append_rotary(cache, q[at:e], k[at:e], v[at:e], tables, seq[at:e], pos[at:e], r, q_weight=w,
                                      k_weight=w)
        assert torch.equal(qr, q_all[at:e])
        lens = torch.tensor([e], dtype=torch.int32).cuda()
        p = "pair" if kv == "bf16" else "f16"
        if n == 1:
            out = P.paged_decode_attention_window(qr, cache, tables, lens, s, window, sinks=sinks)
            p = {"bf16": "pair", "f16": "f32", "fp8": "f32"}[kv]
        else:
            cu = torch.tensor([0, n], dtype=torch.int32).cuda()
            out = P.paged_chunk_attention(qr, cache, tables, lens, cu, n, s, window=window, sinks=sinks)
        ref = R.attend(qr.double().cpu().numpy(), k64[:e], v64[:e], s, positions(e, n), window, sinks)
        R.check(out.double().cpu().numpy(), ref, model, p)
        at = e
    assert at == total and cache.check_error() == 0


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,longest", [
    (16, 8, 128, 16, "fp8", "bf16", 4), (8, 8, 128, 16, "f16", "f16", 5), (16, 8, 64, 8, "fp8", "f16", 3), (16, 8, 64, 16, "bf16", "bf16", 8),
    (16, 8, 128, 16, "fp8", "bf16", 150), (8, 8, 128, 8, "bf16", "bf16", 200), (16, 8, 64, 32, "fp8", "f16", 90),
    (8, 8, 64, 16, "f16", "f16", 300)])
def test_many_items_of_unequal_lengths(hq, hkv, d, bs, kv, model, longest):
    """Several items a CTA, the tiles of an item of one to a dozen key tiles each, some absent: stages of the rings change
    hands at every boundary in another order."""
    g = np.random.default_rng(longest)
    lens = [int(min(1500, np.exp(g.normal(np.log(300), 1)))) + 1 for _ in range(190)] + [0, 1, 2]
    new = [int(min(n, 1 + longest * g.random() ** 2)) for n in lens]
    x = Setup(lens, hq, hkv, d, bs, kv, model)
    got = run(x, new, most=longest)
    cu, q, _ = chunks(x, new)
    first = P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, longest, 0.1)
    assert got.shape == first.shape
    for _ in range(6):
        assert torch.equal(first, P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, longest, 0.1))


FEW_LENS = [1, 2, 3, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 257, 300, 511, 700, 0, 40]


@pytest.mark.parametrize("rows", [8, 16, 24])
@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks", [
    (3, 3, 128, 16, "f16", "f16", 0, 0), (4, 2, 64, 8, "bf16", "bf16", 0, 0), (8, 2, 128, 16, "fp8", "bf16", 0, 0),
    (8, 1, 128, 32, "fp8", "f16", 0, 0), (8, 1, 64, 32, "f16", "f16", 0, 0), (2, 2, 64, 16, "fp8", "bf16", 0, 0),
    (8, 2, 128, 8, "bf16", "bf16", 1, 0), (2, 2, 128, 16, "f16", "f16", 16, 4), (8, 2, 128, 32, "fp8", "bf16", 33, 40),
    (8, 1, 64, 8, "fp8", "f16", 7, 9), (4, 2, 128, 8, "bf16", "bf16", 100, 1), (8, 4, 128, 16, "fp8", "f16", 2, 200),
    (4, 1, 128, 16, "f16", "f16", 2 ** 31 - 1, 2 ** 31 - 1), (1, 1, 64, 8, "bf16", "bf16", 64, 64)])
def test_up_to_three_groups_of_eight_rows(rows, hq, hkv, d, bs, kv, model, window, sinks):
    most = rows * hkv // hq
    new = [min(n, i % (most + 1)) for i, n in enumerate(FEW_LENS, 1)]
    new[-1] = most
    run(Setup(FEW_LENS, hq, hkv, d, bs, kv, model, seed=rows + window % 89), new, window, sinks, most=most, few=True)


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,lens,new,window,sinks", [
    (8, 1, 128, 16, "fp8", "bf16", [40000, 77, 1], [2, 1, 1], 0, 0), (4, 4, 128, 8, "f16", "f16", [9000, 2049, 3], [8, 3, 1], 0, 0),
    (8, 2, 64, 32, "bf16", "bf16", [20000, 19999], [6, 0], 0, 0), (8, 2, 128, 16, "fp8", "f16", [9001, 9000, 6100], [4, 1, 3], 5000, 70),
    (2, 1, 128, 32, "bf16", "bf16", [8000, 3000], [12, 5], 2900, 1), (8, 1, 64, 8, "fp8", "bf16", [33333], [3], 0, 0)])
def test_few_rows_over_many_splits(hq, hkv, d, bs, kv, model, lens, new, window, sinks):
    run(Setup(lens, hq, hkv, d, bs, kv, model), new, window, sinks, few=True)


@pytest.mark.parametrize("hq,hkv,kv,model,count", [(4, 1, "fp8", "bf16", 1100), (2, 2, "f16", "f16", 530), (8, 1, "bf16", "bf16", 257)])
@pytest.mark.parametrize("window", [0, 20])
def test_few_rows_of_more_sequences_than_a_launch_takes(hq, hkv, kv, model, count, window):
    lens = [(i * 37) % 90 for i in range(count)]
    new = [min(n, (i * 5) % 3) for i, n in enumerate(lens)]
    run(Setup(lens, hq, hkv, 64, 8, kv, model), new, window, 2 if window else 0, most=2, few=True)


@pytest.mark.parametrize("hq,hkv,kv", [(8, 2, "fp8"), (4, 4, "f16")])
def test_few_rows_on_streams_in_graphs_and_among_others(hq, hkv, kv):
    lens, new = [5000, 4000, 3001], [2, 1, 2]
    x, y = Setup(lens, hq, hkv, kv=kv), Setup([lens[0], 100, 2500], hq, hkv, kv=kv, width=313)
    if kv == "fp8":
        y.cache.set_scales(*x.scales)
    P.paged_kv_append(y.cache, *(t[:5000] for t in x.given), y.slots[:5000])
    cu, q, _ = chunks(x, new)
    call = lambda z, q, out=None: P.paged_chunk_attention(q, z.cache, z.tables, z.context, cu, 2, 0.1, out=out)
    assert x.tables.shape == y.tables.shape
    assert torch.equal(call(x, q)[:2], call(y, q)[:2])  # the first sequence's rows do not depend on the others' lengths
    qs = [torch.randn_like(q) for _ in range(4)]
    want = [call(x, a) for a in qs]
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for q in qs]
    graphs = []
    for a, o in zip(qs[2:], outs[2:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, a, o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                call(x, qs[i], outs[i]) if i < 2 else graphs[i - 2].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and x.cache.check_error() == 0


@pytest.mark.parametrize("kv", ["f16", "fp8"])
def test_few_rows_pass_over_blocks_that_are_none(kv):
    """A bad entry in sight is reported and its tokens count for nothing; NaN keys reach the rows that see them."""
    x = Setup([100, 64], 4, 2, kv=kv)
    cu, q, q64 = chunks(x, [3, 2])
    x.tables[0, 2] = x.nb + 3
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, 3, R.scale_of(128))
    assert x.cache.check_error() == 1
    k, v = x.rows(0)
    keep = np.r_[0:32, 48:100]
    for r in range(3):
        e = np.searchsorted(keep, 97 + r, side="right")
        ref = R.attend(q64[r:r + 1], k[keep[:e]], v[keep[:e]], R.scale_of(128), [e - 1])
        R.check(out[r:r + 1].double().cpu().numpy(), ref, "f16", p="f32")
    x.tables[0, 2] = 0
    x.spoil(1, [63])  # the last token: seen by the last row alone, and by its own tile's rows through V
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, 3, R.scale_of(128))
    assert out[4].isnan().all()


@pytest.mark.parametrize("kv", ["f16", "fp8", "int4"])
def test_a_pool_of_more_than_four_gigabytes(kv):
    """Blocks behind byte 2^32 of the pool: the appended rows and every path's output are those of a small pool."""
    hq, hkv, d, bs = 16, 8, 128, 32
    elem = {"f16": 2.0, "fp8": 1.0, "int4": (d + 8) / 2 / d}[kv]
    block = int(2 * hkv * bs * d * elem)
    count = (1 << 32) // block + 200
    lens, new = [1500, 1000, 300], [200, 3, 1]
    need = [(n + bs - 1) // bs for n in lens]
    tables = torch.full((3, max(need)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)), 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = [torch.randn(sum(lens), h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv)]
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").half()
    context = torch.tensor(lens, dtype=torch.int32).cuda()
    outs = []
    for blocks, shift in ((200, 0), (count, count - 120)):
        t = torch.where(tables >= 0, tables + shift, tables).to(torch.int32).cuda()
        cache = P.KVCache(blocks, bs, hkv, d, kv_dtype=kv, model_dtype="f16")
        if kv == "fp8":
            cache.set_scales(torch.full((hkv,), 0.01).cuda(), torch.full((hkv,), 0.01).cuda())
        o = [P.paged_kv_append_rotary(cache, *rows, t, seq, pos, P.Rotary(d))]
        for w, s in ((400, 5), (5000, 0)):
            o.append(P.paged_decode_attention_window(q[:3], cache, t, context, 0.1, w, sinks=s))
            if kv == "int4":
                continue
            for n in (new, [3, 2, 1]):
                cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
                o.append(P.paged_chunk_attention(q[:sum(n)], cache, t, context, cu, max(n), 0.1, window=w, sinks=s))
        assert cache.check_error() == 0
        outs.append(o)
        cache.close()
    assert all(torch.equal(a, b) and a.isfinite().all() for a, b in zip(*outs))


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks,longest", [
    (8, 2, 128, 16, "fp8", "bf16", 0, 0, 300), (8, 1, 128, 8, "fp8", "f16", 50, 7, 200), (4, 4, 64, 16, "f16", "f16", 0, 0, 400),
    (8, 2, 128, 16, "bf16", "bf16", 333, 3, 300), (2, 2, 64, 8, "fp8", "bf16", 0, 0, 500), (8, 2, 128, 32, "bf16", "bf16", 0, 0, 130)])
def test_few_rows_beside_many(hq, hkv, d, bs, kv, model, window, sinks, longest):
    """Single tokens, drafted tokens and empty rows beside a few pieces of prompts: two kernels share the call."""
    new = [longest, 1, 1, 0, 2, 1, 3, 4, 1, 8, 9, 1, 16, 17, 1, 2, 24, 25, 1, 1, 60, 1, 5, 1, 1, 1, 0, 1, 2, 1, 1, 33, 1, 1, 1, 1]
    lens = [n + (i * 277) % 1900 for i, n in enumerate(new)]
    lens[1], lens[10] = 1, 9
    x = Setup(lens, hq, hkv, d, bs, kv, model, seed=longest)
    assert len(new) * longest >= 4 * sum(new)
    run(x, new, window, sinks)


def test_few_rows_beside_many_on_streams_in_graphs_and_in_reserved_memory():
    new = [200] + [1, 2, 3, 4, 1, 1, 2, 1] * 4
    x = Setup([n + 3000 * (i % 3 == 0) for i, n in enumerate(new)], 8, 2, kv="fp8")
    cu, q, _ = chunks(x, new)
    call = lambda q, out: P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, 200, 0.1, out=out)
    qs = [torch.randn_like(q) for _ in range(4)]
    outs = [torch.empty_like(q) for _ in qs]
    x.cache.reserve_chunk(len(new), sum(new), 200, 8, x.tables.shape[1])
    free = torch.cuda.mem_get_info()[0]
    call(qs[0], outs[0])
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    want = []
    for a, o in zip(qs, outs):
        want.append(call(a, o).clone())
    torch.cuda.synchronize()
    graphs = []
    for a, o in zip(qs[2:], outs[2:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(a, o)
            o.mul_(1.0)  # (an ordinary kernel behind the call sees all of its rows)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].zero_()
                call(qs[i], outs[i]).mul_(1.0) if i < 2 else graphs[i - 2].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and x.cache.check_error() == 0


@pytest.mark.parametrize("piece", [2, 260])
def test_few_rows_in_several_launches_with_splits(piece):
    """Launches that use the same room for their partial rows one after the other, alone and beside a piece of a prompt."""
    lens = [(i * 37) % 90 + (3100 if i in (3, 250, 256, 299) else 0) for i in range(300)]
    lens[7] = 4000
    new = [min(n, (i * 5) % 3) for i, n in enumerate(lens)]
    new[7] = piece
    run(Setup(lens, 4, 4, 64, 8, "f16", "f16", width=700), new, few=piece == 2)
