"""GPU tests of paged_decode_attention_window against 64 bits: what is in sight is attended to, what is not is not read
(its table entries are -1, or its slots hold NaN and infinities)."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_134_gb300 as P
import seen_ref as R
from seen_setup import Setup

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def weights(x, plain=False):
    """How the weights enter the second product: as pairs, bf16 (2^-16) or fp16 (2^-22, as good as fp32 here); in the
    plain decode grouped heads of 128 go to the tensor cores, where fp16 weights are single and E4M3 queries terms."""
    if x.kv == "int4":
        return dict(p="f32", steps=x.steps)
    if x.kv == "bf16":
        return dict(p="pair")
    if plain and x.d == 128 and x.hq > x.hkv:
        return dict(p="f16", terms=x.kv == "fp8")
    return dict(p="f32")


def reference(x, q64, window, sinks):
    return [R.attend(q64[i:i + 1], *x.rows(i), R.scale_of(x.d), [n - 1], window, sinks) for i, n in enumerate(x.lens)]


def hide(x, window, sinks):
    """Everything out of sight: blocks taken off the tables, single slots spoilt."""
    for i, n in enumerate(x.lens):
        out = np.flatnonzero(~R.seen(n, [n - 1], window, sinks)[0])
        blocks = {b for b in range((n + x.bs - 1) // x.bs)} - {t // x.bs for t in set(range(n)) - set(out)}
        for b in blocks:
            x.tables[i, b] = -1
        x.spoil(i, [t for t in out if t // x.bs not in blocks])


LENS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 100, 127, 128, 129, 200, 257, 300, 511, 700, 0]
CASES = [
    # hq, hkv, d, bs, kv, model, window, sinks
    (4, 4, 128, 16, "f16", "f16", 16, 4), (4, 4, 128, 16, "f16", "f16", 1, 0), (4, 4, 128, 32, "f16", "f16", 33, 1),
    (2, 2, 64, 8, "bf16", "bf16", 7, 9), (3, 3, 64, 32, "f16", "f16", 100, 33), (2, 2, 128, 8, "fp8", "bf16", 64, 64),
    (1, 1, 64, 16, "fp8", "f16", 5, 0), (3, 3, 128, 32, "bf16", "bf16", 2, 31),
    (4, 2, 64, 16, "f16", "f16", 20, 3), (8, 2, 64, 8, "bf16", "bf16", 129, 8), (8, 1, 64, 32, "fp8", "bf16", 30, 2),
    (4, 2, 128, 16, "f16", "f16", 16, 4), (8, 2, 128, 8, "bf16", "bf16", 1, 0), (8, 2, 128, 32, "bf16", "bf16", 33, 40),
    (8, 1, 128, 16, "f16", "f16", 150, 1), (16, 2, 128, 32, "fp8", "bf16", 17, 5), (4, 1, 128, 8, "fp8", "f16", 1, 1),
    (4, 2, 128, 16, "fp8", "bf16", 300, 0), (8, 2, 128, 16, "bf16", "bf16", 10 ** 9, 0),
    (4, 4, 128, 16, "f16", "f16", 2 ** 31 - 1, 2 ** 31 - 1), (8, 2, 128, 16, "bf16", "bf16", 3, 2 ** 31 - 1),
    (2, 2, 128, 16, "int4", "f16", 16, 4), (4, 2, 128, 8, "int4", "bf16", 1, 0), (8, 2, 64, 32, "int4", "f16", 33, 40),
    (8, 1, 128, 32, "int4", "bf16", 150, 1), (1, 1, 64, 8, "int4", "bf16", 7, 9), (8, 1, 64, 16, "int4", "f16", 64, 64),
    (8, 1, 128, 32, "fp8", "f16", 2 ** 31 - 1, 5), (4, 1, 128, 16, "int4", "f16", 2, 2 ** 31 - 1),
    (8, 1, 128, 8, "fp8", "f16", 100, 70), (8, 1, 128, 16, "bf16", "bf16", 40, 3), (8, 1, 64, 8, "bf16", "bf16", 9, 0),
    (8, 1, 128, 16, "fp8", "bf16", 77, 20),
]


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks", CASES)
def test_what_is_in_sight(hq, hkv, d, bs, kv, model, window, sinks):
    x = Setup(LENS, hq, hkv, d, bs, kv, model, seed=window % 97 + sinks % 89)
    q, q64 = x.queries(len(LENS))
    hide(x, window, sinks)
    out = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, R.scale_of(d), window, sinks=sinks)
    assert x.cache.check_error() == 0
    got = out.double().cpu().numpy()
    for i, r in enumerate(reference(x, q64, window, sinks)):
        R.check(got[i:i + 1], r, model, **weights(x))
    assert (got[-1] == 0).all()  # a sequence without tokens


@pytest.mark.parametrize("hq,hkv,d,bs,kv,model,window,sinks", [
    (4, 4, 128, 16, "f16", "f16", 1500, 4), (8, 2, 128, 16, "bf16", "bf16", 2100, 100), (8, 1, 128, 32, "fp8", "bf16", 3001, 7),
    (2, 2, 64, 8, "bf16", "bf16", 999, 0), (2, 1, 64, 16, "f16", "f16", 4000, 1), (2, 2, 128, 16, "int4", "f16", 1500, 33),
    (8, 1, 64, 32, "int4", "bf16", 4000, 0), (4, 2, 64, 8, "fp8", "f16", 2222, 9), (1, 1, 128, 16, "fp8", "bf16", 4096, 1), (8, 1, 128, 8, "bf16", "bf16", 1800, 2)])
def test_windows_of_several_splits(hq, hkv, d, bs, kv, model, window, sinks):
    x = Setup([5000, 1, window - 1, window, window + sinks, window + sinks + 1, 4097], hq, hkv, d, bs, kv, model)
    q, q64 = x.queries(len(x.lens))
    hide(x, window, sinks)
    out = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, R.scale_of(d), window, sinks=sinks)
    assert x.cache.check_error() == 0
    got = out.double().cpu().numpy()
    for i, r in enumerate(reference(x, q64, window, sinks)):
        R.check(got[i:i + 1], r, model, **weights(x))


@pytest.mark.parametrize("hq,hkv,kv,model", [(2, 2, "f16", "f16"), (4, 1, "bf16", "bf16"), (2, 1, "fp8", "f16"),
                                             (4, 1, "int4", "bf16")])
def test_more_sequences_than_a_launch_takes(hq, hkv, kv, model):
    x = Setup([(i * 37) % 90 for i in range(1300)], hq, hkv, 128, 8, kv, model)
    q, q64 = x.queries(1300)
    out = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, R.scale_of(128), 20, sinks=2)
    assert x.cache.check_error() == 0
    got = out.double().cpu().numpy()
    for i, r in enumerate(reference(x, q64, 20, 2)):
        R.check(got[i:i + 1], r, model, **weights(x))


@pytest.mark.parametrize("hq,hkv,kv", [(4, 4, "f16"), (8, 2, "f16"), (8, 2, "fp8"), (4, 4, "int4")])
def test_bits_depend_on_the_row_alone(hq, hkv, kv):
    """The same sequences among others of other lengths, elsewhere in the pool, and once more: equal bits."""
    lens = [900, 40, 1300, 7]
    x, y = Setup(lens, hq, hkv, kv=kv), Setup(lens[:2] + [1100, 1], hq, hkv, kv=kv, width=82)
    q, _ = x.queries(4)
    if kv == "fp8":
        y.cache.set_scales(*x.scales)
    k, v = (t[:940] for t in x.given)
    P.paged_kv_append(y.cache, k, v, y.slots[:940])
    call = lambda z: P.paged_decode_attention_window(q, z.cache, z.tables, z.context, 0.1, 600, sinks=5)
    assert x.tables.shape == y.tables.shape
    a, b = call(x), call(y)
    assert torch.equal(a[:2], b[:2]) and torch.equal(a, call(x))


def test_a_window_over_everything_is_the_plain_decode():
    for hq, hkv, kv, model in ((4, 4, "f16", "f16"), (8, 2, "bf16", "bf16"), (8, 2, "fp8", "bf16"), (4, 2, "int4", "f16")):
        x = Setup([100, 700, 31], hq, hkv, 128, 16, kv, model)
        q, q64 = x.queries(3)
        got = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, R.scale_of(128), 700)
        plain = P.paged_decode_attention(q, x.cache, x.tables, x.context, R.scale_of(128))
        for i, r in enumerate(reference(x, q64, 0, 0)):
            for o in (got, plain):
                R.check(o[i:i + 1].double().cpu().numpy(), r, model, **weights(x, o is plain))


@pytest.mark.parametrize("hq,hkv,kv", [(4, 4, "f16"), (8, 2, "f16"), (8, 2, "fp8"), (8, 2, "int4")])
def test_bad_tables_and_lengths_are_reported(hq, hkv, kv):
    x = Setup([100, 64, 90], hq, hkv, kv=kv)
    q, q64 = x.queries(3)
    x.tables[0, 5] = x.nb  # in sight
    x.tables[1, 0] = x.nb + 7  # out of sight
    P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 40)
    assert x.cache.check_error() == 1
    x.tables[0, 5] = 0
    x.context[2] = 1000  # the table names 7 blocks: 112 tokens
    x.context[0] = -5
    out = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 8)
    assert x.cache.check_error() & 4
    assert (out[0] == 0).all() and x.cache.check_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
def test_streams_and_graphs_have_their_own_workspace(kv):
    x = Setup([3000, 2900, 2048], 8, 2, 128, 16, kv, "bf16")
    qs = [x.queries(3)[0] for _ in range(4)]
    call = lambda q, out=None: P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 2500, sinks=3, out=out)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for q in qs]
    graphs = []
    for q, o in zip(qs[2:], outs[2:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(q, o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                call(qs[i], outs[i]) if i < 2 else graphs[i - 2].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_of_two_threads():
    x = Setup([2000] * 8, 4, 4)
    q, _ = x.queries(8)
    want = P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 1800, sinks=3)
    torch.cuda.synchronize()
    bad = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(30):
                if not torch.equal(P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 1800, sinks=3), want):
                    bad.append(1)

    ts = [threading.Thread(target=work) for _ in range(3)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_refusals():
    x = Setup([20, 30])
    q, _ = x.queries(2)
    call = lambda **k: P.paged_decode_attention_window(**{**dict(q=q, cache=x.cache, block_tables=x.tables, scale=0.1,
                                                                 context_lens=x.context, window=8), **k})
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(q=q[:1]), dict(context_lens=x.context[:1]),
                dict(block_tables=x.tables[:1]), dict(out=q[:1]), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=q.float()), dict(context_lens=x.context.long())):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(P.PagedKVError) as e:
        call(scale=float("nan"))
    assert e.value.status == -1
    with pytest.raises(P.PagedKVError) as e:  # three query heads on two KV heads do not divide; 12 on 4 is no group
        call(q=torch.zeros(2, 12, 128, dtype=torch.float16, device="cuda"))
    assert e.value.status == -4
    assert call(q=q[:0], context_lens=x.context[:0], block_tables=x.tables[:0]).shape == (0, 4, 128)
