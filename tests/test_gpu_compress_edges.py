"""GPU tests of the 4-bit cache and the decode with attention mass where they can lose precision, drop a NaN or keep
state between calls: against 64-bit references, with bounds derived beside them."""
import math
import threading

import numpy as np
import pytest
import torch

import compress_ref as R
import paged_kv_cache_134_gb300 as P
from paged_kv_cache_134_gb300 import runner, workloads as W

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

TORCH = R.TORCH


def fill(k, v, kv, model, bs=16, lens=None, k_scale=None, v_scale=None):
    """A cache of the sequences' rows k, v [N, Hkv, D] (fp32) one after the other: (cache, tables, lengths)."""
    lens = [k.shape[0]] if lens is None else lens
    need = [(n + bs - 1) // bs for n in lens]
    cache = P.KVCache(max(1, sum(need)), bs, k.shape[1], k.shape[2], kv_dtype=kv, model_dtype=model)
    cache.view()[0].fill_(255)
    if kv == "fp8":
        one = torch.ones(k.shape[1], device="cuda")
        cache.set_scales(one if k_scale is None else k_scale, one if v_scale is None else v_scale)
    t = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at, slots = 0, []
    for i, n in enumerate(need):
        t[i, :n] = torch.arange(at, at + n, dtype=torch.int32)
        slots.append(torch.arange(lens[i]) + at * bs)
        at += n
    P.paged_kv_append(cache, k.to(TORCH[model]).contiguous(), v.to(TORCH[model]).contiguous(),
                      torch.cat(slots).cuda())
    return cache, t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ precision

@pytest.mark.parametrize("model", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(32, 32), (64, 16), (64, 8)])
def test_int4_weights_are_not_cut_to_one_side(model, hq, hkv):
    """Rows whose elements 0..63 hold code 8 and read as exactly 0 (offset -8 s): what the output has there is what the
    weights of the codes' sum lost against those of the offsets' sum.

    Bound of the mean over heads, in units of 8 s.  128 tokens, a 32-token tile a warp: two matrix instructions a
    warp and column, each at most 2^-23 of its sum: 2^-22.  Weights rounded to nearest are off by at most 2^-22 of
    themselves, or 2^-25 of a weight that is at least 2^-3 of the largest where the lo part is subnormal; with
    fp32 sums of eight terms (2^-24 each at most) these have no preferred sign: the mean over 32 or more heads of
    128 tokens stays below 6.5 (odds of 10^-9, Hoeffding) * 2^-21 / sqrt(32 * 128) < 2^-24."""
    L, d, s = 128, 128, 64.0
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 16, (L, hkv, d), generator=g, device="cuda").float()
    codes[..., :64], codes[..., 64], codes[..., 65] = 8, 0, 15
    k = torch.randn(L, hkv, d, generator=g, device="cuda")
    cache, tables, lens = fill(k, (codes - 8) * s, "int4", model)
    q = torch.randn(1, hq, d, generator=g, device="cuda").to(TORCH[model])
    out = P.paged_decode_attention(q, cache, tables, lens, 1 / math.sqrt(d))
    off = R.to64(out[0, :, :64]) / (8 * s)
    assert abs(off.mean()) <= 2.0 ** -22 + 2.0 ** -24, off.mean()
    assert cache.check_error() == 0
    cache.close()


def outlier(L, hq, hkv, d, at, shift, gain, seed, channel):
    """fp32 (q, k, v) of one sequence whose token `at` scores `shift` beside the others' scores of about 1, with a V row
    `gain` times as large.  The score comes from one large channel, or from all of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(L, hkv, d, generator=g, device="cuda")
    v = torch.randn(L, hkv, d, generator=g, device="cuda")
    q = torch.randn(1, hq, d, generator=g, device="cuda")
    if channel:
        q[..., 0], k[..., 0] = 8.0, 0.0
        k[at] *= 0.01
        k[at, :, 0] = shift * math.sqrt(d) / 8.0
    else:
        sign = torch.where(torch.rand(d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        q = sign + 0.1 * q
        k[at] = shift / math.sqrt(d) * sign
    v[at] *= gain
    return q, k, v


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("L,at,shift,gain", [
    (256, 5, -20.0, 64.0), (256, 5, -20.0, 1024.0), (1000, 900, -20.0, 1024.0),   # no weight, a great range
    (5000, 3, 16.0, 1.0 / 64), (5000, 3, 16.0, 1.0), (5000, 4990, 16.0, 1.0 / 64),  # nearly all the weight
    (700, 3, -60.0, 3000.0), (700, 3, 40.0, 1e-3),
    (700, 3, -60.0, 30000.0)])                             # past the type: the row reads as NaN, and so does the output
def test_int4_a_token_of_another_magnitude_leaves_the_others_their_weights(L, at, shift, gain, channel, hq, hkv, mass):
    """Bound: half a step of the output, the weights' relative error, and what the codes lose in a product of 16 tokens,
    2^-17 of a step of the largest p s among them: over all groups of 16 at most 16 * 2^-17 sum(p s).  A product p s is
    kept to 2^-22 of itself or 2^-29 of the largest of its warp's tokens of a split, 256 of them: together, times codes of
    at most 15, 15 * 2^-21 sum(p s)."""
    d, model = 128, "f16"
    q, k, v = outlier(L, hq, hkv, d, at, shift, gain, L + hq, channel)
    q = q.to(TORCH[model])
    cache, tables, lens = fill(k, v, "int4", model)
    scale = 1 / math.sqrt(d)
    k64, v64 = (R.values4(*R.quantise4(R.to64(x.to(TORCH[model])), model)) for x in (k, v))
    steps = [R.quantise4(R.to64(x.to(TORCH[model])), model)[1] for x in (k, v)]
    m = torch.zeros(1, hkv, L, device="cuda")
    out = (P.paged_decode_attention_mass(q, cache, tables, lens, scale, m) if mass
           else P.paged_decode_attention(q, cache, tables, lens, scale))
    ref, p, pv, big = R.attention(R.to64(q[0]), k64, v64, scale)
    rel = R.relative_weight_error(big) + R.code_alignment(d, R.to64(q[0]), steps[0], scale)
    ps = np.einsum("ht,th->h", p, np.repeat(steps[1], hq // hkv, 1))[:, None]
    tol = R.HALF_STEP[model] * np.abs(ref) * 1.001 + rel * pv + (2.0 ** -13 + 15 * 2.0 ** -21) * ps + 2.0 ** -24
    err = np.abs(R.to64(out[0]) - ref)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(R.to64(out[0])), nan)
    assert np.all(err[~nan] <= tol[~nan]), (err / tol)[~nan].max()
    if mass:
        want = p.reshape(hkv, hq // hkv, L).sum(1)
        assert np.all(np.abs(R.to64(m[0]) - want) <= rel * want + 2.0 ** -24)
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("kv,model", [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"), ("fp8", "bf16")])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("shift,at", [(12.0, 3), (16.0, 3), (18.0, 3), (20.0, 19990)])
def test_mass_decode_keeps_small_weights_beside_a_dominant_one(kv, model, hq, hkv, shift, at):
    """One token of zeros takes nearly all the weight: the output is the other 19999 tokens' share.

    Bound: half a step of the output; a score of at most 16 fp32 roundings of 2^-23 of sum |q||k| scale, in a weight twice
    that; 2^-19 for exp2 and the sums; 2^-15 for weights as bf16 pairs (2^-22 as fp16 pairs), and 2^-39 of the
    largest weight for each that is no normal fp16 number."""
    L, d = 20000, 128
    q, k, v = outlier(L, hq, hkv, d, at, shift, 1.0, hq, False)
    v = 1000.0 + 100.0 * v
    v[at] = 0.0
    q, k, v = (x.to(TORCH[model]) for x in (q, k, v))
    scales = [(x.float().abs().amax(dim=(0, 2)) / 448).contiguous() for x in (k, v)]
    cache, tables, lens = fill(k, v, kv, model, k_scale=scales[0], v_scale=scales[1])
    scale = 1 / math.sqrt(d)
    m = torch.zeros(1, hkv, L, device="cuda")
    out = P.paged_decode_attention_mass(q, cache, tables, lens, scale, m)
    if kv == "fp8":
        k, v = ((x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s[:, None].double()
                for x, s in zip((k, v), scales))
    ref, p, pv, big = R.attention(R.to64(q[0]), R.to64(k), R.to64(v), scale)
    rel = 2 * 16 * 2.0 ** -23 * big + 2.0 ** -19 + (2.0 ** -15 if kv == "bf16" else 0.0)
    tol = R.HALF_STEP[model] * np.abs(ref) * 1.001 + rel * pv + L * 2.0 ** -39 * float(v.double().abs().max()) + 2.0 ** -24
    err = np.abs(R.to64(out[0]) - ref)
    assert np.all(err <= tol), (err / tol).max()
    want = p.reshape(hkv, hq // hkv, L).sum(1)
    assert np.all(np.abs(R.to64(m[0]) - want) <= rel * want + 2.0 ** -60)
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (4, 1, 128), (8, 1, 64), (8, 1, 128)])
@pytest.mark.parametrize("L,at", [(128, 3), (700, 690), (2500, 5)])
def test_int4_a_warp_without_weight_in_one_head_only(hq, hkv, d, L, at, mass):
    """One head has a token 250 above the others, so that every other warp's weight in that head alone is 0."""
    g = torch.Generator(device="cuda").manual_seed(hq)
    k, v = torch.randn(2, L, hkv, d, generator=g, device="cuda")
    q = torch.randn(1, hq, d, generator=g, device="cuda")
    q[..., 0], k[..., 0] = 0.0, 0.0
    q[:, 1, 0], k[at, :, 0] = 50.0, 5.0 * math.sqrt(d)
    q, k, v = (x.half() for x in (q, k, v))
    cache, tables, lens = fill(k, v, "int4", "f16")
    scale = 1 / math.sqrt(d)
    m = torch.zeros(1, hkv, L, device="cuda")
    out = (P.paged_decode_attention_mass(q, cache, tables, lens, scale, m) if mass
           else P.paged_decode_attention(q, cache, tables, lens, scale))
    quantised = [R.quantise4(R.to64(x), "f16") for x in (k, v)]
    ref, p, pv, big = R.attention(R.to64(q[0]), *(R.values4(*x) for x in quantised), scale)
    rel = R.relative_weight_error(big) + R.code_alignment(d, R.to64(q[0]), quantised[0][1], scale)
    tol = R.HALF_STEP["f16"] * np.abs(ref) * 1.001 + rel * pv + 2.0 ** -13 * float(quantised[1][1].max()) + 2.0 ** -24
    assert np.all(np.abs(R.to64(out[0]) - ref) <= tol)
    assert abs(p[1, at] - 1) < 1e-6 and p[0, at] < 0.5
    assert cache.check_error() == 0
    cache.close()


# ------------------------------------------------------------------------------------------ NaN

# one token behind every multiple that a split may have, and rows that one warp takes
NAN_LENS = [1, 33, 65, 97, 129, 193, 225, 257, 353, 385, 449, 481, 513, 609, 641, 769, 897, 961, 1025, 2049]


@pytest.mark.parametrize("kv,model", [("int4", "f16"), ("int4", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("f16", "f16"),
                                      ("bf16", "bf16")])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (8, 2), (16, 2)])
@pytest.mark.parametrize("lens", [NAN_LENS, [2049], [1], [40] * 200, [1, 2, 31, 32, 7], [20] * 400],
                         ids=["ragged", "long", "one", "many", "short", "manyshort"])
@pytest.mark.parametrize("where", ["query", "key", "value", "far value"])
def test_nan_reaches_the_output_however_a_row_is_split(kv, model, hq, hkv, lens, where):
    """A NaN in a query, in the last token's key, in its value, and in the value of a last token that has no weight (a
    score of -2^11): output and mass are NaN where the formula's are, and nowhere else."""
    d, n = 64, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    k, v = torch.randn(2, n, hkv, d, generator=g, device="cuda")
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda")
    q[..., 0], k[..., 0] = 8.0, 0.0
    last = torch.tensor(lens).cumsum(0) - 1
    if where == "query":
        q[:, -1, 5] = float("nan")
    elif where == "key":
        k[last, 0, 3] = float("nan")
    else:
        v[last, 0, 3] = float("nan")
        if where == "far value":
            k[last, :, 0] = -256.0
    q, k, v = (x.to(TORCH[model]) for x in (q, k, v))
    cache, tables, context = fill(k, v, kv, model, lens=lens)
    mass = torch.zeros(len(lens), hkv, max(lens), device="cuda")
    outs = [P.paged_decode_attention_mass(q, cache, tables, context, 1.0, mass)]
    if kv == "int4":
        outs.append(P.paged_decode_attention(q, cache, tables, context, 1.0))
        outs.append(torch.empty_like(q))
        P.paged_decode_attention_noalloc(q, cache, tables, context, 1.0, outs[-1])
    nan = torch.zeros(q.shape, dtype=torch.bool, device="cuda").view(len(lens), hkv, -1, d)
    bad_mass = torch.zeros(mass.shape, dtype=torch.bool, device="cuda")
    inside = torch.arange(max(lens), device="cuda") < context[:, None]
    if where == "query":
        nan[:, -1, -1] = True
        bad_mass[:, -1] = inside
    elif where == "key":
        nan[:, 0] = True
        bad_mass[:, 0] = inside
    elif kv == "int4":
        nan[:, 0] = True                                   # the whole row reads as NaN
    else:
        nan[:, 0, :, 3] = True
    for out in outs:
        assert torch.equal(out.isnan(), nan.view_as(out)) and torch.isfinite(out[~nan.view_as(out)]).all()
    assert torch.equal(mass.isnan(), bad_mass) and torch.isfinite(mass[~bad_mass]).all()
    assert cache.check_error() == 0
    cache.close()


# ------------------------------------------------------------------------------------------ other sequences, other calls

@pytest.mark.parametrize("kv,model", [("int4", "f16"), ("int4", "bf16"), ("fp8", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("hq,hkv,d,most,seqs", [(32, 32, 64, 200, 120), (32, 8, 128, 300, 200), (16, 4, 64, 900, 160),
                                                (64, 8, 128, 300, 200), (8, 8, 128, 1500, 130)])
def test_a_row_does_not_depend_on_the_other_sequences_lengths(kv, model, hq, hkv, d, most, seqs):
    """Several units a CTA: the other rows' lengths decide which CTA, and which of its warps, a row meets."""
    g = torch.Generator(device="cuda").manual_seed(hq + most)
    lens = torch.randint(1, most + 1, (seqs,), generator=torch.Generator().manual_seed(1)).tolist()
    lens[0] = most
    n = sum(lens)
    k, v = torch.randn(2, n, hkv, d, generator=g, device="cuda").to(TORCH[model])
    q = torch.randn(seqs, hq, d, generator=g, device="cuda").to(TORCH[model])
    cache, tables, context = fill(k, v, kv, model, lens=lens, k_scale=torch.full((hkv,), 0.02, device="cuda"),
                                  v_scale=torch.full((hkv,), 0.02, device="cuda"))
    keep = torch.arange(0, seqs, 3, device="cuda")
    runs = []
    for i in range(3):
        now = context if i == 0 else (context // (4 * i)).int()
        now[keep] = context[keep]
        mass = torch.zeros(seqs, hkv, most, device="cuda")
        out = [P.paged_decode_attention_mass(q, cache, tables, now, d ** -0.5, mass)[keep], mass[keep]]
        if kv == "int4":
            out.append(P.paged_decode_attention(q, cache, tables, now, d ** -0.5)[keep])
        runs.append(out)
    for out in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, runs[0]))
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("seqs,hkv,eager", [(6, 2, 2),     # many splits: joined by a second launch, without counters
                                            (40, 8, 1)])   # at most 16: by the row's last CTA
def test_int4_counters_are_cleared_where_calls_may_have_met(seqs, hkv, eager):
    """The counters that a row's last CTA joins by: a call on the library's fixed scratch, and a captured one, clear them first
    (a launch more), so that nothing an earlier call left there matters; a stream's own workspace is its calls' alone."""
    lens, hq, d = [3000] * (seqs - 1) + [1], 16, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = torch.randn(2, sum(lens), hkv, d, generator=g, device="cuda")
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").half()
    cache, tables, context = fill(k, v, "int4", "f16", lens=lens)
    outs = [torch.empty_like(q) for _ in range(3)]

    def launches(call):
        before = P.kernel_launches()
        call()
        return P.kernel_launches() - before

    assert launches(lambda: P.paged_decode_attention(q, cache, tables, context, 0.1, out=outs[0])) == eager
    assert launches(lambda: P.paged_decode_attention_noalloc(q, cache, tables, context, 0.1, outs[1])) == 2
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert launches(lambda: P.paged_decode_attention(q, cache, tables, context, 0.1, out=outs[2])) == 2
    for _ in range(3):
        outs[2].zero_()
        graph.replay()
        assert torch.equal(outs[2], outs[0]) and torch.equal(outs[1], outs[0])
    assert cache.check_error() == 0
    cache.close()


# ------------------------------------------------------------------------------------------ workspaces

def device_memory_taken():
    """Device memory in use that torch does not hold."""
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free - torch.cuda.memory_reserved()


def ragged_decode(lens, kv="int4", hq=16, hkv=8, d=128, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = torch.randn(2, sum(lens), hkv, d, generator=g, device="cuda").half()
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").half()
    return (q, *fill(k, v, kv, "f16", lens=lens, k_scale=torch.full((hkv,), 0.02, device="cuda"),
                     v_scale=torch.full((hkv,), 0.02, device="cuda")))


def test_every_reserve_adds_a_workspace():
    """Two streams and a capture after three reserves: none of their calls allocates."""
    q, cache, tables, context = ragged_decode([3000] * 39 + [1])
    want = torch.empty_like(q)
    P.paged_decode_attention_noalloc(q, cache, tables, context, 0.1, want)   # loads the kernels
    outs = [torch.empty_like(q) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                                            # (what a capture allocates for itself)
        outs[0].fill_(0)
    del graph
    for _ in range(3):
        cache.reserve(40, 16, tables.shape[1])
    before = device_memory_taken()
    for s, out in zip(streams, outs):
        with torch.cuda.stream(s):
            P.paged_decode_attention(q, cache, tables, context, 0.1, out=out)
    assert device_memory_taken() == before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.paged_decode_attention(q, cache, tables, context, 0.1, out=outs[2])
    after = device_memory_taken()
    graph.replay()
    torch.cuda.synchronize()
    assert after - before < 1 << 20          # (a graph's own nodes; a workspace of these sizes takes 2 MB)
    assert all(torch.equal(out, want) for out in outs)
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("kv", ["f16", "fp8", "int4"])
def test_reserved_mass_workspace_covers_smaller_calls(kv):
    """No mass call of at most the reserved sizes allocates, whichever way its rows are split."""
    seqs, width, hkv, d, bs = 450, 700, 2, 128, 8
    q = torch.randn(seqs, 16, d, device="cuda").half()
    tables = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    mass = torch.zeros(seqs * hkv * width * bs, device="cuda")
    for reserved in (False, True):                         # (the first cache's calls load the kernels)
        cache = P.KVCache(1, bs, hkv, d, kv_dtype=kv, model_dtype="f16")
        if reserved:
            cache.reserve_mass(seqs, 16, width, width * bs)
        before = device_memory_taken()
        for n in (450, 1, 2, 3, 20, 101, 390):
            for w in (700, 5, 17, 62, 333, 512):
                for hq in (16, 2, 4):
                    for t in (w * bs, w * bs // 3):
                        P.paged_decode_attention_mass(q[:n, :hq].contiguous(), cache, tables[:n, :w].contiguous(),
                                                      lens[:n].contiguous(), 1.0,
                                                      mass[: n * hkv * t].view(n, hkv, t))
        grown = device_memory_taken() - before
        assert grown == 0 if reserved else grown > 0
        assert cache.check_error() == 0
        cache.close()


def test_reserved_mass_workspace_is_used():
    q, cache, tables, context = ragged_decode([3000] * 7 + [1], kv="f16", hq=8, hkv=2)
    mass = [torch.zeros(8, 2, 3000, device="cuda") for _ in range(2)]
    want = P.paged_decode_attention_mass(q, cache, tables, context, 0.1, mass[0])
    cache.reserve_mass(8, 8, tables.shape[1], 3000)
    before = device_memory_taken()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = P.paged_decode_attention_mass(q, cache, tables, context, 0.1, mass[1])
    assert device_memory_taken() == before
    assert torch.equal(out, want) and torch.equal(mass[0], mass[1])
    assert P.binding.lib().kv_cache_reserve_mass(cache.handle, -1, 8, 1, 1) == -1
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("kv", ["int4", "f16"])
def test_workspaces_do_not_pile_up(kv):
    """A stream keeps one workspace however often it was outgrown, and those of streams and captures are given back."""
    q, cache, tables, context = ragged_decode([3000] * 64, kv=kv, hq=8, hkv=2)
    mass = torch.zeros(64, 2, 3000, device="cuda")
    out = torch.empty_like(q)

    def call(n):
        P.paged_decode_attention_mass(q[:n], cache, tables[:n], context[:n], 0.1, mass[:n], out=out[:n], decay=0.0)

    call(64)
    want = (out.clone(), mass.clone())
    torch.cuda.synchronize()
    cache.release_workspaces()
    empty = device_memory_taken()
    call(64)
    one = device_memory_taken() - empty
    assert one >= 6 << 20                                  # the scores of 64 x 8 x 3000 alone
    cache.release_workspaces()
    assert device_memory_taken() == empty
    for n in range(1, 65, 3):                              # outgrown 21 times
        call(n)
    call(64)
    assert device_memory_taken() - empty <= 2 * one
    assert all(torch.equal(a, b) for a, b in zip((out, mass), want))
    graphs = []
    for _ in range(3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(5)
            call(64)
        graphs.append(g)
    cache.release_workspaces()                             # leaves the graphs theirs
    out.zero_(), mass.fill_(2.0)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, mass), want))
    held = device_memory_taken() - empty
    graphs.clear()
    del g
    cache.release_workspaces(graphs=True)
    assert device_memory_taken() - empty <= held - 3 * one
    call(64)                                               # and the cache goes on
    assert all(torch.equal(a, b) for a, b in zip((out, mass), want))
    assert cache.check_error() == 0
    cache.close()


def test_two_host_threads_grow_one_streams_workspace():
    """A call that replaces the stream's workspace does not take it from another thread's call that has yet to launch."""
    q, cache, tables, context = ragged_decode([2000] * 24, hq=8, hkv=2)
    want = P.paged_decode_attention(q, cache, tables, context, 0.1)
    sizes = [[1, 3, 7, 15, 24], [2, 5, 9, 18, 24]]
    first = {n: P.paged_decode_attention(q[:n], cache, tables[:n], context[:n], 0.1) for s in sizes for n in s}
    outs = [[torch.empty_like(q[:n]) for n in s * 10] for s in sizes]
    torch.cuda.synchronize()
    cache.release_workspaces()

    def run(sizes, outs):
        for n, out in zip(sizes * 10, outs):
            P.paged_decode_attention(q[:n], cache, tables[:n], context[:n], 0.1, out=out)

    threads = [threading.Thread(target=run, args=a) for a in zip(sizes, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for s, out in zip(sizes, outs):
        assert all(torch.equal(o, first[n]) for n, o in zip(s * 10, out))
    assert torch.equal(first[24], want)
    assert cache.check_error() == 0
    cache.close()


# ------------------------------------------------------------------------------------------ step helpers

@pytest.mark.parametrize("model", ["f16", "bf16"])
@pytest.mark.parametrize("fused", [True, False])
def test_the_decode_step_takes_a_4_bit_cache(model, fused):
    w = W.small_decode("int4", [0, 1, 37, 300], hq=8, hkv=2, d=128, bs=16, kv_dtype="int4", model_dtype=model)
    got = runner.run_decode(w, fused=fused)
    assert got["err"] == 0 and got["pool"].dtype == np.uint8
    assert got["pool"].size == w.num_blocks * 2 * 16 * (128 + 8)
    q = R.to64(runner.dev(w.q, TORCH[model]))
    for s in range(4):
        k, v = (R.to64(runner.dev(x, TORCH[model])) for x in W.logical_kv(w, s))
        (ck, sk, lk), (cv, sv, lv) = R.quantise4(k, model), R.quantise4(v, model)
        scale = float(w.scale)
        ref, _, pv, big = R.attention(q[s], R.values4(ck, sk, lk), R.values4(cv, sv, lv), scale)
        rel = R.relative_weight_error(big) + R.code_alignment(128, q[s], sk, scale)
        tol = R.HALF_STEP[model] * np.abs(ref) * 1.001 + rel * pv + 2.0 ** -13 * float(sv.max()) + 2.0 ** -24
        assert np.all(np.abs(got["out"][s] - ref) <= tol)


def test_the_prefill_step_takes_a_4_bit_cache():
    w = W.prefill(lengths=[5, 40, 1], heads=4, kv_heads=2, d=64, dtype="f16", kv_dtype="int4")
    plain = W.prefill(lengths=[5, 40, 1], heads=4, kv_heads=2, d=64, dtype="f16")
    got, want = runner.run_prefill(w, keep_cache=True), runner.run_prefill(plain)
    assert got["err"] == 0 and np.array_equal(got["out"], want["out"])   # the attention reads the packed k and v
    pos = np.concatenate([np.arange(n) for n in w.lengths])
    seq = np.repeat(np.arange(3), w.lengths)
    slots = torch.from_numpy(w.block_tables[seq, pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
    k, v = P.paged_kv_gather(got["cache"], slots)
    for x, back in ((w.k, k), (w.v, v)):
        x = runner.dev(x, torch.float16)
        want = torch.from_numpy(R.values4(*R.quantise4(R.to64(x), "f16")).astype(np.float32)).half()
        assert torch.equal(back.cpu(), want)
    got["cache"].close()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("at", [40, 5])
def test_int4_a_great_range_without_any_weight(hq, hkv, at):
    """All the weight on a token of range 2^-80; the others, of range 2^80, have none (scores 400 below): the output is
    that token's row, to half a step and 2^-12 of a step (the codes' products)."""
    L, d, model = 300, 128, "bf16"
    g = torch.Generator(device="cuda").manual_seed(at)
    k, v = torch.randn(2, L, hkv, d, generator=g, device="cuda")
    q = torch.randn(1, hq, d, generator=g, device="cuda")
    q[..., 0], k[..., 0] = 50.0, 0.0
    k[at, :, 0] = 8.0
    v *= torch.where(torch.arange(L, device="cuda") == at, 2.0 ** -80, 2.0 ** 80)[:, None, None]
    q = q.to(TORCH[model])
    cache, tables, lens = fill(k, v, "int4", model)
    quantised = R.quantise4(R.to64(v.to(TORCH[model])), model)
    want, step = np.repeat(R.values4(*quantised)[at], hq // hkv, 0), np.repeat(quantised[1][at], hq // hkv, 0)[:, None]
    tol = (R.HALF_STEP[model] * np.abs(want) + 2.0 ** -12 * step) * 1.001
    m = torch.zeros(1, hkv, L, device="cuda")
    for out in (P.paged_decode_attention(q, cache, tables, lens, 1.0),
                P.paged_decode_attention_mass(q, cache, tables, lens, 1.0, m)):
        assert np.all(np.abs(R.to64(out[0]) - want) <= tol)
    assert torch.equal(m[0, :, at], torch.full((hkv,), hq / hkv, device="cuda"))
    assert cache.check_error() == 0
    cache.close()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("lens", [[1, 5, 32], [1, 40, 700, 2100]], ids=["short", "long"])
def test_infinities_in_a_16_bit_cache(kv, hq, hkv, lens):
    """A score of -infinity takes no weight, a row of nothing else is zeros; +infinity gives NaN; an infinity in V something
    that is not finite, in its element alone."""
    d, n = 64, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = torch.randn(2, n, hkv, d, generator=g, device="cuda")
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").to(TORCH[kv])
    q[..., 0] = 1.0
    inf, last = float("inf"), torch.tensor(lens).cumsum(0) - 1
    for where in ("low", "all low", "high", "value"):
        kk, vv = k.clone(), v.clone()
        if where == "low":
            kk[last[1:], :, 0] = -inf                      # (the row of one token keeps it)
        elif where == "all low":
            kk[..., 0] = -inf
        elif where == "high":
            kk[last, :, 0] = inf
        else:
            vv[last, :, 3] = inf
        cache, tables, context = fill(kk, vv, kv, kv, lens=lens)
        mass = torch.full((len(lens), hkv, max(lens)), 0.5, device="cuda")
        out = P.paged_decode_attention_mass(q, cache, tables, context, 0.1, mass).float()
        inside = (torch.arange(max(lens), device="cuda") < context[:, None])[:, None].expand_as(mass)
        if where == "low":
            assert torch.isfinite(out).all() and torch.isfinite(mass).all()
            end = mass[torch.arange(1, len(lens)), :, torch.tensor(lens[1:]) - 1]
            assert torch.equal(end, torch.full_like(end, 0.5))
            total = (mass - 0.5).sum(-1)
            assert torch.allclose(total, torch.full_like(total, hq / hkv), rtol=1e-3)
        elif where == "all low":
            assert not out.any() and torch.equal(mass, torch.full_like(mass, 0.5))
        elif where == "high":
            assert out.isnan().all() and torch.equal(mass.isnan(), inside)
        else:
            assert not torch.isfinite(out[..., 3]).any() and torch.isfinite(mass).all()
            assert torch.isfinite(torch.cat([out[..., :3], out[..., 4:]], -1)).all()
        assert cache.check_error() == 0
        cache.close()


@pytest.mark.parametrize("mass_first", [True, False])
def test_a_decode_leaves_the_larger_workspace_to_the_mass_call(mass_first):
    q, cache, tables, context = ragged_decode([3000] * 39 + [1])
    mass = torch.zeros(40, 8, 3000, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    P.paged_decode_attention(q, cache, tables, context, 0.1, out=outs[0])            # loads the kernels
    P.paged_decode_attention_mass(q, cache, tables, context, 0.1, mass, out=outs[1])
    cache.release_workspaces()
    reserve = [lambda: cache.reserve(40, 16, tables.shape[1]), lambda: cache.reserve_mass(40, 16, tables.shape[1], 3000)]
    for i in (1, 0) if mass_first else (0, 1):
        reserve[i]()
    streams = [torch.cuda.Stream() for _ in range(2)]
    before = device_memory_taken()
    with torch.cuda.stream(streams[0]):
        P.paged_decode_attention(q, cache, tables, context, 0.1, out=outs[0])
    with torch.cuda.stream(streams[1]):
        P.paged_decode_attention_mass(q, cache, tables, context, 0.1, mass, out=outs[1])
    assert device_memory_taken() == before
    assert cache.check_error() == 0
    cache.close()
