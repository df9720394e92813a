"""GPU tests at the edges of a step's operators (rotation with append, windowed decode, chunk attention): numbers at the
ends of their types, workspaces, reservations, against 64 bits."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_134_gb300 as P
import seen_ref as R
from seen_setup import MODEL, Setup

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

WIDEST = 2 ** 31 - 1


def packed(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()


def weights(x):
    """How the weights enter the second product where a sequence has more than 24 rows a KV head."""
    return dict(p="pair" if x.kv == "bf16" else "f16")


@pytest.mark.parametrize("window", [WIDEST, WIDEST - 3, 2 ** 30, 10 ** 6])
@pytest.mark.parametrize("hq,hkv,kv,model,lens,new", [
    (4, 2, "f16", "f16", [40, 3, 20], [60, 40, 20]), (8, 1, "bf16", "bf16", [5, 1, 8], [12, 6, 8]),
    (4, 2, "fp8", "bf16", [40, 3, 20], [60, 40, 20]), (4, 4, "f16", "f16", [300, 3, 200], [500, 140, 200]),
    (8, 1, "bf16", "bf16", [150, 40, 100], [250, 90, 100]), (2, 2, "fp8", "f16", [300, 3, 200], [500, 140, 200])])
def test_windows_of_any_length_over_sequences_shorter_than_their_chunk(hq, hkv, kv, model, lens, new, window):
    """Rows before the first token see nothing; the others see all up to their own: position less window has 33 bits."""
    x = Setup(lens, hq, hkv, kv=kv, model=model, seed=3)
    q, q64 = x.queries(sum(new))
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, packed(new), max(new), R.scale_of(x.d), window=window,
                                  sinks=2)
    assert x.cache.check_error() == 0
    got, at = out.double().cpu().numpy(), 0
    for i, (length, n) in enumerate(zip(lens, new)):
        r = R.attend(q64[at:at + n], *x.rows(i), R.scale_of(x.d), list(range(length - n, length)), window, 2)
        R.check(got[at:at + n], r, model, **weights(x))
        assert (got[at:at + max(n - length, 0)] == 0).all()
        at += n


@pytest.mark.parametrize("most", [2 ** 29, 2 ** 30, WIDEST, 2 ** 32, 2 ** 32 + 1])
@pytest.mark.parametrize("hq,hkv,kv,new", [(8, 1, "f16", [20]), (4, 1, "bf16", [30, 2]), (2, 1, "f16", [100, 1, 40]),
                                           (8, 1, "fp8", [20, 300]), (8, 2, "bf16", [3, 1]), (4, 4, "fp8", [1, 9])])
def test_longest_piece_may_be_overstated(hq, hkv, kv, new, most):
    """Any max_seqlen from the longest piece on, to the ends of its type and past it, gives the same rows."""
    model = "bf16" if kv == "bf16" else "f16"
    x = Setup([n + 77 * i for i, n in enumerate(new, 1)], hq, hkv, kv=kv, model=model)
    q, q64 = x.queries(sum(new))
    s = R.scale_of(x.d)
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, packed(new), most, s)
    assert x.cache.check_error() == 0
    assert torch.equal(out, P.paged_chunk_attention(q, x.cache, x.tables, x.context, packed(new), sum(new), s))
    got, at = out.double().cpu().numpy(), 0
    for i, n in enumerate(new):
        r = R.attend(q64[at:at + n], *x.rows(i), s, list(range(x.lens[i] - n, x.lens[i])))
        R.check(got[at:at + n], r, model, **weights(x))
        at += n


def test_reservations_of_the_longest_pieces():
    x = Setup([300], 8, 1)
    for most in (WIDEST, 2 ** 40):
        x.cache.reserve_chunk(1, 100, most, 8, x.tables.shape[1])
    with pytest.raises(P.PagedKVError) as e:
        x.cache.reserve_chunk(1, 100, -2 ** 40, 8, x.tables.shape[1])
    assert e.value.status == -1


@pytest.mark.parametrize("kv,model", [("f16", "f16"), ("fp8", "f16"), ("fp8", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("seqs,new,bits", [(10, 40, 25.2), (10, 100, 30.0), (3, 300, 25.2), (3, 300, 30.0), (16, 24, 30.0)])
def test_many_small_weights_beside_a_large_one(seqs, new, bits, kv, model):
    """One token of weight 1 whose value is 0, thousands of weight 2^-bits whose value is 1: the sum of the small ones is
    the output.  Keys are not split (32 key tiles, as many row tiles as fill the SMs).

    Tolerance: half a step of the output type; a weight as one fp16 2^-11 where it is a normal number, and an error of at
    most 2^-31 of the base's where it is not (the base's own weight is 2^6 or more, and half a step of an fp16
    subnormal 2^-25), as a bf16 pair 2^-16; exp2, sums and quotient 2^-18; the scores are exact but for a product of three
    fp32 factors of about 25, 2 * 25 * 2^-23 in the exponent."""
    d, bs, hkv, length = 64, 16, 32, 4000
    md = MODEL[model]
    blocks = length // bs
    k = torch.zeros(length, hkv, d, dtype=md)
    k[0, :, 0] = 32.0
    v = torch.ones(length, hkv, d, dtype=md)
    v[0] = 0
    cache = P.KVCache(blocks, bs, hkv, d, kv_dtype=kv, model_dtype=model)
    table = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    pos = torch.arange(length)
    slots = table[pos // bs].long() * bs + pos % bs
    P.paged_kv_append(cache, k.cuda(), v.cuda(), slots.cuda())
    q = torch.zeros(seqs * new, hkv, d, dtype=md)
    q[..., 0] = 1.0
    scale = bits * np.log(2) / 32  # the first token's score, in log2 units: bits
    tables = table[None].repeat(seqs, 1).contiguous().cuda()
    lens = torch.full((seqs,), length, dtype=torch.int32).cuda()
    out = P.paged_chunk_attention(q.cuda(), cache, tables, lens, packed([new] * seqs), new, scale)
    assert cache.check_error() == 0
    seen = np.tile(np.arange(length - new, length), seqs).astype(np.float64)  # tokens but the first that a row sees
    small = 2.0 ** -(np.float64(np.float32(scale)) * 32 / np.log(2))
    want = seen * small / (1 + seen * small)
    lost = want * ((2.0 ** -16 if kv == "bf16" else 2.0 ** -11) + 2.0 ** -18 + 2 * 25 * 2.0 ** -23)
    if kv != "bf16":
        lost = lost + seen * 2.0 ** -31
    half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[model]
    tol = half * (want + lost) + lost + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - want[:, None, None]).max((1, 2))
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("kv,length", [("f16", 5000), ("f16", 70000), ("fp8", 30000)])
def test_room_for_partial_rows_is_bounded_under_wide_tables(kv, length):
    """A piece of 5000 tokens, a table for a million: the splits follow the table's width, their room stays at 2 GB."""
    n, hq, hkv = 5000, 8, 1
    x = Setup([length], hq, hkv, kv=kv, width=65536)
    q, q64 = x.queries(n)
    out = torch.empty_like(q)
    cu = packed([n])
    warm = Setup([300], hq, hkv, kv=kv)  # (loads the kernels)
    P.paged_chunk_attention(q[:300], warm.cache, warm.tables, warm.context, packed([300]), 300, 0.1)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, n, R.scale_of(128), out=out)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= (2 << 30) + (64 << 20)
    assert x.cache.check_error() == 0
    rows = np.arange(3, n, 97)
    r = R.attend(q64[rows], *x.rows(0), R.scale_of(128), length - n + rows)
    R.check(out.double().cpu().numpy()[rows], r, "f16", **weights(x))


@pytest.mark.parametrize("tokens,most", [(5000, 5000), (5000, 64), (2 ** 40, 5000)])
def test_reservations_are_bounded_too(tokens, most):
    x = Setup([300], 8, 1, width=65536)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    x.cache.reserve_chunk(1, tokens, most, 8, 65536)
    assert free - torch.cuda.mem_get_info()[0] <= (2 << 30) + (64 << 20)
    x.cache.close()


@pytest.mark.parametrize("hq,hkv,new,tokens,width", [(8, 1, [40], 1024, 8192), (8, 1, [40, 30], 3000, 4096), (4, 1, [200], 2000, 8192),
                                                     (8, 2, [3, 2], 5000, 8192)])
def test_a_padded_q_stays_within_its_reservation(hq, hkv, new, tokens, width):
    """Rows of q behind the last sequence count for the workspace, not for the number of splits."""
    x = Setup([3000 + 400 * i for i in range(len(new))], hq, hkv, width=width)
    q, q64 = x.queries(tokens)
    out, cu = torch.full_like(q, 9.0), packed(new)
    P.paged_chunk_attention(q, Setup([20] * len(new), hq, hkv).cache, x.tables, x.context * 0, cu, max(new), 0.1)  # loads the kernels
    x.cache.reserve_chunk(len(new), tokens, max(new), hq, width)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    P.paged_chunk_attention(q, x.cache, x.tables, x.context, cu, max(new), R.scale_of(128), out=out)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free and x.cache.check_error() == 0
    got, at = out.double().cpu().numpy(), 0
    for i, n in enumerate(new):
        r = R.attend(q64[at:at + n], *x.rows(i), R.scale_of(128), list(range(x.lens[i] - n, x.lens[i])))
        R.check(got[at:at + n], r, "f16", **weights(x))
        at += n
    assert (got[at:] == 9).all()


TWO_PI = Fraction(2 * 3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def reduced(position, freq):
    """position * freq radians, less whole turns, in [-pi, pi], rounded once."""
    angle = position * Fraction(freq)
    return float(angle - round(angle / TWO_PI) * TWO_PI)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_angles_of_far_positions(interleaved, sign):
    """Angles against a product without rounding, at positions near 2^31 where the sine is small, so that its own rounding
    does not hide them.

    Tolerance: as in test_gpu_rotary.py, relative to |y_a| + |y_b| = 2: half a step of fp16 and 2^-20."""
    freqs = [1.0, 0.1, 3.7, 100.7, 12345.678, 1e6 + 0.25, 7.3e9, 1.1e11]
    pos = [WIDEST]
    for f in freqs:  # for each frequency the four positions of the smallest sines, of two thousand
        some = range(WIDEST - 2000, WIDEST)
        pos += sorted(some, key=lambda p: abs(math.sin(reduced(p, f))))[:4]
    n = len(pos)
    x = torch.ones(n, 1, 64, dtype=torch.float16, device="cuda")
    cache = P.KVCache(4, 16, 1, 64, kv_dtype="f16", model_dtype="f16")
    seq, place = torch.zeros(n, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    tables = torch.arange(4, dtype=torch.int32)[None].cuda()
    x[..., 8:16] = 0  # (pairs of halves: (1, 0) turns to (cos, sin))
    if interleaved:
        x[..., 0:16:2], x[..., 1:16:2] = 1, 0
    r = P.Rotary.from_frequencies([sign * f for f in freqs], interleaved=interleaved)
    got = P.paged_kv_append_rotary(cache, x, x, x, tables, seq, place, r,
                                   rotary_positions=torch.tensor(pos, dtype=torch.int32).cuda()).double().cpu().numpy()[:, 0]
    angle = np.array([[reduced(p, sign * f) for f in freqs] for p in pos])
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    for y, w in ((got[:, a], np.cos(angle)), (got[:, b], np.sin(angle))):
        assert (np.abs(y - w) <= 2.0 ** -11 * (np.abs(w) + 2.0 ** -19) + 2.0 ** -19 + 2.0 ** -25).all(), np.abs(y - w).max(0)
    assert (got[:, 16:] == 1).all()


def taken():
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free


@pytest.mark.parametrize("kv", ["f16", "fp8", "int4"])
def test_reserved_window_workspace_covers_smaller_calls(kv):
    """No windowed call of at most the reserved sizes allocates, however its sight is split; graphs take one of their own."""
    seqs, width, hkv, d, bs = 450, 3000, 2, 128, 8
    q = torch.randn(seqs, 16, d, device="cuda").half()
    tables = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    for reserved in (False, True):  # (the first cache's calls load the kernels)
        cache = P.KVCache(1, bs, hkv, d, kv_dtype=kv, model_dtype="f16")
        if reserved:
            cache.reserve_window(seqs, 16, width, 9000, 300)
        before = taken()
        for n in (450, 1, 2, 3, 20, 101, 313):
            for w in (3000, 5, 62, 333, 1200):
                for hq in (16, 2, 4):
                    for window, sinks in ((9000, 300), (1, 0), (100, 4), (1500, 0), (3100, 33), (5000, 300)):
                        P.paged_decode_attention_window(q[:n, :hq].contiguous(), cache, tables[:n, :w].contiguous(),
                                                        lens[:n].contiguous(), 1.0, window, sinks=sinks)
        grown = taken() - before
        assert grown == 0 if reserved else grown > 0
        assert cache.check_error() == 0
        cache.close()


def test_reserved_window_workspace_is_used_and_small():
    x = Setup([9000] * 7 + [1], 8, 2, width=8192)
    q, _ = x.queries(8)
    call = lambda out=None: P.paged_decode_attention_window(q, x.cache, x.tables, x.context, 0.1, 5000, sinks=3, out=out)
    want, out = call(), torch.empty_like(q)
    first = torch.cuda.CUDAGraph()  # (the process's first graph takes memory of the driver's)
    with torch.cuda.graph(first):
        call(out)
    first.replay()
    before = taken()
    for _ in range(2):
        x.cache.reserve_window(8, 8, 8192, 5000, 3)
    reserved = taken()
    assert reserved - before <= 32 << 20  # (what a window shows, not what the tables hold)
    with torch.cuda.stream(torch.cuda.Stream()):
        assert torch.equal(call(out), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    out.zero_()
    graph.replay()
    assert taken() - reserved <= 2 << 20 and torch.equal(out, want)  # (a graph's own nodes)


def test_window_reservations_refused():
    cache = P.KVCache(4, 16, 2, 64, kv_dtype="f16", model_dtype="f16")
    for bad in ((1, 2, 4, 0), (1, 2, 4, -5), (1, 2, 4, 8, -1)):
        with pytest.raises(ValueError):
            cache.reserve_window(*bad)
    for bad, status in (((-1, 2, 4, 8), -1), ((1, -2, 4, 8), -1), ((1, 2, -4, 8), -1), ((1, 3, 4, 8), -4), ((1, 12, 4, 8), -4)):
        with pytest.raises(P.PagedKVError) as e:
            cache.reserve_window(*bad)
        assert e.value.status == status
    lib = P.lib()
    assert lib.kv_cache_reserve_window(cache.handle, 1, 2, 4, 0, 0) == -1
    assert lib.kv_cache_reserve_window(None, 1, 2, 4, 1, 0) == -1
    before = taken()
    cache.reserve_window(0, 2, 4, 8)
    cache.reserve_window(1, 0, 4, 8)
    assert taken() == before


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_reserved_chunk_workspace_covers_smaller_calls(kv):
    """No chunk call of at most the reserved sizes allocates, whichever kernels take it, with padded rows or without."""
    seqs, tokens, width, hkv, d, bs = 70, 700, 3000, 2, 128, 8
    q = torch.randn(tokens, 16, d, device="cuda").to(torch.bfloat16)
    tables = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    for reserved in (False, True):
        cache = P.KVCache(1, bs, hkv, d, kv_dtype=kv, model_dtype="bf16")
        if reserved:
            cache.reserve_chunk(seqs, tokens, 300, 16, width)
        before = taken()
        for n in (70, 1, 2, 9, 33):
            for new in ([1] * n, [300] + [1] * (n - 1), [24] + [2] * (n - 1), [40] * min(n, 9) + [0] * max(0, n - 9)):
                for t in {sum(new), tokens}:
                    for w in (3000, 17, 333):
                        for hq in (16, 2, 8):
                            for window in (0, 4000):
                                P.paged_chunk_attention(q[:t, :hq].contiguous(), cache, tables[:n, :w].contiguous(),
                                                        lens[:n].contiguous(), packed(new), max(new), 1.0, window=window)
        grown = taken() - before
        assert grown == 0 if reserved else grown > 0
        assert cache.check_error() == 0
        cache.close()


def test_windows_that_tables_exceed_are_at_most_two_to_the_thirty():
    """A window no shorter than the tables is none; longer ones than 2^30 tokens under wider tables are refused."""
    x = Setup([100], 4, 2, bs=32)
    q, _ = x.queries(40)
    wide = torch.full((1, 2 ** 25 + 8), -1, dtype=torch.int32, device="cuda")
    call = lambda tables, window: P.paged_chunk_attention(q, x.cache, tables, x.context, packed([40]), 40, 0.1, window=window)
    with pytest.raises(P.PagedKVError) as e:
        call(wide, 2 ** 30 + 1)
    assert e.value.status == -4
    assert torch.equal(call(x.tables, 2 ** 30 + 1), call(x.tables, 0)) and torch.equal(call(x.tables, 128), call(x.tables, 0))


@pytest.mark.parametrize("window,sinks", [(10 ** 6, 2), (200, 40)])
@pytest.mark.parametrize("hq,hkv,kv,model,lens,new", [
    (4, 2, "f16", "f16", [40, 3, 420], [60, 40, 20]), (8, 1, "fp8", "bf16", [700, 40, 100], [250, 90, 100]),
    (8, 2, "bf16", "bf16", [300, 3, 900], [500, 140, 200])])
def test_windows_under_tables_that_hold_more(hq, hkv, kv, model, lens, new, window, sinks):
    x = Setup(lens, hq, hkv, kv=kv, model=model, seed=5, width=1 << 17)
    q, q64 = x.queries(sum(new))
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, packed(new), max(new), R.scale_of(x.d), window=window,
                                  sinks=sinks)
    assert x.cache.check_error() == 0
    got, at = out.double().cpu().numpy(), 0
    for i, (length, n) in enumerate(zip(lens, new)):
        r = R.attend(q64[at:at + n], *x.rows(i), R.scale_of(x.d), list(range(length - n, length)), window, sinks)
        R.check(got[at:at + n], r, model, **weights(x))
        at += n


def test_splits_of_a_million_tokens():
    """A table for 134 million tokens: more key tiles a split than the list's classes of cost."""
    n, hq = 2300, 16
    x = Setup([3000], hq, 2, bs=32, width=1 << 22)
    q, q64 = x.queries(n)
    out = P.paged_chunk_attention(q, x.cache, x.tables, x.context, packed([n]), n, R.scale_of(128))
    assert x.cache.check_error() == 0
    rows = np.arange(3, n, 101)
    r = R.attend(q64[rows], *x.rows(0), R.scale_of(128), 3000 - n + rows)
    R.check(out.double().cpu().numpy()[rows], r, "f16", **weights(x))
