"""Frequencies of Rotary against their definitions, and its refusals (host only)."""
import ctypes
import math
import threading

import numpy as np
import pytest

import paged_kv_cache_134_gb300 as P


def plain(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot)


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0)])
def test_frequencies(rot, base):
    r = P.Rotary(rot, base=base)
    assert r.rotary_dim == rot and r.gain == 1.0 and not r.interleaved
    np.testing.assert_allclose(r.inv_freq, plain(rot, base), rtol=1e-14)


def test_linear():
    np.testing.assert_allclose(P.Rotary(64, scaling=dict(type="linear", factor=8)).inv_freq, plain(64) / 8, rtol=1e-14)


def test_ntk_keeps_the_fastest_and_divides_the_slowest():
    f, g = P.Rotary(128, scaling=dict(type="ntk", factor=4)).inv_freq, plain(128)
    assert f[0] == g[0]
    np.testing.assert_allclose(f[-1], g[-1] / 4, rtol=1e-13)
    assert all(b / 4 * (1 - 1e-13) <= a <= b for a, b in zip(f, g))


def test_yarn_ends_ramp_and_gain():
    s = dict(type="yarn", factor=32.0, original_max_position=4096, beta_fast=32, beta_slow=1)
    r, g = P.Rotary(128, scaling=s, interleaved=True), plain(128)
    assert r.interleaved and r.gain == pytest.approx(0.1 * math.log(32) + 1)
    f = np.array(r.inv_freq)
    turns = g * 4096 / (2 * math.pi)
    # whole dimensions bound the ramp, so a pair within one of a bound may lie on either side of it
    fast = turns > 32 * 10000 ** (2 / 128)
    slow = turns < 1 / 10000 ** (2 / 128)
    np.testing.assert_allclose(f[fast], g[fast], rtol=1e-14)
    np.testing.assert_allclose(f[slow], g[slow] / 32, rtol=1e-13)
    share = (f / g - 1 / 32) / (1 - 1 / 32)  # 1 fast .. 0 slow, falling by equal steps
    mid = (share > 1e-9) & (share < 1 - 1e-9)
    assert mid.sum() > 8
    np.testing.assert_allclose(np.diff(share[mid]), np.diff(share[mid])[0], rtol=1e-9)
    assert P.Rotary(128, scaling=dict(s, attention_factor=1.0)).gain == 1.0


def test_own_frequencies():
    f = [1.0 / (i + 1) for i in range(24)]
    r = P.Rotary.from_frequencies(f, gain=0.5)
    assert r.inv_freq == tuple(f) and r.rotary_dim == 48 and r.gain == 0.5


@pytest.mark.parametrize("args", [
    dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=-16), dict(rotary_dim=64, base=1.0),
    dict(rotary_dim=64, base=math.inf), dict(rotary_dim=64, base=math.nan),
    dict(rotary_dim=64, scaling=dict(type="linear")), dict(rotary_dim=64, scaling=dict(type="linear", factor=0.5)),
    dict(rotary_dim=64, scaling=dict(type="cubic", factor=2)),
    dict(rotary_dim=64, scaling=dict(type="yarn", factor=2)),
    dict(rotary_dim=64, scaling=dict(type="yarn", factor=2, original_max_position=4096, beta_fast=1, beta_slow=2)),
    dict(rotary_dim=64, scaling=dict(type="linear", factor=2, beta=1)),
])
def test_refusals(args):
    with pytest.raises(ValueError):
        P.Rotary(**args)


@pytest.mark.parametrize("freq,gain", [([], 1.0), ([1.0] * 7, 1.0), ([math.nan] * 8, 1.0), ([1.0] * 8, math.inf)])
def test_own_frequencies_refused(freq, gain):
    with pytest.raises(ValueError):
        P.Rotary.from_frequencies(freq, gain=gain)


def test_library_refuses_a_null_cache():
    r, got = P.Rotary(64), []

    def call():  # (a thread of its own: the message of the last failure is a thread's)
        st = P.lib().paged_kv_append_rotary(None, None, 0, None, 0, None, 0, 0, None, 0, 0, None, None, None, 0, r._ref,
                                            None, None, ctypes.c_float(0.0), None, 0, None, None)
        got.append((st, P.lib().pkv_last_error()))

    t = threading.Thread(target=call)
    t.start()
    t.join()
    assert got[0][0] == -1 and b"NULL" in got[0][1]
