"""Pins of the references that the GPU tests of the 4-bit cache, the attention mass and the eviction use, and the
refusals of the library's calls that need no GPU."""
import ctypes

import numpy as np
import pytest

import compress_ref as R


def test_a_row_of_sixteen_steps_is_exact():
    x = np.arange(16, dtype=np.float64)[None] - 5.0
    codes, step, low = R.quantise4(x, "f16")
    assert step[0] == 1.0 and low[0] == -5.0 and list(codes[0]) == list(range(16))
    assert np.array_equal(R.values4(codes, step, low), x)


@pytest.mark.parametrize("model", ["f16", "bf16"])
def test_values_are_within_half_a_step(model):
    rng = np.random.default_rng(3)
    x = R.round_model(rng.normal(size=(200, 128)) * 10.0 ** rng.uniform(-3, 3, size=(200, 1)), model)
    codes, step, low = R.quantise4(x, model)
    err = np.abs(R.values4(codes, step, low) - x)
    # half a step, plus what rounding the step moves the top code by (15 half-steps of the type's spacing)
    assert np.all(err <= step[:, None] * (0.5 + 15 * R.HALF_STEP[model] + 1e-6))


def test_special_rows():
    x = np.zeros((4, 8))
    x[0] = 3.0                 # constant
    x[1, 2] = np.nan
    x[2, 5] = np.inf
    x[3, 1] = 1e-39            # a range whose step is below 2^-126
    codes, step, low = R.quantise4(x, "bf16")
    assert step[0] == 0 and low[0] == 3.0 and not codes[0].any()
    assert np.isnan(step[1]) and np.isnan(low[1]) and np.isnan(step[2])
    assert step[3] == 0 and not codes[3].any()


def test_attention_of_equal_keys_is_the_mean():
    k = np.ones((5, 2, 4))
    v = np.arange(40, dtype=np.float64).reshape(5, 2, 4)
    out, p, _, _ = R.attention(np.ones((4, 4)), k, v, 0.5)
    assert np.allclose(p, 0.2) and np.allclose(out[0], v[:, 0].mean(0)) and np.allclose(out[3], v[:, 1].mean(0))


def test_evict_ties_recent_and_short_rows():
    m = [1, 5, 5, 0, 5, 2, 9]
    assert R.evict(m, 7, 4, 2) == [1, 2, 5, 6]
    assert R.evict(m, 7, 3, 3) == [4, 5, 6]
    assert R.evict(m, 7, 2, 0) == [1, 6]
    assert R.evict(m, 3, 4, 2) == [0, 1, 2]
    assert R.evict([float("nan"), 0.0, -1.0, 2.0], 4, 2, 0) == [1, 3]


@pytest.fixture(scope="module")
def library():
    from paged_kv_cache_134_gb300 import build
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    build.build()
    import paged_kv_cache_134_gb300 as P
    return P.lib()


def test_null_cache_is_refused_before_any_gpu_work(library):
    f = ctypes.c_float
    assert library.paged_kv_gather(None, None, 1, None, None, None) == -1
    assert library.paged_decode_attention_mass(None, None, None, 1, None, 1, 1, f(1), f(1), None, 1, None, None) == -1
    assert library.paged_kv_evict(None, None, 1, None, 1, None, 1, 1, 0, None, 1, None, None, None, 1, None) == -1
    assert b"NULL" in library.pkv_last_error()


@pytest.mark.parametrize("kv,model,status", [(4, 0, -1), (3, 3, -1), (3, 2, -1)])
def test_bad_dtypes_are_refused(library, kv, model, status):
    h = ctypes.c_void_p()
    assert library.kv_cache_create(4, 16, 1, 64, kv, model, ctypes.byref(h)) == status and not h


def test_int4_cache_shapes_are_refused_like_any(library):
    h = ctypes.c_void_p()
    assert library.kv_cache_create(4, 16, 1, 96, 3, 0, ctypes.byref(h)) == -4
    assert library.kv_cache_create(4, 24, 1, 64, 3, 0, ctypes.byref(h)) == -4
