"""The 8-bit pre-fill's planner, on the host (no GPU): into how many runs a
retrieval item's key tiles are cut, through the C ABI's testing hooks."""

import numpy as np
import pytest

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import build as BUILD

SMS = 148
PARTIALS = 296  # items x runs that the workspace holds


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.lib()


def _cache(hq, hkv, n_ret, kv="fp8", batch=1, D=128):
    return B.duo_cache_create(layers=1, batch=batch, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, kv_dtype=kv,
                              capacity=1 << 20, head_mask=[1] * n_ret + [0] * (hkv - n_ret), S=4, R=60)


def _plan(lens, C, hq, hkv, n_ret, kv="fp8", sms=SMS, forced=0):
    h = _cache(hq, hkv, n_ret, kv, len(lens))
    try:
        if forced:
            B.duo_test_force_prefill_runs(h, forced)
        return B.duo_test_plan_prefill(h, 0, lens, C, sms)
    finally:
        B.duo_cache_destroy(h)


@pytest.mark.parametrize("lens,C,hq,hkv,n_ret", [
    ([4000], 7, 8, 2, 1), ([3000], 300, 8, 4, 2), ([5000, 40], 20, 4, 2, 1), ([1, 2000, 130], 129, 6, 2, 2),
    ([2500], 1, 16, 2, 1), ([4000], 7, 8, 2, 1), ([3001], 300, 8, 2, 1), ([15000], 1000, 32, 8, 4)])
def test_shapes_that_split(lib, lens, C, hq, hkv, n_ret):
    """The shapes whose outputs the GPU tests compare are cut into runs."""
    assert _plan(lens, C, hq, hkv, n_ret) > 1
    assert _plan(lens, C, hq, hkv, n_ret, "bf16") == _plan(lens, C, hq, hkv, n_ret, "int4") == 1


def test_no_split(lib):
    assert _plan([0], 128, 8, 2, 1) == 1         # one tile
    assert _plan([10000], 4096, 32, 8, 8) == 1   # items for every SM
    assert _plan([10000], 100, 8, 2, 0) == 1     # no retrieval head


def test_partials_fit_the_workspace(lib):
    r = np.random.default_rng(5)
    for _ in range(300):
        hkv = int(r.choice([1, 2, 4, 8]))
        g, n_ret, rows = int(r.integers(1, 9)), int(r.integers(1, hkv + 1)), int(r.integers(1, 9))
        lens = [int(2 ** r.uniform(0, 17)) for _ in range(rows)]
        C, sms = int(2 ** r.uniform(0, 12)), int(r.choice([1, 84, 132, 148, 160]))
        items = rows * n_ret * g * -(-C // 256)
        tiles = -(-max(lens) // 128) + -(-C // 128)
        runs = _plan(lens, C, g * hkv, hkv, n_ret, sms=sms)
        assert runs == 1 or (items * runs <= PARTIALS and 2 <= runs <= tiles)
        forced = int(r.integers(1, PARTIALS + 1))
        runs = _plan(lens, C, g * hkv, hkv, n_ret, sms=sms, forced=forced)
        assert runs == max(1, min(forced, PARTIALS // items))


def test_hook_arguments(lib):
    h = _cache(8, 2, 1)
    try:
        for lens, C, sms in (([], 4, SMS), ([-1], 4, SMS), ([5] * 129, 4, SMS), ([5], 0, SMS), ([5], 4, 0)):
            with pytest.raises(B.DuoError) as e:
                B.duo_test_plan_prefill(h, 0, lens, C, sms)
            assert e.value.name == "DUO_ERR_ARG"
        with pytest.raises(B.DuoError):
            B.duo_test_plan_prefill(h, 1, [5], 4, SMS)
        for runs in (-1, PARTIALS + 1):
            with pytest.raises(B.DuoError) as e:
                B.duo_test_force_prefill_runs(h, runs)
            assert e.value.name == "DUO_ERR_ARG"
    finally:
        B.duo_cache_destroy(h)
    h = _cache(8, 2, 1, "bf16")
    try:
        with pytest.raises(B.DuoError) as e:
            B.duo_test_force_prefill_runs(h, 2)
        assert e.value.name == "DUO_ERR_UNSUPPORTED"
    finally:
        B.duo_cache_destroy(h)
    h = _cache(8, 2, 1, "f32", D=64)
    try:
        with pytest.raises(B.DuoError) as e:
            B.duo_test_plan_prefill(h, 0, [5], 4, SMS)
        assert e.value.name == "DUO_ERR_UNSUPPORTED"
    finally:
        B.duo_cache_destroy(h)
