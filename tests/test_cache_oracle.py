"""Pins of the cache operators' fp64 oracle: worked examples and properties that do not restate its formulas."""
import numpy as np
import pytest

from oracle import cache_ops as C


def test_codes_of_the_grid_and_its_midpoints():
    x = np.zeros(32)
    x[:16] = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5]
    x[16:20] = [5, 7, -5, 0.26]
    code, scale = C.quantise(x)
    assert scale.tolist() == [127]  # the largest magnitude, 7, lies in [4, 8)
    assert code[:10].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 9, 15]
    # ties go to the even code, 7 saturates
    assert code[10:20].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 14, 1]


def test_scale_bytes():
    for amax, want in ((0.0, 0), (4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (2.0 ** -124, 1), (2.0 ** -133, 1),
                       (3.0e38, 252), (np.inf, 255), (np.nan, 255)):
        x = np.zeros(32)
        x[5] = amax
        assert C.quantise(x)[1].tolist() == [want], amax


def test_quantising_what_was_read_changes_nothing():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 128)) * 2.0 ** rng.integers(-30, 30, (40, 1))
    once = C.values(*C.quantise(x))
    step = np.abs(x).reshape(40, 4, 32).max(-1).repeat(32, -1)
    # between two codes half a step at most; saturation takes up to a quarter of the largest magnitude
    assert (np.abs(once - x) <= step / 4).all()
    assert (C.values(*C.quantise(once)) == once).all()


@pytest.mark.parametrize("D", [64, 128])
def test_records_hold_every_code_once(D):
    rng = np.random.default_rng(4)
    record = np.full(17 * D, 255, np.uint8)
    want = {}
    for is_v in (False, True):
        for slot in range(16):
            code, scale = rng.integers(0, 16, D), rng.integers(0, 256, D // 32)
            C.put(record, slot, D, is_v, code, scale)
            want[is_v, slot] = code, scale
    for is_v in (False, True):
        code, scale = C.get(record, D, is_v)
        for slot in range(16):
            assert (code[slot] == want[is_v, slot][0]).all() and (scale[slot] == want[is_v, slot][1]).all()


def test_eviction_worked_example():
    # eight tokens, budget five, two recent: of slots 0-5 the three best are 4 (9), 1 (7) and 3 (5, before the other 5)
    scores = np.array([1.0, 7, 2, 5, 9, 5, 0, 0])
    assert C.evict_source(scores, 8, 5, 2) == [3, 1, 4, 6, 7]
    assert C.evict_source(scores, 8, 5, 5) == [3, 4, 5, 6, 7]
    assert C.evict_source(scores, 8, 0, 0) == []
    assert C.evict_source(np.array([np.nan, -np.inf, 1.0, np.nan]), 4, 2, 0) == [0, 2]


def test_weights_sum_to_the_group():
    rng = np.random.default_rng(5)
    out, w, reach, _ = C.attend(rng.standard_normal((8, 64)), rng.standard_normal((2, 33, 64)),
                                np.ones((2, 33, 64)), 0.125, 4)
    assert np.allclose(w.sum(1), 4) and np.allclose(out, 1) and np.allclose(reach, 1)
