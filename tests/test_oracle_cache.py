"""Pins of oracle/cache.py (CPU): the format against its definition by
exhaustive search, the record layout as a permutation, the attention against a
direct softmax."""
import itertools

import numpy as np
import pytest

from oracle import cache as C


def test_scale_is_the_smallest_power_of_two_that_holds_the_block():
    for a in (1e-30, 0.3, 0.4375, 0.43750003, 0.875, 1.0, 1.75, 1.7500001, 7.0, 7.0000005, 8.0, 3.0e38):
        x = np.zeros(32)
        x[5] = -a
        _, e = C.quantise(x)
        s = 2.0 ** (int(e[0]) - 127)
        assert a <= 7 * s or e[0] == 252
        assert a > 7 * s / 2 or e[0] == 3


def test_codes_are_nearest_with_ties_to_even():
    x = np.zeros(32)
    x[0] = 6.0                                                   # scale 1
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    for tie, to in ties.items():
        x[1], x[2] = tie, -tie
        got = C.values(*C.quantise(x))
        assert got[1] == to and got[2] == -to
        x[1], x[2] = np.nextafter(tie, 9), np.nextafter(tie, 0)
        hi, lo = C.values(*C.quantise(x))[1:3]
        assert (lo, hi) == tuple(sorted((lo, hi))) and lo < tie < hi
    x[0] = 7.0
    assert C.values(*C.quantise(x))[0] == 6.0


def test_zero_tiny_and_infinite_blocks():
    x = np.zeros(64)
    codes, e = C.quantise(x)
    assert not codes.any() and (e == 3).all()
    x[:] = 2.0 ** -126                                           # half of the smallest step: to even, 0
    assert not (C.quantise(x)[0] & 7).any()
    x[40] = np.inf
    v = C.values(*C.quantise(x))
    assert np.isnan(v[32:]).all() and not np.isnan(v[:32]).any()


def test_quantised_numbers_are_fixed_points_of_their_scale():
    """A block holding a code of 4 or 6 keeps its numbers when quantised again."""
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (50, 64)).astype(np.uint8)
    codes[:, ::32] = 7
    e = rng.integers(3, 253, (50, 2)).astype(np.uint8)
    v = C.values(codes, e)
    again, e2 = C.quantise(v)
    assert (e == e2).all() and (C.values(again, e2) == v).all()


@pytest.mark.parametrize("page,dim", itertools.product((32, 64, 128, 256), (64, 128, 256)))
def test_a_record_is_filled_without_overlap(page, dim):
    seen = np.zeros(page * (dim + dim // 16), dtype=int)
    for r in range(page):
        k, v, ks, vs = C.places(page, dim, r)
        np.add.at(seen, np.concatenate([k, v]), 1)
        np.add.at(seen, np.concatenate([ks, vs]), 2)
    assert (seen == 2).all()


def test_write_then_read_is_the_quantised_number():
    rng = np.random.default_rng(4)
    page, dim, H = 32, 64, 3
    data = rng.integers(0, 256, (5, H, page * (dim + dim // 16))).astype(np.uint8)
    table = [4, 0, 2]
    want = {}
    for t in (0, 1, 16, 31, 32, 47, 95):
        k, v = rng.standard_normal((2, H, dim))
        C.write(data, table, page, dim, t, k, v)
        want[t] = C.values(*C.quantise(k)), C.values(*C.quantise(v))
    for t, (k, v) in want.items():
        gk, gv = C.read(data, table, page, dim, t)
        assert (gk == k).all() and (gv == v).all()


def test_sees():
    t = np.arange(12)
    assert C.sees(4, 2, 5, t).tolist() == [True] * 7 + [False] * 5
    assert C.sees(4, 2, 5, t, window=3).tolist() == [False] * 4 + [True] * 3 + [False] * 5
    assert C.sees(4, 2, 5, t, bits=0b1101).tolist() == [True] * 5 + [False, True, True] + [False] * 4
    assert C.sees(0, 0, 2, t[:2], bits=0).tolist() == [False, False]
    assert C.sees(4, 0, 1, t, bits=0b11).tolist() == [True] * 5 + [False] * 7    # bits past count


def test_attend_is_a_softmax():
    rng = np.random.default_rng(5)
    q, K, V = rng.standard_normal(64), rng.standard_normal((9, 64)), rng.standard_normal((9, 64))
    o, lse, _, _, _ = C.attend(q, K, V, 0.3)
    w = np.exp(0.3 * K @ q)
    assert np.allclose(o, w @ V / w.sum(), atol=1e-14) and np.isclose(lse, np.log(w.sum()), atol=1e-13)
    o, lse, *_ = C.attend(q, K[:0], V[:0], 0.3)
    assert not o.any() and lse == -np.inf
    K[3, 2] = np.nan
    assert np.isnan(C.attend(q, K, V, 0.3)[0]).all()
