"""Pins of the decoding oracle (CPU): the quantiser against exact rational arithmetic, attention against a
plain softmax, the page choice against enumeration."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import cache_oracle as co


def _bf16_values():
    """Every finite bf16 near 1 and a spread of others, as Fractions' float sources."""
    out = []
    for e in (-100, -3, 0, 5, 90):
        out += [float(np.ldexp(128 + k, e - 7)) for k in range(0, 128, 17)]
    return out


@pytest.mark.parametrize("v", _bf16_values())
def test_bf16_roundings(v):
    step = float(np.spacing(np.float32(v))) * 65536
    for f in (0.0, 0.25, 0.5, 0.75):
        x = v + f * step
        assert co.floor_bf16(np.array([x]))[0] == v
        assert co.floor_bf16(np.array([-x]))[0] == (-v if f == 0 else -(v + step))
        near = co.round_bf16(np.array([x]))[0]
        odd = int(round(v / step)) % 2 == 1
        want = v if f < 0.5 or (f == 0.5 and not odd) else v + step
        assert near == want


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("group", [32, 64])
def test_codes_against_rationals(seed, group):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(64).astype(np.float32)
    if seed % 2:  # bf16 values on a coarse grid: exact ties occur
        x = np.round(x * 4) / 4
    c, s, z = co.oracle_quantise(x.astype(np.float64), group)
    for i, xi in enumerate(x):
        g = i // group
        fs, fz = Fraction(float(s[g])), Fraction(float(z[g]))
        part = [Fraction(float(t)) for t in x[g * group:(g + 1) * group]]
        assert fz <= min(part)
        # s is a nearest bf16 to (max - z) / 15
        exact = (max(part) - fz) / 15
        m, e = np.frexp(float(s[g]))
        ulp = Fraction(2) ** int(e - 8)
        assert abs(fs - exact) <= ulp / 2
        t = (Fraction(float(xi)) - fz) / fs
        lo = t.numerator // t.denominator
        f = t - lo
        want = lo if f < Fraction(1, 2) else lo + 1 if f > Fraction(1, 2) else lo + lo % 2
        assert c[i] == min(15, want)


def test_quantiser_special_groups():
    x = np.zeros((7, 32))
    x[1] = 3.0
    x[2, 5] = np.inf
    x[3, 0] = np.nan
    x[4, :2] = [3e38, -3e38]
    x[5] = 2.0 ** -120 * np.arange(32)
    x[6] = -1.5
    c, s, z = co.oracle_quantise(x, 32)
    assert (c[[0, 1, 2, 3, 4, 5, 6]] == 0).all()
    assert np.isnan(s[[2, 3, 4], 0]).all()
    assert (s[[0, 1, 5, 6], 0] == 0).all()
    st = co.oracle_stored(x, 32)
    assert (st[1] == 3.0).all() and (st[6] == -1.5).all() and np.isnan(st[2]).all()


def test_stored_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 128)).astype(np.float32).astype(np.float64)
    c, s, z = co.oracle_quantise(x, 64)
    err = np.abs(co.oracle_stored(x, 64) - x).reshape(50, 2, 64)
    # half a step inside the range; s rounded down by up to 2^-9 leaves 15 * 2^-9 of a step at its end
    assert (err <= s[..., None] * (0.5 + 15 * 2.0 ** -9)).all()


def test_attend_row_is_a_softmax():
    rng = np.random.default_rng(4)
    K, V, q = rng.standard_normal((9, 8)), rng.standard_normal((9, 8)), rng.standard_normal(8)
    inv = co.oracle_key_inv(K)
    out, lse, w, keys = co.oracle_cache_attend_row(q, K, V, inv, 5, 9, None, 16, True, True, True, None)
    assert list(keys) == [0, 1, 2, 3, 4]
    z = (K[:5] / np.linalg.norm(K[:5], axis=1, keepdims=True)) @ q / np.sqrt(8)
    e = np.exp(z)
    assert np.allclose(out, e @ V[:5] / e.sum()) and np.isclose(lse, np.log(e.sum()))
    # the only key is its own; nothing at all; a page twice
    assert list(co.oracle_cache_attend_row(q, K, V, inv, 0, 9, None, 16, True, True, True, None)[3]) == [0]
    assert co.oracle_cache_attend_row(q, K, V, inv, 5, 9, [], 4, True, True, True, None)[1] == -np.inf
    _, l2, _, k2 = co.oracle_cache_attend_row(q, K, V, inv, 8, 9, [0, 0, 7], 4, True, True, True, None)
    _, l1, _, _ = co.oracle_cache_attend_row(q, K, V, inv, 8, 9, [0], 4, True, True, True, None)
    assert list(k2) == [0, 1, 2, 3] * 2 and np.isclose(l2, l1 + np.log(2))


def test_select_orders_by_score_then_page():
    tags = np.array([[1, 1, 2, 2, 1, 3, 1, 1]])
    sel, sc = co.oracle_cache_select(tags, np.array([[1]]), 7, 8, 2, 6, 3, 0, True)
    assert sc == [2, 0, 1, 2, -1, -1] and sel == [0, 2, 3]
    sel, _ = co.oracle_cache_select(tags, np.array([[1]]), 7, 8, 2, 6, 2, 1, True)
    assert sel == [0, 3]
    sel, sc = co.oracle_cache_select(tags, np.array([[1]]), 2, 8, 2, 6, 4, 1, True)
    assert sel == [0, 1, -1, -1] and sc[:3] == [2, 0, -1]
