"""The reference of the microscaled cache against closed forms and its own definition."""
import numpy as np
import pytest

from oracle import mx4_ref as M


def test_values_of_all_codes():
    codes = M.pack(np.arange(16, dtype=np.uint8).repeat(2).reshape(1, 32))
    got = M.values(codes, np.array([[127]], np.uint8))[0]
    want = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]
    np.testing.assert_array_equal(got, np.repeat(want, 2))
    assert np.isnan(M.values(codes, np.array([[255]], np.uint8))).all()
    np.testing.assert_array_equal(M.values(codes, np.array([[120]], np.uint8))[0], got / 128)


def test_ties_go_to_the_even_code():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, -0.25, -5.0])
    np.testing.assert_array_equal(M.encode(x), [0, 2, 2, 4, 4, 6, 6, 7, 8, 14])


@pytest.mark.parametrize("top,exp", [(7.0, 0), (7.01, 1), (3.5, -1), (3.51, 0), (6.0, 0), (1.0, -2), (0.0, -126),
                                     (2.0 ** -130, -126), (7 * 2.0 ** -126, -126), (3.3895313892515355e38, 126)])
def test_scale_exponent(top, exp):
    assert M.scale_exponent(np.array([0.0, -top, top / 3])) == exp


def test_no_value_is_off_by_more_than_its_scale():
    rng = np.random.default_rng(2)
    rows = rng.standard_normal((300, 64)) * np.exp2(rng.integers(-20, 20, (300, 1)))
    for row in rows:
        codes, scales = M.quantise(row)
        s = np.repeat(2.0 ** (scales.astype(float) - 127), 32)
        assert np.all(np.abs(M.values(codes, scales) - row) <= s)
        a = np.abs(row.reshape(2, 32)).max(1)
        assert np.all(a <= 7 * s[::32]) and np.all(a > 3.5 * s[::32])


def test_infinities_and_nan():
    row = np.zeros(64)
    row[3], row[5], row[40] = np.inf, 3.0, np.nan
    codes, scales = M.quantise(row)
    v = M.values(codes, scales)
    assert scales[1] == 255 and np.isnan(v[32:]).all() and v[5] == 3.0 and v[3] == 6 * 2.0 ** (int(scales[0]) - 127)


def test_compact_reads_before_it_writes():
    pool = np.arange(4 * 16 * 2).reshape(4, 1, 16, 2)
    got = M.compact(pool, [3, 5, 20, 21], [0, 4], [2], [[1, 3]])
    flat = lambda p: p[[1, 3], 0].reshape(32, 2)  # noqa: E731
    want = flat(pool).copy()
    want[2:6] = flat(pool)[[3, 5, 20, 21]]
    np.testing.assert_array_equal(flat(got), want)
    np.testing.assert_array_equal(got[[0, 2]], pool[[0, 2]])
