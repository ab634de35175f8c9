"""The three parts that the linear attention's state product takes for a decayed value,
restated in numpy bit for bit: exact, none of a number's zero or of another sign (so
that an infinity times the parts, or an infinity's parts, do not meet in NaN), and
needed all three: the tests of the returned states' precision would see two."""
import numpy as np
import pytest

U32 = 2.0 ** -24


def _sub1(x):
    bits = x.view(np.uint32)
    return np.where(bits == 0, np.uint32(0), bits - np.uint32(1)).astype(np.uint32).view(np.float32)


def _cut(x):
    return (x.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)


def split3(x):
    with np.errstate(all="ignore"):
        x = x + np.float32(0)  # never -0
        a = _cut(_sub1(x))
        b = _cut(_sub1(x - a))
        return a, b, _cut(x - a - b)


def _values():
    rng = np.random.default_rng(1)
    bits = rng.integers(0, 1 << 32, 2000000, dtype=np.uint64).astype(np.uint32)
    x = bits.view(np.float32)
    few = (rng.integers(0, 1 << 16, 300000, dtype=np.uint64).astype(np.uint32) << 16).view(np.float32)  # bf16 values
    low = (few.view(np.uint32) | rng.integers(0, 4, few.size, dtype=np.uint64).astype(np.uint32)).view(np.float32)
    powers = np.float32(2.0) ** np.arange(-100, 128, dtype=np.float32)
    x = np.concatenate([x, few, low, powers, -powers])
    return x[np.isfinite(x) & (np.abs(x) > 2.0 ** -100)]


def test_parts_of_a_number_are_exact_and_of_one_sign():
    x = _values()
    a, b, c = split3(x)
    assert (a.astype(np.float64) + b + c == x).all()
    for p in (a, b, c):
        assert (np.sign(p) == np.sign(x)).all()


def test_parts_of_zeros_infinities_and_nan():
    for z in (0.0, -0.0):
        assert all(p == 0 for p in split3(np.array([z], np.float32)))
    for s in (1, -1):
        a, b, c = split3(np.array([s * np.inf], np.float32))
        assert np.isfinite(a) and np.isfinite(b) and a * s > 0 and b * s > 0 and c == s * np.inf
    for bits in (0x7fc00000, 0x7f800001, 0xffc00000, 0xff800001, 0x7fffffff):
        with np.errstate(all="ignore"):
            a, b, c = split3(np.array([bits], np.uint32).view(np.float32))
            assert np.isnan(a + b + c)


@pytest.mark.parametrize("units", [19, 250])  # the tightest and the loosest bound of those tests
def test_two_parts_would_be_seen(units):
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(128) * np.exp(-0.05 * rng.random(128))).astype(np.float32)
    a, b, c = split3(x)
    assert (np.abs(a.astype(np.float64) + b - x) > units * U32 * np.abs(x)).any()
