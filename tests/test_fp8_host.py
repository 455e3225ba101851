"""What the data of the fp8 product's tests can tell apart, on the CPU."""
import numpy as np
import pytest

import fp8_plain


def _e4m3(v):
    """Whether every element is an e4m3 number."""
    m = np.abs(v.astype(np.float64))
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(m, 2.0 ** -6))), -6) - 3)
    return bool(np.all(m <= 448) and np.all(np.rint(m / step) * step == m))


@pytest.mark.parametrize("k", [128, 264])
def test_wide_products_need_every_bit(k):
    """Products 2^-13 of their group's largest lost, and the sums are off by far more than a rounding; kept to 2^-18, and
    none is."""
    rng = np.random.default_rng([1, k])
    x, xs, w, ws, want = fp8_plain.wide(rng, 12, k, 20)
    assert _e4m3(x) and _e4m3(w) and np.array_equal(want.astype(np.float32), want)
    lost = fp8_plain.dropping(x, w, 13)
    assert np.all(lost == 0) and np.count_nonzero(want) > 0.9 * want.size
    assert np.array_equal(fp8_plain.dropping(x, w, 18), want)
    # partial sums in fp32, forwards and backwards
    for order in (np.arange(k), np.arange(k)[::-1]):
        acc = np.zeros(want.shape, np.float32)
        for i in order:
            acc = acc + np.outer(x[:, i], w[:, i]).astype(np.float32)
        assert np.array_equal(acc, want)


def test_integers_are_exact():
    rng = np.random.default_rng(2)
    x, xs, w, ws, want = fp8_plain.integers(rng, 5, 4000, 130)
    assert _e4m3(x) and _e4m3(w) and np.array_equal(want.astype(np.float32), want)
    b = np.arange(4000) // 128
    acc = np.zeros(want.shape, np.float32)
    for i in range(4000):
        term = np.outer(x[:, i] * xs[b[i]], w[:, i] * ws[np.arange(130) // 128, b[i]]).astype(np.float32)
        acc = acc + term
    assert np.array_equal(acc, want)
    # a scale one block off, and two blocks exchanged, are seen
    assert not np.array_equal(fp8_plain._scaled(x, np.roll(xs, 1, 0), w, ws), want)
    swapped = np.concatenate([x[:, 128:256], x[:, :128], x[:, 256:]], axis=1)
    assert not np.array_equal(fp8_plain._scaled(swapped, xs, w, ws), want)
