"""Data of the fp8 product whose every partial sum, in any order, is an fp32 number, and its exact values."""
import numpy as np

F32 = np.float32


def _scaled(x, xs, w, ws):
    """sum_b xs[b, m] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k] in 64 bits."""
    b = np.arange(x.shape[1]) // 128
    return (x * xs.T[:, b]).astype(np.float64) @ (w * ws[np.arange(w.shape[0]) // 128][:, b]).astype(np.float64).T


def integers(rng, m, k, n):
    """Integers up to 4 and scales 2^-1 .. 2^1: a term is at most 4 * 4 * 2 * 2 = 2^6 and a multiple of 2^-2, so a sum of
    K of them is at most 2^8 K steps of 2^-2: an fp32 number for K up to 2^16."""
    assert k <= 1 << 16
    x, w = rng.integers(-4, 5, (m, k)).astype(F32), rng.integers(-4, 5, (n, k)).astype(F32)
    xs = np.exp2(rng.integers(-1, 2, (-(-k // 128), m))).astype(F32)
    ws = np.exp2(rng.integers(-1, 2, (-(-n // 128), -(-k // 128)))).astype(F32)
    return x, xs, w, ws, _scaled(x, xs, w, ws)


def wide(rng, m, k, n):
    """Every eight neighbouring k hold two large products, +-2^16 and its negative, and six of 2^-2 .. 2^2 with either sign:
    2^14 to 2^18 times smaller.  A block's partial sums are at most 16 * 2^16 + 96 * 2^2 < 2^21 and multiples of 2^-2,
    so they are fp32 numbers; the large ones cancel in every block, and what is left, at most 96 * 2^2 for each, is a
    multiple of 2^-2 too: below 2^24 steps for K up to 2^20."""
    assert k % 8 == 0 and k <= 1 << 20
    x = (np.exp2(rng.integers(-1, 2, (m, k))) * rng.choice([-1, 1], (m, k))).astype(F32)
    w = np.exp2(rng.integers(-1, 2, (n, k))).astype(F32)
    sign = rng.choice([-1, 1], (m, k // 8)).astype(F32)
    for g in range(k // 8):
        i, j = 8 * g + rng.permutation(8)[:2]
        x[:, i], x[:, j] = 256 * sign[:, g], -256 * sign[:, g]
        w[:, i] = w[:, j] = 256
    xs, ws = np.ones((-(-k // 128), m), F32), np.ones((-(-n // 128), -(-k // 128)), F32)
    return x, xs, w, ws, _scaled(x, xs, w, ws)


def dropping(x, w, bits):
    """The product if, of every eight neighbouring k, products below 2^-bits of the largest were lost."""
    y = np.zeros((x.shape[0], w.shape[0]))
    for g in range(0, x.shape[1], 8):
        p = x[:, None, g:g + 8].astype(np.float64) * w[None, :, g:g + 8]
        y += np.where(np.abs(p) >= np.abs(p).max(axis=2, keepdims=True) * 2.0 ** -bits, p, 0).sum(axis=2)
    return y
