"""Plain NumPy forms, in 64 bits or in the documented 32-bit steps, of the gated feed-forward
block, the BitLinear gradients and the W8A8 product, for the GPU tests."""
import math

import numpy as np

U = 2.0 ** -24            # half a unit in the last place of fp32, relative
F32 = np.float32


def pack(w_hat):
    """int8 ternary [N, K] -> uint8 [N, K/4], code W + 1 at bits 2 (k % 4)."""
    c = (w_hat + 1).astype(np.uint8).reshape(w_hat.shape[0], -1, 4)
    return c[:, :, 0] | (c[:, :, 1] << 2) | (c[:, :, 2] << 4) | (c[:, :, 3] << 6)


def ternary(rng, n, k):
    return rng.integers(-1, 2, size=(n, k)).astype(np.int8)


def absmax(x):
    """bitlinear_quantize_act in its 32-bit steps."""
    x = x.astype(F32)
    beta = (np.abs(x).max(axis=1) + F32(1e-8)).astype(F32)
    q = np.rint((x * F32(127)) / beta[:, None])
    return np.clip(q, -127, 127).astype(np.int8), beta


def int_product(x_q, w):
    """x_q . w^T, exact."""
    return np.rint(x_q.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)


def project(x_q, beta, w_hat, alpha, bias):
    """bitlinear_forward in its 32-bit steps."""
    s = (np.float64(alpha) * beta.astype(np.float64) / 127.0).astype(F32)
    y = int_product(x_q, w_hat).astype(F32) * s[:, None]
    return y if bias is None else (y + bias).astype(F32)


_erfc = np.vectorize(math.erfc)


def activation(g, act):
    """a(g) and a'(g) in 64 bits."""
    g = g.astype(np.float64)
    if act == "silu":
        s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        sc = np.where(g >= 0, np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))), 1 / (1 + np.exp(-np.abs(g))))
        return g * s, s + g * s * sc
    if act == "relu2":
        r = np.maximum(g, 0)
        return r * r, 2 * r
    cdf = 0.5 * _erfc(-g / math.sqrt(2))
    return g * cdf, cdf + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def gated_gradients(dh, g, u, x_q, beta, wg, ag, wu, au, act):
    """dx, dWg, dWu, dbias_g, dbias_u in 64 bits, and the root sum of squares of the terms of each
    (what the errors of sums are counted in)."""
    a, slope = activation(g, act)
    d = [dh.astype(np.float64) * u * slope, dh.astype(np.float64) * a]
    return _gradients(d, [wg, wu], [ag, au], x_q, beta)


def linear_gradients(dy, x_q, beta, w, alpha):
    return _gradients([dy.astype(np.float64)], [w], [alpha], x_q, beta)


def _gradients(d, ws, alphas, x_q, beta):
    xd = x_q.astype(np.float64) * beta.astype(np.float64)[:, None] / 127
    dx = sum(float(al) * (di @ w.astype(np.float64)) for di, w, al in zip(d, ws, alphas))
    dx2 = np.sqrt(sum(float(al) ** 2 * (di ** 2 @ w.astype(np.float64) ** 2) for di, w, al in zip(d, ws, alphas)))
    dws = [di.T @ xd for di in d]
    dws2 = [np.sqrt((di ** 2).T @ xd ** 2) for di in d]
    dbs = [di.sum(0) for di in d]
    dbs2 = [np.sqrt((di ** 2).sum(0)) for di in d]
    return [dx] + dws + dbs, [dx2] + dws2 + dbs2


def gradient_tolerance(terms, length, total=0.0):
    """Bound on a gradient's error.  A term carries at most 24 half units: a few fp32 roundings of
    a(g), a'(g) and the products that form d (12), the factor alpha or beta / 127 (2), and the 22
    significant bits it is multiplied with (2^-22 = 4).  Each of the `length` additions rounds a
    partial sum by one unit at most (2 half units, whatever the rounding of the matrix cores'
    additions); partial sums stay below about four root sums of squares, and the errors, being
    independent, add as their squares: 2 * 4 * sqrt(length).

    That holds for terms of either sign.  Where they share one (a gradient that follows its input),
    the sum `total` is many root sums of squares, and the partial sum after l of L terms lies near
    total l / L besides: the rounding errors' squares then add up to
    sum_l (2 U total l / L)^2 = 4 U^2 total^2 L / 3, their root 2 U |total| sqrt(L / 3); and the terms'
    own roundings, independent too, stay inside 24 U times the root sum of squares."""
    return U * ((24 + 8 * math.sqrt(length)) * terms + 2 * math.sqrt(length / 3) * np.abs(total))
