"""Plain NumPy forms of the products grouped by expert, in 64 bits or in the documented 32-bit steps."""
import numpy as np

import ffn_plain as plain


def groups(offsets, m):
    """(expert, first row, end) of the groups as they are taken: offsets within 0 .. m."""
    c = np.clip(np.asarray(offsets, dtype=np.int64), 0, m)
    return [(e, int(c[e]), int(c[e + 1])) for e in range(len(c) - 1) if c[e + 1] > c[e]]


def tokens(x_q, beta, rows, m):
    """x_q and beta of every row; indices out of range read zeros."""
    if rows is None:
        return x_q, beta
    t = x_q.shape[0]
    ok = (rows >= 0) & (rows < t)
    r = np.where(ok, rows, 0)
    return np.where(ok[:, None], x_q[r], 0).astype(np.int8), np.where(ok, beta[r], np.float32(0)).astype(np.float32)


def forward(x_q, beta, offsets, w, alpha, bias, y):
    """Rows of y under their experts, in the 32-bit steps of bitlinear_forward; other rows as they are."""
    y = y.copy()
    for e, i, j in groups(offsets, x_q.shape[0]):
        y[i:j] = plain.project(x_q[i:j], beta[i:j], w[e], alpha[e], None if bias is None else bias[e])
    return y


def gate_sizes(dh, g, u, act):
    """What the roundings of dg = dh u a'(g) and du = dh a(g) are counted in: their own sizes, but for SiLU's
    a' = s + g s sc (s, sc the logistic function of g and -g), a sum of two terms that cancel near g = -1.28.
    There the size is |dh u| (s + |g| s sc).  With U half a unit: e = exp(-|g|) carries 4 U; t = 1 / (1 + e)
    at most 2 (from e), 1 (the sum) and 2 (the reciprocal); p = e t then 10; the second term p t and its
    factor g 17; the sum, dh u, its product with a' and alpha one each: 21 U of that size, within the 24
    that gradient_tolerance counts."""
    a, slope = plain.activation(g, act)
    if act == "silu":
        e = np.exp(-np.abs(g.astype(np.float64)))
        s, sc = np.where(g >= 0, 1, e) / (1 + e), np.where(g >= 0, e, 1) / (1 + e)
        slope = s + np.abs(g) * s * sc
    return [np.abs(dh.astype(np.float64) * u * slope), np.abs(dh.astype(np.float64) * a)]


def gradients(d, ws, alphas, x_q, beta, offsets, dx, sizes=None):
    """dx (other rows as given), dW and dbias of every projection in 64 bits, and the root sums of squares
    of their terms (with `sizes` in place of d) and the numbers of terms."""
    m, k = x_q.shape
    e_n, n = ws[0].shape[:2]
    values = [dx.astype(np.float64)] + [np.zeros((e_n, n, k)) for _ in d] + [np.zeros((e_n, n)) for _ in d]
    terms = [np.zeros(v.shape) for v in values]
    length = 1
    p = len(d)
    for e, i, j in groups(offsets, m):
        out, sq = plain._gradients([di[i:j] for di in d], [w[e] for w in ws], [al[e] for al in alphas], x_q[i:j], beta[i:j])
        if sizes is not None:
            sq = plain._gradients([di[i:j] for di in sizes], [w[e] for w in ws], [al[e] for al in alphas], x_q[i:j], beta[i:j])[1]
        length = max(length, j - i)
        values[0][i:j], terms[0][i:j] = out[0], sq[0]
        for q in range(p):
            values[1 + q][e], terms[1 + q][e] = out[1 + q], sq[1 + q]
            values[1 + p + q][e], terms[1 + p + q][e] = out[1 + p + q], sq[1 + p + q]
    lengths = [p * n] + [length] * (2 * p)
    return values, terms, lengths
