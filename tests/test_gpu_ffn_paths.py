"""GPU tests of the gated feed-forward block, the BitLinear gradients and the W8A8 product, path by
path: every kernel instance that the choices by size, alignment and type can take, values at the ends
of the range, and calls on a stream that is not the current one."""
import numpy as np
import pytest

import ffn_plain as plain
from ffn_plain import U
from test_gpu_ffn import _code, _f32, _layer, _np, _say, _step, _step_state, _t, dev  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- streams
def test_buffers_of_a_given_stream_leave_queued_work_alone(dev):  # noqa: F811
    """Tensors dropped while the current stream still has work on them queued, of the sizes that calls
    on another stream then allocate: the queued work and the calls both give what they would alone."""
    torch, bl = dev
    m, k, f = 96, 512, 700
    s = _step_state(torch, bl, m, k, f, 41)
    want = [t.clone() for t in _step(torch, bl, s)]
    sizes = [4 * m * f, 4 * m * k, 4 * f * k, 4 * f * k, m * k, 4 * m, bl.bitlinear_gated_backward_workspace_size(m, k, f),
             bl.bitlinear_backward_workspace_size(m, f, k)]
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for rep in range(3):
        _say(f"dropped tensors, repetition {rep}")
        dropped = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        out = torch.empty(4096, 4096, device="cuda")
        for _ in range(10):
            torch.mm(busy, busy, out=out)
        sums = []
        for i, t in enumerate(dropped):
            t.fill_(i + 1)
        torch.mm(busy, busy, out=out)
        for t in dropped:
            sums.append(t.to(torch.int64).sum())
        del t, dropped
        h = bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], stream=side)
        dx, dwg, dwu, _, _ = bl.bitlinear_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["Wg"], s["ag"],
                                                         s["Wu"], s["au"], s["act"], stream=side)
        _, dwd, _ = bl.bitlinear_backward(s["dy"], s["h_q"], s["hbeta"], s["Wd"], s["ad"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        got = [h.clone(), dx.clone(), dwg.clone(), dwu.clone(), dwd.clone()]
        # handed back to the allocator before the copies have run, and asked for again on the other stream
        del h, dx, dwg, dwu, dwd
        bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], stream=side)
        torch.cuda.synchronize()
        assert [int(v) for v in sums] == [(i + 1) * n for i, n in enumerate(sizes)]
        assert all(torch.equal(a, b) for a, b in zip(got, [want[0], want[4], want[5], want[6], want[3]]))


# ------------------------------------------------------------------- values at the ends of the range
def _gates():
    """Gates over the whole range, the borders of the exponential's range densely."""
    ends = [0.0, -0.0, -88.0, 88.0, -87.33, -87.34, 3e38, -3e38, 1e-40, -1e-40, 1e-38, -1e-38]
    g = np.concatenate([np.linspace(-90, -85, 4001), np.linspace(80, 130, 2001), np.linspace(-140, 140, 8001),
                        np.linspace(-9, 9, 8001), ends])
    return _f32(g)


NOT_FINITE = _f32([np.inf, -np.inf, np.nan, -np.nan])


def _limits(act):
    """a and a' at NOT_FINITE (SiLU and its slope at -infinity: within the bounds of their zero limits)."""
    nan = np.nan
    return {"silu": ([np.inf, 0, nan, nan], [1, 0, nan, nan]), "gelu": ([np.inf, nan, nan, nan], [1, 0, nan, nan]),
            "relu2": ([np.inf, 0, nan, nan], [np.inf, 0, nan, nan])}[act]


def _same(got, want, slack):
    nan = np.isnan(want)
    inf = np.isinf(want)
    rest = ~nan & ~inf
    return (np.array_equal(np.isnan(got), nan) and np.array_equal(got[inf], np.asarray(want)[inf])
            and bool(np.all(np.abs(got[rest] - np.asarray(want)[rest]) <= slack)))


@pytest.mark.parametrize("act", ["gelu", "silu", "relu2"])
@pytest.mark.parametrize("m", [1, 2, 70])
def test_gated_forward_activation_over_the_range(dev, act, m):  # noqa: F811
    """The gate driven through its bias (all codes zero), u = 1: h is a(g).  One token, the streaming
    kernel, the GEMM (2 x 173 tiles).  Bounds: the header's for SiLU; one rounding for squared ReLU, and
    for GELU one rounding of a value that 64 bits hold to a few 2^-53 times its exponent's size."""
    torch, bl = dev
    g = np.concatenate([_gates(), NOT_FINITE])
    f, end = len(g), len(NOT_FINITE)
    _say(f"activation over the range {act} M={m} F={f}")
    x = torch.zeros(m, 64, device="cuda")
    w = torch.full((f, 16), 0x55, dtype=torch.uint8, device="cuda")
    al = torch.ones(1, device="cuda")
    gk, uk = torch.empty(m, f, device="cuda"), torch.empty(m, f, device="cuda")
    h = bl.bitlinear_gated_forward(x, w, al, w, al, _code(bl, act), bias_g=_t(torch, g), bias_u=torch.ones(f, device="cuda"),
                                   g=gk, u=uk)
    h2 = bl.bitlinear_gated_forward(x, w, al, w, al, _code(bl, act), bias_g=_t(torch, g), bias_u=torch.ones(f, device="cuda"))
    h, h2 = _np(h).astype(np.float64), _np(h2).astype(np.float64)
    assert np.array_equal(h, h2, equal_nan=True)
    with np.errstate(over="ignore"):
        ref = plain.activation(g[:-end], act)[0]
    for row in h:
        got = row[:-end]
        big = np.abs(ref) > np.finfo(np.float32).max
        assert np.all(np.isinf(got[big])) and np.all(np.isfinite(got[~big]))
        n, low = {"silu": (7, 2.0 ** -120), "gelu": (1.001, 2.0 ** -149), "relu2": (1, 2.0 ** -150)}[act]
        err = np.abs(got[~big] - ref[~big]) - n * U * np.abs(ref[~big]) - low
        assert err.max() <= 0, (float(g[:-end][~big][err.argmax()]), float(err.max()))
        assert _same(row[-end:], _limits(act)[0], 2.0 ** -120)


@pytest.mark.parametrize("act", ["gelu", "silu", "relu2"])
@pytest.mark.parametrize("m", [1, 20, 70])
def test_gated_backward_activation_over_the_range(dev, act, m):  # noqa: F811
    """dh = u = 1 in the first token, zero in the others: the bias sums are a'(g) and a(g).  One pass, one
    pass on the matrix cores, panels (too many tiles for one pass).  Roundings of SiLU: the exponential 4,
    1 + e 1, its reciprocal 2, e / (1 + e) 1, so 8 of s and s(-g) and 9 of a; 18 of g s s(-g) and the sum's,
    so at most 20 of the parts of a'.  An exponential below 2^-126 is zero: 2^-119 with the factor g.  The
    others have fewer."""
    torch, bl = dev
    g = np.concatenate([_gates(), NOT_FINITE])
    k = {1: 4, 20: 4, 70: 2052}[m]
    f, end = len(g), len(NOT_FINITE)
    _say(f"slopes over the range {act} M={m} F={f} K={k}")
    dh = torch.zeros(m, f, device="cuda")
    dh[0] = 1
    gk, u = torch.zeros(m, f, device="cuda"), torch.ones(m, f, device="cuda")
    gk[0] = _t(torch, g)
    x_q = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    w = torch.full((f, k // 4), 0x55, dtype=torch.uint8, device="cuda")
    al, beta = torch.ones(1, device="cuda"), torch.ones(m, device="cuda")
    dbg, dbu = torch.empty(f, device="cuda"), torch.empty(f, device="cuda")
    bl.bitlinear_gated_backward(dh, gk, u, x_q, beta, w, al, w, al, _code(bl, act), dbias_g=dbg, dbias_u=dbu)
    gd = g[:-end].astype(np.float64)
    with np.errstate(over="ignore"):
        a, slope = plain.activation(g[:-end], act)
    e = np.exp(-np.abs(gd))
    cdf = np.where(gd != 0, a / np.where(gd != 0, gd, 1), 0.5)                 # or s(g)
    parts = {"silu": cdf + np.abs(gd) * e, "gelu": cdf + 0.4 * np.abs(gd) * np.exp(-gd * gd / 2), "relu2": np.abs(slope)}[act]
    got_a, got_s = _np(dbu).astype(np.float64), _np(dbg).astype(np.float64)
    big = np.abs(a) > np.finfo(np.float32).max
    big_s = np.abs(slope) > np.finfo(np.float32).max
    assert np.all(np.isinf(got_a[:-end][big])) and np.all(np.isinf(got_s[:-end][big_s]))
    # GELU's tail below -8 is good to 1e-14 absolute
    low = 1e-14 if act == "gelu" else 2.0 ** -119
    assert np.all(np.abs(got_a[:-end][~big] - a[~big]) <= 12 * U * np.abs(a[~big]) + low)
    assert np.all(np.abs(got_s[:-end][~big_s] - slope[~big_s]) <= 20 * U * parts[~big_s] + low)
    assert _same(got_a[-end:], _limits(act)[0], 0) and _same(got_s[-end:], _limits(act)[1], 0)


# ------------------------------------------------------ gradients of very different sizes in a row
# (M, K, N): one pass in fp32; one pass on the matrix cores, one group of tokens and several; panels, with
# up to 64 tokens, with sums in parts and whole
RANGES = [(12, 132, 90), (40, 132, 90), (64, 260, 130), (150, 132, 90), (64, 2052, 2100), (300, 1028, 1100),
          (700, 132, 4100)]


def _within(got, want, terms, length, name, slack=0.0):
    """Every element within its own bound: gradient_tolerance counts the terms that enter it."""
    err = np.abs(got.astype(np.float64) - want)
    tol = plain.gradient_tolerance(terms, length) + slack
    bad = err > tol
    assert not bad.any(), (name, int(bad.sum()), float((err[bad] / np.maximum(np.abs(want[bad]), 1e-300)).max()))


@pytest.mark.parametrize("m,k,n", RANGES)
@pytest.mark.parametrize("s", [20, 24, 30, 45])
def test_backward_dominated_by_one_token_and_one_channel(dev, m, k, n, s):  # noqa: F811
    """A token and a channel 2^s larger than the others, whose code and whose weights are zero in every
    third column: there the sums are those of the others, and hold their own accuracy."""
    torch, bl = dev
    _say(f"backward dominated M={m} K={k} N={n} 2^{s}")
    rng = np.random.default_rng([60, m, k, n, s])
    dy = rng.standard_normal((m, n))
    dy[m // 2] *= 2.0 ** s
    dy[:, n // 3] *= 2.0 ** s
    dy = _f32(dy)
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    x_q[m // 2, ::3] = 0
    w, al, _ = _layer(rng, n, k, False)
    w[n // 3, ::3] = 0
    dx, dw, _ = bl.bitlinear_backward(_t(torch, dy), _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    want, terms = plain.linear_gradients(dy, x_q, beta, w, al[0])
    _within(_np(dx), want[0], terms[0], n, "dx")
    _within(_np(dw), want[1], terms[1], m, "dW")


@pytest.mark.parametrize("m,k,n", RANGES)
@pytest.mark.parametrize("gated", [False, True])
def test_backward_over_a_hundred_binades(dev, m, k, n, gated):  # noqa: F811
    """Elements of sizes spread over 2^-100 .. 1, most codes and weights zero, so that in many columns
    the largest elements are absent; rows and columns of zeros among them."""
    torch, bl = dev
    _say(f"backward hundred binades M={m} K={k} N={n} gated={gated}")
    rng = np.random.default_rng([61, m, k, n])
    dy = _f32(rng.standard_normal((m, n)) * np.exp2(rng.integers(-100, 1, (m, n))))
    dy[1] = 0
    dy[:, 2] = 0
    sparse = lambda a, keep: (a * (rng.random(a.shape) < keep)).astype(np.int8)
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    x_q = sparse(x_q, 0.2)
    tx, tb = _t(torch, x_q), _t(torch, beta)
    w0, al, _ = _layer(rng, n, k, False)
    w0 = sparse(w0, 0.2)
    if not gated:
        dx, dw, _ = bl.bitlinear_backward(_t(torch, dy), tx, tb, _t(torch, plain.pack(w0)), _t(torch, al))
        want, terms = plain.linear_gradients(dy, x_q, beta, w0, al[0])
        _within(_np(dx), want[0], terms[0], n, "dx")
        _within(_np(dw), want[1], terms[1], m, "dW")
        assert not dx[1].any() and not dw[2].any()
        return
    w1, al1, _ = _layer(rng, n, k, False)
    w1 = sparse(w1, 0.2)
    g, u = (_f32(np.abs(rng.standard_normal((m, n))) + 0.1) for _ in range(2))
    dx, dwg, dwu, _, _ = bl.bitlinear_gated_backward(_t(torch, dy), _t(torch, g), _t(torch, u), tx, tb,
                                                     _t(torch, plain.pack(w0)), _t(torch, al), _t(torch, plain.pack(w1)),
                                                     _t(torch, al1), bl.BITLINEAR_ACT_RELU2)
    want, terms = plain.gated_gradients(dy, g, u, x_q, beta, w0, al[0], w1, al1[0], "relu2")
    for t, w, s, length, name in zip((dx, dwg, dwu), want, terms, (2 * n, m, m), ("dx", "dWg", "dWu")):
        _within(_np(t), w, s, length, name)
    assert not dx[1].any() and not dwg[2].any() and not dwu[2].any()
