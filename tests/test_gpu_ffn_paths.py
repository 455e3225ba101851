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


# ------------------------------------------------------------------ every kernel of the choices by size
def _int_product(torch, x_q, w):
    """x_q . w^T, exact: sums of integers below 2^53 in 64-bit floating point on the device."""
    return _np(_t(torch, x_q).double() @ _t(torch, w).double().t().contiguous())


def _off(torch, a, n):
    """A contiguous view of a's values that starts n elements into its buffer."""
    if a is None:
        return None
    t = _t(torch, a)
    v = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")[n:].view(t.shape)
    v.copy_(t)
    return v


def _gated_case(dev, m, k, f, act, bias, keep, views=False):  # noqa: F811
    """One call against the documented 32-bit steps: x_q, beta, g and u bit for bit, h within the
    activation's roundings; what lies behind the outputs stays."""
    torch, bl = dev
    _say(f"gated_forward M={m} K={k} F={f} {act} bias={bias} keep={keep} views={views}")
    rng = np.random.default_rng([70, m, k, f])
    x = _f32(rng.standard_normal((m, k)))
    wg, ag, bg = _layer(rng, f, k, bias)
    wu, au, bu = _layer(rng, f, k, bias)
    put = (lambda a, n: _off(torch, a, n)) if views else (lambda a, n: _t(torch, a))
    room = [torch.full((m * f + 64,), 7.0, device="cuda") for _ in range(3)]
    s = 1 if views else 0
    h, g, u = (r[s:s + m * f].view(m, f) for r in room)
    bytes_ = torch.empty(m * k + 3, dtype=torch.int8, device="cuda")
    x_q = bytes_[3 * s:3 * s + m * k].view(m, k)
    beta = torch.empty(m, device="cuda")
    bl.bitlinear_gated_forward(put(x, 1), put(plain.pack(wg), 1), put(ag, 1), put(plain.pack(wu), 3), put(au, 3),
                               _code(bl, act), bias_g=put(bg, 1), bias_u=put(bu, 1), h=h, g=g if keep else None,
                               u=u if keep else None, x_q=x_q, beta=beta)
    xq_p, beta_p = plain.absmax(x)
    assert np.array_equal(_np(x_q), xq_p) and np.array_equal(_np(beta), beta_p)

    def project(w, alpha, b):
        y = _int_product(torch, xq_p, w).astype(np.float32) * (np.float64(alpha) * beta_p.astype(np.float64) / 127).astype(np.float32)[:, None]
        return y if b is None else y + b

    g_p, u_p = project(wg, ag[0], bg), project(wu, au[0], bu)
    assert g_p.dtype == np.float32
    if keep:
        assert np.array_equal(_np(g), g_p) and np.array_equal(_np(u), u_p)
    else:
        assert bool((room[1] == 7).all()) and bool((room[2] == 7).all())
    if act == "gelu":
        v = torch.from_numpy(g_p).double()
        a = (0.5 * v * torch.special.erfc(-v * 0.5 ** 0.5)).numpy()
    else:
        a = plain.activation(g_p, act)[0]
    ref = a * u_p.astype(np.float64)
    n = {"silu": 8, "gelu": 2, "relu2": 2}[act]
    assert np.all(np.abs(_np(h) - ref) <= 1.01 * n * U * np.abs(ref) + 2.0 ** -120)
    assert bool((room[0][:s] == 7).all()) and bool((room[0][s + m * f:] == 7).all())


ACTS = ["gelu", "silu", "relu2"]
# more than 64 tiles of 64 x 128, so the GEMM: tiles of 32 tokens (102 of them), of 64 (170, since 340 of 32) and of
# 128 (426, more than 384); the last row and column of tiles partial
GEMM = [(65, 4300), (300, 4300), (700, 9000)]


@pytest.mark.parametrize("m,f", GEMM)
@pytest.mark.parametrize("i,k", list(enumerate([64, 128, 192, 256, 320, 384, 448, 512, 1088])))
def test_gated_gemm(dev, m, f, i, k):  # noqa: F811
    """Rows on 16-byte boundaries: no whole step of 128, one to four, with and without a last half step."""
    _gated_case(dev, m, k, f, ACTS[i % 3], bias=i % 2 == 0, keep=i % 4 < 2)


@pytest.mark.parametrize("m,f", GEMM)
@pytest.mark.parametrize("i,k", list(enumerate([4, 60, 132, 260, 388, 1028])))
def test_gated_gemm_any_rows(dev, m, f, i, k):  # noqa: F811
    """Rows off those boundaries: fewer than 16 bytes, part steps alone and after one to eight whole ones."""
    _gated_case(dev, m, k, f, ACTS[i % 3], bias=i % 2 == 1, keep=i % 4 > 1)


@pytest.mark.parametrize("m,f", GEMM)
@pytest.mark.parametrize("act", ACTS)
def test_gated_gemm_unaligned_views(dev, m, f, act):  # noqa: F811
    _gated_case(dev, m, 256, f, act, bias=True, keep=True, views=True)


# Pairs of rows a wave, pairs at a time: K <= 4096: 2 of 2, 3 of 4, 6 of 6, 7 of 4 (twice), 10 of 4 (three times);
# two chunks of 4096: 3 of 2, three chunks: 3 of 1, four: 2 of 1 and (the last chunk partial) 3 of 1
@pytest.mark.parametrize("k,f", [(320, 3000), (4096, 5000), (1024, 11008), (640, 13000), (64, 20011), (8192, 5000), (9024, 4099),
                                 (16384, 4090), (12352, 4100)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_one_token(dev, k, f, act):  # noqa: F811
    _gated_case(dev, 1, k, f, act, bias=f % 2 == 0, keep=act == "silu")


# Token blocks of a workgroup, column blocks: 1 x 1, 2 x 1, 3 x 1, 4 x 1, 3 x 2, 4 x 2, and 4 x 2 in several slices
@pytest.mark.parametrize("m,f", [(9, 500), (30, 700), (41, 900), (64, 1000), (48, 4500), (64, 4500), (130, 2100)])
@pytest.mark.parametrize("i,k", list(enumerate([64, 256, 2368, 4, 260, 1100])))
def test_gated_few_tokens(dev, m, f, i, k):  # noqa: F811
    """The streaming kernel: a part step alone, one whole step, more steps than waves and a part; aligned or not."""
    _gated_case(dev, m, k, f, ACTS[(i + m) % 3], bias=i % 2 == 0, keep=m % 2 == 0)


def _i8_case(dev, m, k, n):  # noqa: F811
    torch, bl = dev
    _say(f"forward_i8 M={m} K={k} N={n}")
    rng = np.random.default_rng([71, m, k, n])
    xq = rng.integers(-127, 128, (m, k)).astype(np.int8)
    wq = rng.integers(-127, 128, (n, k)).astype(np.int8)
    beta, gamma = _f32(rng.random(m) + 0.5), _f32(rng.random(n) + 0.5)
    b = _f32(rng.standard_normal(n)) if (m + k) % 2 else None
    out = torch.full((m + 2, n), 3.0, device="cuda")
    _, acc = bl.bitlinear_forward_i8(_t(torch, xq), _t(torch, beta), _t(torch, wq), _t(torch, gamma), bias=_t(torch, b),
                                     y=out[1:m + 1], acc=True)
    ref = _int_product(torch, xq, wq).astype(np.int32)
    assert np.array_equal(_np(acc), ref)
    f = np.float32
    y = (ref.astype(f) * (beta / f(127))[:, None]) * (gamma / f(127))[None]
    assert np.array_equal(_np(out[1:m + 1]), y if b is None else y + b)
    assert bool((out[0] == 3).all()) and bool((out[m + 1] == 3).all())


# Token blocks, channel blocks: 3 x 2, 4 x 2, 4 x 2 in two slices
@pytest.mark.parametrize("m,n", [(48, 5000), (33, 4111), (64, 4500), (100, 2100)])
@pytest.mark.parametrize("k", [16, 272, 1552, 260, 1100, 15, 257, 1001])
def test_forward_i8_few_tokens_two_blocks(dev, m, n, k):  # noqa: F811
    """The streaming kernel with two blocks of channels, rows on 16-byte and dword boundaries and off them."""
    _i8_case(dev, m, k, n)


@pytest.mark.parametrize("m,n", [(70, 4200), (520, 4200), (1100, 4200)])
@pytest.mark.parametrize("k", [133136, 133144, 133143])
def test_forward_i8_largest_sums_in_tiles(dev, m, n, k):  # noqa: F811
    """Codes of +-127 at the largest K in every tile size of the GEMM (34, 153 and 306 tiles of 64 x 256)."""
    torch, bl = dev
    _say(f"forward_i8 largest sums M={m} K={k} N={n}")
    x_q = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
    x_q[1::3] = -127
    w_q = torch.full((n, k), -127, dtype=torch.int8, device="cuda")
    w_q[1::2] = 127
    _, acc = bl.bitlinear_forward_i8(x_q, torch.ones(m, device="cuda"), w_q, torch.ones(n, device="cuda"), acc=True)
    want = (torch.where(torch.arange(m) % 3 == 1, -1, 1)[:, None] * torch.where(torch.arange(n) % 2 == 1, 1, -1)) * (127 * 127 * k)
    assert torch.equal(acc.cpu().long(), want)


# 64 tokens x 256 columns a tile of the maxima (561 tiles, at least 512), the last of both directions partial
@pytest.mark.parametrize("gated", [False, True])
def test_backward_large_tiles_of_the_maxima(dev, gated):  # noqa: F811
    torch, bl = dev
    m, k, n = 2100, 68, 4100
    _say(f"backward M={m} K={k} N={n} gated={gated}")
    rng = np.random.default_rng([72, gated])
    dy = _f32(rng.standard_normal((m, n)) * np.exp(rng.standard_normal((m, 1))) / m)
    dy[:, 5] *= 1000
    dy[7] *= 1000
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    tx, tb = _t(torch, x_q), _t(torch, beta)
    w0, al, _ = _layer(rng, n, k, False)
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    if not gated:
        out = bl.bitlinear_backward(_t(torch, dy), tx, tb, _t(torch, plain.pack(w0)), _t(torch, al), dx=nan(m, k), dW=nan(n, k),
                                    dbias=nan(n))
        want, terms = plain.linear_gradients(dy, x_q, beta, w0, al[0])
        lengths = [n, m, m]
    else:
        w1, al1, _ = _layer(rng, n, k, False)
        g, u = (_f32(rng.standard_normal((m, n))) for _ in range(2))
        out = bl.bitlinear_gated_backward(_t(torch, dy), _t(torch, g), _t(torch, u), tx, tb, _t(torch, plain.pack(w0)),
                                          _t(torch, al), _t(torch, plain.pack(w1)), _t(torch, al1), bl.BITLINEAR_ACT_RELU2,
                                          dx=nan(m, k), dWg=nan(n, k), dWu=nan(n, k), dbias_g=nan(n), dbias_u=nan(n))
        want, terms = plain.gated_gradients(dy, g, u, x_q, beta, w0, al[0], w1, al1[0], "relu2")
        lengths = [2 * n, m, m, m, m]
    for i, (t, w, s, length) in enumerate(zip(out, want, terms, lengths)):
        _within(_np(t), w, s, length, i)


def test_forward_i8_three_token_blocks_on_dwords(dev):  # noqa: F811
    _i8_case(dev, 41, 260, 900)


# One pass in fp32 with room for 4, 8 and 16 tokens; one pass on the matrix cores; panels, up to 64 tokens and more
@pytest.mark.parametrize("m,k,f", [(3, 68, 70), (8, 260, 300), (16, 260, 300), (40, 260, 300), (33, 4100, 4200), (300, 1028, 1100)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_every_activation(dev, m, k, f, act):  # noqa: F811
    torch, bl = dev
    _say(f"gated_backward M={m} K={k} F={f} {act}")
    rng = np.random.default_rng([73, m, k, f])
    dh = _f32(rng.standard_normal((m, f)) / m)
    g, u = (_f32(rng.standard_normal((m, f)) * 2) for _ in range(2))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    wg, ag, _ = _layer(rng, f, k, False)
    wu, au, _ = _layer(rng, f, k, False)
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    out = bl.bitlinear_gated_backward(_t(torch, dh), _t(torch, g), _t(torch, u), _t(torch, x_q), _t(torch, beta),
                                      _t(torch, plain.pack(wg)), _t(torch, ag), _t(torch, plain.pack(wu)), _t(torch, au),
                                      _code(bl, act), dx=nan(m, k), dWg=nan(f, k), dWu=nan(f, k), dbias_g=nan(f),
                                      dbias_u=nan(f))
    want, terms = plain.gated_gradients(dh, g, u, x_q, beta, wg, ag[0], wu, au[0], act)
    # a'(g) of SiLU and GELU passes through zero, where its error is that of its parts, at most 2 in size:
    # counted as roundings of dh u
    d0 = 24 * U * np.abs(dh.astype(np.float64) * u) * (act != "relu2")
    xd = np.abs(x_q.astype(np.float64)) * beta[:, None] / 127
    slack = [d0 @ np.abs(wg).astype(np.float64) * ag[0], d0.T @ xd, 0, d0.sum(0), 0]
    for t, w, s, n, sl, name in zip(out, want, terms, [2 * f, m, m, m, m], slack, ("dx", "dWg", "dWu", "dbias_g", "dbias_u")):
        _within(_np(t), w, s, n, name, sl)


@pytest.mark.parametrize("m,k,n", RANGES)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_backward_keeps_what_is_not_finite_in_its_row_and_column(dev, m, k, n, bad):  # noqa: F811
    """One gradient that is not a number or infinite: its token's dx and its channel's dW and dbias are
    not finite, everything else is what it is without it."""
    torch, bl = dev
    _say(f"backward with {bad} M={m} K={k} N={n}")
    rng = np.random.default_rng([74, m, k, n])
    dy = _f32(rng.standard_normal((m, n)))
    i, j = m // 3, n // 2
    dy[i, j] = 0
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    w, al, _ = _layer(rng, n, k, False)
    rest = (_t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    e = lambda *s: torch.empty(s, device="cuda")
    want = bl.bitlinear_backward(_t(torch, dy), *rest, dx=e(m, k), dW=e(n, k), dbias=e(n))
    dy[i, j] = bad
    got = bl.bitlinear_backward(_t(torch, dy), *rest, dx=e(m, k), dW=e(n, k), dbias=e(n))
    for t, c, row in zip(got, want, (i, j, j)):
        assert not torch.isfinite(t[row]).any()
        others = torch.arange(t.shape[0], device="cuda") != row
        assert torch.equal(t[others], c[others])


@pytest.mark.parametrize("m,k,n", [(40, 132, 90), (700, 132, 4100)])
def test_backward_over_a_hundred_binades_in_a_graph(dev, m, k, n):  # noqa: F811
    """Captured once; replays with other inputs, ordinary ones among them, and eager work between give the eager bits."""
    torch, bl = dev
    _say(f"backward hundred binades in a graph M={m} K={k} N={n}")
    rng = np.random.default_rng([75, m, k, n])
    x_q, beta = plain.absmax(rng.standard_normal((m, k)) * (rng.random((m, k)) < 0.2))
    w, al, _ = _layer(rng, n, k, False)
    w = (w * (rng.random((n, k)) < 0.2)).astype(np.int8)
    e = lambda *s: torch.empty(s, device="cuda")
    dy = _t(torch, _f32(rng.standard_normal((m, n))))
    ws = torch.empty(bl.bitlinear_backward_workspace_size(m, k, n), dtype=torch.uint8, device="cuda")
    args = (dy, _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    out = dict(dx=e(m, k), dW=e(n, k), dbias=e(n), workspace=ws)
    bl.bitlinear_backward(*args, **out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.bitlinear_backward(*args, **out)
    for rep, spread in enumerate((100, 0, 60, 100)):
        dy.copy_(_t(torch, _f32(rng.standard_normal((m, n)) * np.exp2(rng.integers(-spread, 1, (m, n))))))
        bl.bitlinear_backward(*args, **out)
        eager = [out[q].clone() for q in ("dx", "dW", "dbias")]
        for q in ("dx", "dW", "dbias"):
            out[q].fill_(float("nan"))
        ws.fill_(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, out[q]) for a, q in zip(eager, ("dx", "dW", "dbias")))
