"""GPU tests of the e4m3 quantizers and the fp8 product against plain 64-bit forms: codes and scales bit for
bit, exact small integers exactly, other products within bounds counted in roundings."""
import numpy as np
import pytest

import ffn_plain as plain
from ffn_plain import U

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bitlinear_matmul_absmean_amd as bl
    return torch, bl


def _t(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _off(torch, t, n):
    """t as a contiguous view that starts n elements into its buffer."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
    v = buf[n:].view(t.shape)
    v.copy_(t)
    return v


# every e4m3 value by its code; 0x7f and 0xff are NaN
def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


TABLE = _e4m3_table()


def _values(t):
    import torch
    return TABLE[t.view(torch.uint8).cpu().numpy()]


def _round(q):
    """64-bit values of magnitude up to 448 rounded to e4m3, ties to even."""
    m = np.abs(q)
    exponent = np.maximum(np.frexp(np.maximum(m, 2.0 ** -60))[1] - 1, -6)
    step = np.ldexp(1.0, exponent - 3)
    return np.copysign(np.rint(m / step) * step, q)


def _quantize(x, high):
    """Codes' values and scales [R / high, K / 128] in the documented 32-bit steps."""
    r, k = x.shape
    nr, nk = -(-r // high), -(-k // 128)
    p = np.zeros((nr * high, nk * 128), F32)
    p[:r, :k] = x
    p = p.reshape(nr, high, nk, 128)
    s = (np.abs(p).max(axis=(1, 3)) / F32(448)).astype(F32)
    d = np.where(s > 0, s, F32(1))[:, None, :, None]
    with np.errstate(over="ignore"):
        q = np.where(s[:, None, :, None] > 0, np.clip((p / d).astype(F32), F32(-448), F32(448)), F32(0))
    return _round(q.astype(np.float64)).reshape(nr * high, nk * 128)[:r, :k], s


def _data(rng, r, k):
    x = rng.standard_normal((r, k)).astype(F32)
    x[rng.random((r, k)) < 0.01] *= 50
    return x


SIZES = [(1, 1), (1, 127), (1, 128), (1, 129), (1, 4096), (2, 3), (3, 260), (5, 1001), (8, 512), (9, 640), (64, 127), (127, 36),
         (128, 128), (129, 257), (130, 1000), (300, 384)]


@pytest.mark.parametrize("r,k", SIZES)
def test_quantizers(dev, r, k):
    torch, bl = dev
    rng = np.random.default_rng([1, r, k])
    x = _data(rng, r, k)
    x[r // 2] = 0                                                   # a token of zeros
    x[:, : min(k, 128)] *= F32(2.0 ** -40) if r % 2 else F32(1)
    for off in (0, 1):
        v = _off(torch, _t(torch, x), off)
        x_q = _off(torch, torch.empty(r, k, dtype=torch.uint8, device="cuda"), off).view(torch.float8_e4m3fn)
        bl.bitlinear_quantize_act_fp8(v, x_q=x_q)
        x_q2, xs = bl.bitlinear_quantize_act_fp8(v)
        w_q, ws = bl.bitlinear_quantize_weights_fp8(v)
        torch.cuda.synchronize()
        want, s = _quantize(x, 1)
        assert np.array_equal(_values(x_q), want) and np.array_equal(_values(x_q2), want)
        assert xs.shape == s.T.shape and np.array_equal(xs.cpu().numpy(), s.T)
        want, s = _quantize(x, 128)
        assert np.array_equal(_values(w_q), want) and np.array_equal(ws.cpu().numpy(), s)


@pytest.mark.parametrize("r,k", [(2500, 1281), (3100, 1028), (1, 3200001), (6, 640128), (24600, 128)])
def test_quantizers_of_many_blocks(dev, r, k):
    test_quantizers(dev, r, k)


def test_quantizer_extremes(dev):
    """Ties, subnormal codes, subnormal scales, the largest floats, blocks of zeros."""
    torch, bl = dev
    rng = np.random.default_rng(3)
    x = np.zeros((7, 512), F32)
    x[0, :256] = TABLE[np.isfinite(TABLE)].repeat(2)[:256]
    # midpoints between neighbouring codes, with 448 in the block so that the scale is 1
    v = np.sort(TABLE[np.isfinite(TABLE) & (TABLE >= 0)])
    x[1, :126] = (v[1:] + v[:-1])[:126] / 2
    x[1, 127] = 448
    x[1, 128:254] = -x[1, :126]
    x[1, 255] = 448
    x[2] = rng.standard_normal(512) * 1e-38
    x[3] = rng.standard_normal(512) * 1e-43                         # scales that are subnormal, or zero
    x[4] = rng.standard_normal(512) * 1e37
    x[5, 3] = np.finfo(F32).max
    for high, call in ((1, bl.bitlinear_quantize_act_fp8), (128, bl.bitlinear_quantize_weights_fp8)):
        q, s = call(_t(torch, x))
        want, ws = _quantize(x, high)
        assert np.array_equal(s.cpu().numpy(), ws.T if high == 1 else ws)
        assert np.array_equal(_values(q), want)


@pytest.mark.parametrize("k", [128, 300, 1001])
def test_what_is_not_finite_stays_so(dev, k):
    """NaN and infinities have the code NaN, whatever else is in their block, and make the products of their
    token, or of their channel, not finite; other blocks are as without them."""
    torch, bl = dev
    rng = np.random.default_rng([23, k])
    m, n = 9, 140
    x, w = _data(rng, m, k), _data(rng, n, k)
    bad = x.copy()
    bad[1, 5], bad[2, k - 1], bad[4, 0] = np.nan, np.inf, -np.inf
    bad[6, :128] = 0
    bad[6, 100] = np.nan                                            # alone in a block of zeros
    bad[7, :] = np.nan
    gone = ~np.isfinite(bad)
    q, s = bl.bitlinear_quantize_act_fp8(_t(torch, bad))
    assert np.isnan(_values(q)[gone]).all() and not np.isnan(_values(q)[~gone]).any()
    want, scale = _quantize(x, 1)
    rows = ~gone.any(axis=1)
    assert np.array_equal(_values(q)[rows], want[rows]) and np.array_equal(s.cpu().numpy().T[rows], scale[rows])
    w_q, ws = bl.bitlinear_quantize_weights_fp8(_t(torch, w))
    for tokens in (m, 200):                                         # the streaming kernel and the tiles
        qs, ss = q.view(torch.uint8).repeat(tokens // m + 1, 1)[:tokens].view(q.dtype), s.repeat(1, tokens // m + 1)[:, :tokens].contiguous()
        y = bl.bitlinear_forward_fp8(qs.contiguous(), ss, w_q, ws).cpu().numpy()
        there = np.resize(rows, (tokens // m + 1) * m)[:tokens]
        assert np.isfinite(y[there]).all() and not np.isfinite(y[~there]).any()
    wide = w.copy()
    wide[3, k // 2] = np.nan
    q2, _ = bl.bitlinear_quantize_weights_fp8(_t(torch, wide))
    assert np.isnan(_values(q2)[3, k // 2]) and np.isnan(_values(q2)).sum() == 1
    wide[3, k // 2] = -np.inf
    q2, s2 = bl.bitlinear_quantize_weights_fp8(_t(torch, wide))
    assert np.isnan(_values(q2)[3, k // 2]) and np.isnan(_values(q2)).sum() == 1
    assert np.isinf(s2.cpu().numpy()).sum() == 1


# ------------------------------------------------------------------------------------ the product
PRODUCT = [(1, 1, 1), (1, 16, 5), (1, 128, 16), (1, 4096, 300), (1, 11008, 64), (1, 1001, 129), (1, 500, 33), (2, 256, 31),
           (7, 1024, 100), (15, 384, 128), (16, 2048, 256), (16, 130, 130), (17, 512, 48), (33, 1000, 65), (48, 1024, 512),
           (64, 640, 33), (64, 4096, 2048), (65, 384, 1024), (100, 1001, 257), (127, 4096, 640), (128, 256, 4096), (200, 500, 1000),
           (256, 1024, 2048), (300, 2176, 4096), (513, 896, 4352), (640, 144, 8200), (1025, 336, 2050)]


def _bound(xv, xs, wv, ws, terms_of=None):
    """y in 64 bits, and the bound on the error of its sum.  A term x_scale W_scale x_q W_q carries the
    rounding of the scales' product (1); a block's sum of 128 exact products, times that, is added in fp32:
    counted as gradient_tolerance does for a sum of K + K / 128 terms."""
    k = xv.shape[1]
    b = np.arange(k) // 128
    x = xv * xs.astype(np.float64)[:, b]
    w = wv * ws.astype(np.float64)[np.arange(wv.shape[0]) // 128][:, b]
    y = x @ w.T
    terms = np.sqrt((x ** 2) @ (w ** 2).T)
    return y, plain.gradient_tolerance(terms, k + k / 128, np.abs(y))


@pytest.mark.parametrize("m,k,n", PRODUCT)
def test_product(dev, m, k, n):
    torch, bl = dev
    print(f"forward_fp8 M={m} K={k} N={n}", flush=True)
    rng = np.random.default_rng([2, m, k, n])
    x, w = _data(rng, m, k), (_data(rng, n, k) * F32(0.02))
    bias = (rng.standard_normal(n) * 0.1).astype(F32) if (m + n) % 2 else None
    (xv, xs), (wv, ws) = _quantize(x, 1), _quantize(w, 128)
    x_q, x_scale = bl.bitlinear_quantize_act_fp8(_t(torch, x))
    w_q, w_scale = bl.bitlinear_quantize_weights_fp8(_t(torch, w))
    y = bl.bitlinear_forward_fp8(x_q, x_scale, w_q, w_scale, bias=_t(torch, bias)).cpu().numpy().astype(np.float64)
    want, tol = _bound(xv, xs, wv, ws)
    if bias is not None:
        want = want + bias
        tol = tol + U * np.abs(want)
    assert np.all(np.abs(y - want) <= tol * 1.001 + 2.0 ** -140)
    # the same again, and on views that start off any alignment, within the bound
    again = bl.bitlinear_forward_fp8(x_q, x_scale, w_q, w_scale, bias=_t(torch, bias)).cpu().numpy()
    assert np.array_equal(again, y.astype(F32))
    out = torch.full((m * n + 8,), 7.0, device="cuda")
    o8 = lambda t, i: _off(torch, t.view(torch.uint8), i).view(torch.float8_e4m3fn)
    bl.bitlinear_forward_fp8(o8(x_q, 3), _off(torch, x_scale, 1), o8(w_q, 1), _off(torch, w_scale, 3),
                             bias=None if bias is None else _off(torch, _t(torch, bias), 1), y=out[3:3 + m * n].view(m, n))
    out = out.cpu().numpy()
    assert np.all(out[:3] == 7) and np.all(out[3 + m * n:] == 7)
    assert np.all(np.abs(out[3:3 + m * n].reshape(m, n) - want) <= tol * 1.001 + 2.0 ** -140)


@pytest.mark.parametrize("m,k,n", PRODUCT)
def test_exact_sums(dev, m, k, n):
    """Small integers and scales that are powers of two: every partial sum is a float, and y is exact."""
    torch, bl = dev
    rng = np.random.default_rng([4, m, k, n])
    nb = -(-k // 128)
    xv, wv = rng.integers(-4, 5, (m, k)).astype(F32), rng.integers(-4, 5, (n, k)).astype(F32)
    xs = np.exp2(rng.integers(-2, 3, (nb, m))).astype(F32)
    ws = np.exp2(rng.integers(-2, 3, (-(-n // 128), nb))).astype(F32)
    x_q, w_q = _t(torch, xv).to(torch.float8_e4m3fn), _t(torch, wv).to(torch.float8_e4m3fn)
    y = bl.bitlinear_forward_fp8(x_q, _t(torch, xs), w_q, _t(torch, ws)).cpu().numpy()
    b = np.arange(k) // 128
    want = (xv * xs.T[:, b]).astype(np.float64) @ (wv * ws[np.arange(n) // 128][:, b]).astype(np.float64).T
    # up to 11008 terms of 16 * 16, in steps of 2^-4: below 2^24 steps up to K = 2^16 / 4
    assert np.array_equal(y, want.astype(F32))


def test_product_of_wide_ranges(dev):
    """Small products beside large ones in a block: each is counted to within the bound on the block's sum,
    and where the large ones cancel exactly, the small ones are the sum."""
    torch, bl = dev
    m, k, n = 32, 256, 64
    x, w = np.zeros((m, k), F32), np.zeros((n, k), F32)
    x[:, 0], x[:, 1] = 448, -448
    w[:, 0] = w[:, 1] = 448
    x[:, 2:128], w[:, 2:128] = 2.0 ** -6, 2.0 ** -2
    one = np.ones((2, m), F32)
    y = bl.bitlinear_forward_fp8(_t(torch, x).to(torch.float8_e4m3fn), _t(torch, one), _t(torch, w).to(torch.float8_e4m3fn),
                                 _t(torch, np.ones((1, 2), F32))).cpu().numpy()
    # 126 products of 2^-8 beside two of 448^2: sums round by a unit of 448^2 at most at each of 128 steps
    assert np.all(np.abs(y - 126 * 2.0 ** -8) <= 128 * 2 * U * 448.0 ** 2)


def test_a_scale_of_zero_and_rows_of_zeros(dev):
    torch, bl = dev
    rng = np.random.default_rng(8)
    x, w = _data(rng, 70, 300), _data(rng, 200, 300)
    x[5], w[128:] = 0, 0
    x_q, xs = bl.bitlinear_quantize_act_fp8(_t(torch, x))
    w_q, ws = bl.bitlinear_quantize_weights_fp8(_t(torch, w))
    y = bl.bitlinear_forward_fp8(x_q, xs, w_q, ws).cpu().numpy()
    assert np.all(y[5] == 0) and np.all(y[:, 128:] == 0) and np.all(np.isfinite(y))


@pytest.mark.parametrize("m,k,n", [(1, 1024, 200), (40, 512, 300), (300, 640, 2048)])
def test_graphs_and_streams(dev, m, k, n):
    """A captured pass replayed with other inputs, between eager work; the same on a stream of its own."""
    torch, bl = dev
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    x = torch.randn(m, k, device="cuda", generator=gen)
    w_q, ws = bl.bitlinear_quantize_weights_fp8(torch.randn(n, k, device="cuda", generator=gen))
    x_q, xs = bl.bitlinear_quantize_act_fp8(x)
    y = torch.empty(m, n, device="cuda")

    def step():
        bl.bitlinear_quantize_act_fp8(x, x_q=x_q, x_scale=xs)
        bl.bitlinear_forward_fp8(x_q, xs, w_q, ws, y=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        x.copy_(torch.randn(m, k, device="cuda", generator=gen))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        a, b = bl.bitlinear_quantize_act_fp8(x)
        assert torch.equal(got, bl.bitlinear_forward_fp8(a, b, w_q, ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = bl.bitlinear_quantize_act_fp8(x, stream=side)
    z = bl.bitlinear_forward_fp8(a, b, w_q, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, got)


def test_past_32_bit_offsets(dev):
    """Codes of W past 2^32 bytes and outputs past 2^32 bytes."""
    torch, bl = dev
    k, n = 8192, 600000
    w_q = torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    w_q[-3:, :5] = 0x38                                             # 1.0
    ws = torch.full((-(-n // 128), k // 128), 2.0, device="cuda")
    for m in (1, 20, 2048):
        print(f"forward_fp8 M={m} K={k} N={n}", flush=True)
        x_q = torch.full((m, k), 0x40, dtype=torch.uint8, device="cuda")           # 2.0
        y = bl.bitlinear_forward_fp8(x_q.view(torch.float8_e4m3fn), torch.ones(k // 128, m, device="cuda"),
                                     w_q.view(torch.float8_e4m3fn), ws)
        torch.cuda.synchronize()
        assert bool((y[:, -3:] == 20).all()) and bool((y[:, :-3] == 0).all())
        del y
