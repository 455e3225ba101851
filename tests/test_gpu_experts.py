"""GPU tests of the products grouped by expert and of their gradients against plain 64-bit forms: integer
sums and documented 32-bit steps bit for bit, activations and gradients within bounds counted in roundings."""
import numpy as np
import pytest

import experts_plain
import ffn_plain as plain
from ffn_plain import U

pytestmark = pytest.mark.gpu
F32 = np.float32
ACTS = ["gelu", "silu", "relu2"]


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bitlinear_matmul_absmean_amd as bl
    return torch, bl


def _say(*a):
    print(*a, flush=True)


def _code(bl, act):
    return {"gelu": bl.BITLINEAR_ACT_GELU, "silu": bl.BITLINEAR_ACT_SILU, "relu2": bl.BITLINEAR_ACT_RELU2}[act]


def _t(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.cpu().numpy()


def _bits(a):
    return np.ascontiguousarray(a).view(np.uint32)


def _off(torch, a, n):
    """a on the GPU as a contiguous view that starts n elements into its buffer."""
    t = _t(torch, a)
    if t is None:
        return None
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
    v = buf[n:].view(t.shape)
    v.copy_(t)
    return v


def _weights(rng, e, n, k, bias):
    w = rng.integers(-1, 2, size=(e, n, k)).astype(np.int8)
    alpha = rng.uniform(0.01, 0.02, e).astype(F32)
    return w, alpha, (rng.standard_normal((e, n)) * 0.1).astype(F32) if bias else None


def _pack(w):
    return np.stack([plain.pack(x) for x in w])


def _layout(rng, counts, gather, before=0, behind=0):
    """offsets of `counts` rows an expert after `before` rows of none, and the rows' tokens."""
    offsets = before + np.concatenate([[0], np.cumsum(counts)])
    m = int(offsets[-1]) + behind
    if not gather:
        return offsets.astype(np.int64), None, m, m
    t = max(1, m // 2)
    return offsets.astype(np.int64), rng.integers(0, t, m).astype(np.int64), m, t


# counts of rows for each expert, K, N, rows gathered from tokens, rows before and behind the groups
CASES = [
    ([1], 4, 1, False, 0, 0), ([0, 1], 64, 16, True, 0, 0), ([1, 1], 4096, 100, True, 0, 0), ([3, 0, 2], 256, 33, False, 1, 2),
    ([1] * 8, 320, 130, True, 0, 3), ([5, 0, 0, 11, 1, 16, 17], 512, 48, True, 0, 0), ([2] * 65, 128, 40, True, 2, 0),
    ([0] * 130 + [3] + [0] * 69 + [4], 192, 17, False, 0, 1), ([33, 1, 0, 40], 100, 70, True, 0, 0), ([16, 15], 1088, 77, False, 0, 0),
    ([64, 0, 31], 2048, 96, True, 0, 0), ([70, 200, 3], 256, 300, False, 0, 5), ([129, 0, 1, 64], 1028, 257, True, 0, 0),
    ([300, 20], 512, 513, True, 7, 9), ([1, 500], 640, 260, False, 0, 0), ([40] * 16, 192, 384, True, 0, 0),
    ([128, 128], 64, 1024, False, 0, 0), ([257, 130, 0, 511], 576, 640, True, 0, 0),
]


def _name(c):
    counts = c[0] if len(c[0]) <= 8 else [len(c[0]), sum(c[0])]
    return f"{'-'.join(map(str, counts))}_K{c[1]}_N{c[2]}"


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_forward(dev, case):
    torch, bl = dev
    counts, k, n, gather, before, behind = case
    rng = np.random.default_rng([1, len(counts), sum(counts), k, n])
    offsets, rows, m, t = _layout(rng, counts, gather, before, behind)
    bias = n % 2 == 1
    _say(f"grouped_forward counts={counts[:10]} M={m} T={t} K={k} N={n} bias={bias}")
    w, alpha, b = _weights(rng, len(counts), n, k, bias)
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    y = torch.full((m, n), 7.0, device="cuda")
    args = (_t(torch, x_q), _t(torch, beta), _t(torch, offsets), _t(torch, _pack(w)), _t(torch, alpha))
    kw = dict(rows=_t(torch, rows), bias=_t(torch, b))
    out = bl.bitlinear_grouped_forward(*args, y=y, **kw)
    assert out is y
    want = experts_plain.forward(*experts_plain.tokens(x_q, beta, rows, m), offsets, w, alpha, b, np.full((m, n), 7, F32))
    assert np.array_equal(_np(y), want)
    # views that start off any vector alignment
    buf = torch.full((m * n + 8,), 7.0, device="cuda")
    bl.bitlinear_grouped_forward(_off(torch, x_q, 3), _off(torch, beta, 1), _off(torch, offsets, 1), _off(torch, _pack(w), 1),
                                 _off(torch, alpha, 3), rows=_off(torch, rows, 1), bias=_off(torch, b, 1),
                                 y=buf[3:3 + m * n].view(m, n))
    buf = _np(buf)
    assert np.array_equal(buf[3:3 + m * n].reshape(m, n), want) and np.all(buf[:3] == 7) and np.all(buf[3 + m * n:] == 7)


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_gated_forward(dev, case):
    torch, bl = dev
    counts, k, f, gather, before, behind = case
    act = ACTS[(len(counts) + k // 4 + f) % 3]
    rng = np.random.default_rng([2, len(counts), sum(counts), k, f])
    offsets, rows, m, t = _layout(rng, counts, gather, before, behind)
    bias = f % 2 == 0
    _say(f"grouped_gated_forward counts={counts[:10]} M={m} T={t} K={k} F={f} {act} bias={bias}")
    wg, ag, bg = _weights(rng, len(counts), f, k, bias)
    wu, au, bu = _weights(rng, len(counts), f, k, bias)
    x = rng.standard_normal((t, k)).astype(F32)
    g, u, h = (torch.full((m, f), 7.0, device="cuda") for _ in range(3))
    x_q, beta = torch.empty((t, k), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    args = (_t(torch, x), _t(torch, offsets), _t(torch, _pack(wg)), _t(torch, ag), _t(torch, _pack(wu)), _t(torch, au),
            _code(bl, act))
    kw = dict(rows=_t(torch, rows), bias_g=_t(torch, bg), bias_u=_t(torch, bu))
    bl.bitlinear_grouped_gated_forward(*args, h=h, g=g, u=u, x_q=x_q, beta=beta, **kw)
    h2 = bl.bitlinear_grouped_gated_forward(*args, **kw)
    torch.cuda.synchronize()
    xq_p, beta_p = plain.absmax(x)
    assert np.array_equal(_np(x_q), xq_p) and np.array_equal(_bits(_np(beta)), _bits(beta_p))
    xr, br = experts_plain.tokens(xq_p, beta_p, rows, m)
    seven = np.full((m, f), 7, F32)
    g_p = experts_plain.forward(xr, br, offsets, wg, ag, bg, seven)
    u_p = experts_plain.forward(xr, br, offsets, wu, au, bu, seven)
    assert np.array_equal(_np(g), g_p) and np.array_equal(_np(u), u_p)
    # roundings of a(g): SiLU 7, GELU and squared ReLU 1, and the product's, to first order
    lo, hi = before, m - behind
    ref = plain.activation(g_p, act)[0] * u_p.astype(np.float64)
    n = {"silu": 8, "gelu": 2, "relu2": 2}[act]
    h, h2 = _np(h), _np(h2)
    assert np.all(np.abs(h - ref)[lo:hi] <= 1.01 * n * U * np.abs(ref)[lo:hi] + 1e-37)
    assert np.all(h[:lo] == 7) and np.all(h[hi:] == 7)
    assert np.array_equal(_bits(h2[lo:hi]), _bits(h[lo:hi]))
    # views that start off any vector alignment
    buf = torch.full((m * f + 8,), 7.0, device="cuda")
    bl.bitlinear_grouped_gated_forward(_off(torch, x, 1), _off(torch, offsets, 1), _off(torch, _pack(wg), 1), _off(torch, ag, 1),
                                       _off(torch, _pack(wu), 3), _off(torch, au, 3), _code(bl, act), rows=_off(torch, rows, 1),
                                       bias_g=_off(torch, bg, 1), bias_u=_off(torch, bu, 1), h=buf[1:1 + m * f].view(m, f),
                                       x_q=torch.empty(t * k + 3, dtype=torch.int8, device="cuda")[3:].view(t, k))
    assert np.array_equal(_bits(_np(buf)[1:1 + m * f].reshape(m, f)), _bits(h)) and float(buf[0]) == 7 and np.all(_np(buf)[1 + m * f:] == 7)


# experts' rows of the one token, K, F, rows of none before and behind, rows whose token is not there
ONE = [([1], 64, 1, 0, 0, []), ([0, 1, 0, 1], 4096, 2500, 0, 0, []), ([1, 0, 0, 1, 1, 0, 0, 0], 1024, 100, 1, 1, [2]),
       ([0, 2, 0, 1], 4160, 333, 0, 1, [0]), ([0] * 70 + [1] + [0] * 29 + [2], 2048, 5000, 1, 0, [3]), ([1, 0, 1], 8256, 40, 0, 0, [0, 1]),
       ([0, 0, 1], 16384, 77, 0, 2, []), ([1] * 64, 640, 256, 0, 0, [5, 63]), ([0, 3, 0], 192, 3000, 0, 0, [])]


@pytest.mark.parametrize("case", ONE, ids=_name)
@pytest.mark.parametrize("act", ACTS)
def test_one_token(dev, case, act):
    """The gated block of one token, quantized in the launch that multiplies it."""
    torch, bl = dev
    counts, k, f, before, behind, gone = case
    rng = np.random.default_rng([29, len(counts), k, f])
    offsets = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int64)
    e, m = len(counts), int(offsets[-1]) + behind
    rows = np.zeros(m, np.int64)
    rows[gone] = [1, -1, 1 << 33][: len(gone)]
    wg, ag, bg = _weights(rng, e, f, k, act != "gelu")
    wu, au, bu = _weights(rng, e, f, k, True)
    x = rng.standard_normal((1, k)).astype(F32)
    x[0, k // 2] = 20
    h, g, u = (torch.full((m, f), 7.0, device="cuda") for _ in range(3))
    x_q, beta = torch.empty((1, k), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    args = [_t(torch, a) for a in (x, offsets, _pack(wg), ag, _pack(wu), au)] + [_code(bl, act)]
    kw = dict(rows=_t(torch, rows) if gone or m > 1 else None, bias_g=_t(torch, bg), bias_u=_t(torch, bu))
    bl.bitlinear_grouped_gated_forward(*args, h=h, g=g, u=u, x_q=x_q, beta=beta, **kw)
    h2 = torch.full((m, f), 7.0, device="cuda")
    bl.bitlinear_grouped_gated_forward(*args, h=h2, **kw)
    xq_p, beta_p = plain.absmax(x)
    assert np.array_equal(_np(x_q), xq_p) and np.array_equal(_bits(_np(beta)), _bits(beta_p))
    xr, br = experts_plain.tokens(xq_p, beta_p, rows, m)
    seven = np.full((m, f), 7, F32)
    g_p = experts_plain.forward(xr, br, offsets, wg, ag, bg, seven)
    u_p = experts_plain.forward(xr, br, offsets, wu, au, bu, seven)
    assert np.array_equal(_np(g), g_p) and np.array_equal(_np(u), u_p)
    lo, hi = before, m - behind
    ref = plain.activation(g_p, act)[0] * u_p.astype(np.float64)
    h, n = _np(h), {"silu": 8, "gelu": 2, "relu2": 2}[act]                  # as in test_gated_forward
    assert np.all(np.abs(h - ref)[lo:hi] <= 1.01 * n * U * np.abs(ref)[lo:hi] + 1e-37)
    assert np.all(h[:lo] == 7) and np.all(h[hi:] == 7) and np.array_equal(_bits(_np(h2)), _bits(h))


def _check_gradients(got, values, terms, lengths, note):
    for i, (a, v, t, l) in enumerate(zip(got, values, terms, lengths)):
        if a is None:
            continue
        a = _np(a).astype(np.float64)
        tol = plain.gradient_tolerance(t, l, v) + 2.0 ** -126
        over = np.abs(a - v) - tol
        assert np.all(over <= 0), (note, i, float(np.max(np.abs(a - v) / tol)))


def _gradient_inputs(rng, m, n):
    size = np.exp(0.7 * rng.standard_normal((m, 1))) / max(m, 1)
    return (rng.standard_normal((m, n)) * size).astype(F32)


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_backward(dev, case):
    torch, bl = dev
    counts, k, n, gather, before, behind = case
    rng = np.random.default_rng([3, len(counts), sum(counts), k, n])
    offsets, rows, m, t = _layout(rng, counts, gather, before, behind)
    e = len(counts)
    _say(f"grouped_backward counts={counts[:10]} M={m} T={t} K={k} N={n}")
    w, alpha, _ = _weights(rng, e, n, k, False)
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    dy = _gradient_inputs(rng, m, n)
    values, terms, lengths = experts_plain.gradients([dy.astype(np.float64)], [w], [alpha],
                                                     *experts_plain.tokens(x_q, beta, rows, m), offsets, np.full((m, k), 7.0))
    args = [dy, x_q, beta, offsets, _pack(w), alpha]

    def outputs(off):
        flat = [torch.full((s + off + 4,), 7.0, device="cuda") for s in (m * k, e * n * k, e * n)]
        return flat, [f[off:off + s].view(shape) for f, s, shape in
                      zip(flat, (m * k, e * n * k, e * n), ((m, k), (e, n, k), (e, n)))]

    whole, out = outputs(0)
    bl.bitlinear_grouped_backward(*[_t(torch, a) for a in args], rows=_t(torch, rows), dx=out[0], dW=out[1], dbias=out[2])
    _check_gradients(out, values, terms, lengths, "all")
    lo, hi = before, m - behind
    assert np.all(_np(out[0])[:lo] == 7) and np.all(_np(out[0])[hi:] == 7)
    # each output alone has the same bits
    for i, name in enumerate(("dx", "dW", "dbias")):
        alone = torch.full(out[i].shape, 7.0, device="cuda")
        bl.bitlinear_grouped_backward(*[_t(torch, a) for a in args], rows=_t(torch, rows), **{name: alone})
        assert np.array_equal(_bits(_np(alone)), _bits(_np(out[i]))), name
    # views that start off any vector alignment
    flat, off = outputs(3)
    bl.bitlinear_grouped_backward(*[_off(torch, a, 1 if a.dtype != np.int8 else 3) for a in args], rows=_off(torch, rows, 1),
                                  dx=off[0], dW=off[1], dbias=off[2])
    _check_gradients(off, values, terms, lengths, "views")
    for f in flat:
        assert bool((f[:3] == 7).all()) and bool((f[-1:] == 7).all())


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_gated_backward(dev, case):
    torch, bl = dev
    counts, k, f, gather, before, behind = case
    act = ACTS[(len(counts) + k // 4 + f) % 3]
    rng = np.random.default_rng([4, len(counts), sum(counts), k, f])
    offsets, rows, m, t = _layout(rng, counts, gather, before, behind)
    e = len(counts)
    _say(f"grouped_gated_backward counts={counts[:10]} M={m} T={t} K={k} F={f} {act}")
    wg, ag, _ = _weights(rng, e, f, k, False)
    wu, au, _ = _weights(rng, e, f, k, False)
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    g, u = (rng.standard_normal((m, f)).astype(F32) * F32(1.5) for _ in range(2))
    dh = _gradient_inputs(rng, m, f)
    a, slope = plain.activation(g, act)
    d = [dh.astype(np.float64) * u * slope, dh.astype(np.float64) * a]
    values, terms, lengths = experts_plain.gradients(d, [wg, wu], [ag, au], *experts_plain.tokens(x_q, beta, rows, m), offsets,
                                                     np.full((m, k), 7.0), experts_plain.gate_sizes(dh, g, u, act))
    dx = torch.full((m, k), 7.0, device="cuda")
    dws = [torch.full((e, f, k), 7.0, device="cuda") for _ in range(2)]
    dbs = [torch.full((e, f), 7.0, device="cuda") for _ in range(2)]
    args = [_t(torch, v) for v in (dh, g, u, x_q, beta, offsets, _pack(wg), ag, _pack(wu), au)]
    bl.bitlinear_grouped_gated_backward(*args, _code(bl, act), rows=_t(torch, rows), dx=dx, dWg=dws[0], dWu=dws[1],
                                        dbias_g=dbs[0], dbias_u=dbs[1])
    _check_gradients([dx] + dws + dbs, values, terms, lengths, act)
    # one bias gradient alone, and dx alone
    alone = torch.full((e, f), 7.0, device="cuda")
    bl.bitlinear_grouped_gated_backward(*args, _code(bl, act), rows=_t(torch, rows), dbias_u=alone)
    assert torch.equal(alone, dbs[1])
    dx2, a2, b2, _, _ = bl.bitlinear_grouped_gated_backward(*args, _code(bl, act), rows=_t(torch, rows))
    lo, hi = before, m - behind
    assert torch.equal(dx2[lo:hi], dx[lo:hi]) and torch.equal(a2, dws[0]) and torch.equal(b2, dws[1])


# tiles of 128 rows with sums shorter than a step, of one step, cut into parts; short groups beside a long one, sums
# in parts, sums shorter than a step
MORE = [([100, 3], 64, 40, True, 0, 0), ([200], 256, 7, False, 0, 0), ([90, 0, 60], 1000, 63, True, 1, 1), ([129, 70], 516, 64, False, 0, 0),
        ([65, 64], 1024, 2500, True, 0, 0), ([20] * 3, 512, 2100, True, 0, 0), ([150] + [0] * 7, 132, 200, False, 2, 2),
        ([33, 31, 1, 0], 2048, 15, True, 0, 0), ([32, 32], 260, 16, False, 0, 0), ([17], 8, 17, True, 0, 0), ([4] * 9, 400, 1031, True, 0, 1)]


@pytest.mark.parametrize("case", MORE, ids=_name)
def test_backward_of_other_tiles(dev, case):
    test_backward(dev, case)


@pytest.mark.parametrize("case", MORE, ids=_name)
def test_gated_backward_of_other_tiles(dev, case):
    test_gated_backward(dev, case)


@pytest.mark.parametrize("m", [40, 400])
def test_indices_and_offsets_out_of_range(dev, m):
    """Tokens that are not there are zeros; offsets beyond the rows are taken as their ends."""
    torch, bl = dev
    rng = np.random.default_rng(11)
    e, k, n, t = 5, 256, 160, 9
    offsets = np.array([-7, 3, 3, m // 2, m // 2 + 1, m + 50], dtype=np.int64)
    rows = rng.integers(0, t, m).astype(np.int64)
    rows[[0, 5, m - 1]] = [-1, t, 1 << 40]
    rows[7] = -(1 << 62)
    w, alpha, b = _weights(rng, e, n, k, True)
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    args = [_t(torch, a) for a in (x_q, beta, offsets, _pack(w), alpha)]
    y = bl.bitlinear_grouped_forward(*args, rows=_t(torch, rows), bias=_t(torch, b))
    xr, br = experts_plain.tokens(x_q, beta, rows, m)
    assert np.array_equal(_np(y), experts_plain.forward(xr, br, offsets, w, alpha, b, np.zeros((m, n), F32)))
    dy = _gradient_inputs(rng, m, n)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((m, k), (e, n, k), (e, n)))
    bl.bitlinear_grouped_backward(_t(torch, dy), *args, rows=_t(torch, rows), dx=dx, dW=dw, dbias=db)
    values, terms, lengths = experts_plain.gradients([dy.astype(np.float64)], [w], [alpha], xr, br, offsets, np.zeros((m, k)))
    _check_gradients([dx, dw, db], values, terms, lengths, "range")


@pytest.mark.parametrize("m,e", [(40, 9), (700, 60), (1 << 14, 4096)])
def test_offsets_that_decrease_touch_nothing_else(dev, m, e):
    """Groups that share rows make more tiles than were launched: outputs are unspecified, what lies around
    them is not touched, and the next call is right."""
    torch, bl = dev
    rng = np.random.default_rng([19, m])
    k, n = 64, 40
    offsets = np.where(np.arange(e + 1) % 2 == 0, 0, m).astype(np.int64)
    w, alpha, _ = _weights(rng, e, n, k, False)
    x_q, beta = rng.integers(-127, 128, (m, k)).astype(np.int8), rng.uniform(0.5, 4, m).astype(F32)
    dy = rng.standard_normal((m, n)).astype(F32)
    xt, bt, ot, wt, at, dyt = [_t(torch, a) for a in (x_q, beta, offsets, _pack(w), alpha, dy)]

    def between(*shape):
        size = int(np.prod(shape))
        buf = torch.full((size + 512,), 7.0, device="cuda")
        return buf, buf[256:256 + size].view(shape)

    bufs, (y, dx, dw, db) = zip(*[between(*s) for s in ((m, n), (m, k), (e, n, k), (e, n))])
    bl.bitlinear_grouped_forward(xt, bt, ot, wt, at, y=y)
    bl.bitlinear_grouped_backward(dyt, xt, bt, ot, wt, at, dx=dx, dW=dw, dbias=db)
    torch.cuda.synchronize()
    for b in bufs:
        assert bool((b[:256] == 7).all()) and bool((b[-256:] == 7).all())
    one = np.full(e + 1, m, np.int64)
    one[0] = 0
    y = bl.bitlinear_grouped_forward(xt[:33], bt[:33], _t(torch, np.minimum(one, 33)), wt, at)
    assert np.array_equal(_np(y), experts_plain.forward(x_q[:33], beta[:33], np.minimum(one, 33), w, alpha, None, np.zeros((33, n), F32)))


def test_no_rows(dev):
    torch, bl = dev
    e, k, n = 3, 64, 40
    w = torch.zeros(e, n, k // 4, dtype=torch.uint8, device="cuda")
    alpha, offsets = torch.ones(e, device="cuda"), torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    for t, rows in ((0, None), (4, none), (0, none)):
        x_q, beta = torch.zeros(t, k, dtype=torch.int8, device="cuda"), torch.ones(t, device="cuda")
        assert bl.bitlinear_grouped_forward(x_q, beta, offsets, w, alpha, rows=rows).shape == (0, n)
        x = torch.ones(t, k, device="cuda")
        assert bl.bitlinear_grouped_gated_forward(x, offsets, w, alpha, w, alpha, bl.BITLINEAR_ACT_SILU, rows=rows, x_q=x_q,
                                                  beta=beta).shape == (0, n)
        assert bool((x_q == 127).all())
        dw, db = torch.full((e, n, k), 7.0, device="cuda"), torch.full((e, n), 7.0, device="cuda")
        bl.bitlinear_grouped_backward(torch.empty(0, n, device="cuda"), x_q, beta, offsets, w, alpha, rows=rows, dW=dw, dbias=db)
        assert bool((dw == 0).all()) and bool((db == 0).all())
        z = torch.empty(0, n, device="cuda")
        _, dwg, dwu, _, _ = bl.bitlinear_grouped_gated_backward(z, z, z, x_q, beta, offsets, w, alpha, w, alpha,
                                                                bl.BITLINEAR_ACT_GELU, rows=rows)
        assert bool((dwg == 0).all()) and bool((dwu == 0).all())


def test_gradients_that_are_not_finite_stay(dev):
    """NaN and infinities in dy reach their row of dx and their row of dW only."""
    torch, bl = dev
    rng = np.random.default_rng(13)
    counts, k, n = [40, 0, 200, 9], 256, 150
    offsets, _, m, _ = _layout(rng, counts, False)
    w, alpha, _ = _weights(rng, 4, n, k, False)
    x_q, beta = rng.integers(1, 128, (m, k)).astype(np.int8), rng.uniform(0.5, 4, m).astype(F32)
    dy = _gradient_inputs(rng, m, n)
    args = [_t(torch, a) for a in (x_q, beta, offsets, _pack(w), alpha)]
    clean = bl.bitlinear_grouped_backward(_t(torch, dy), *args)
    bad = dy.copy()
    bad[50, 7], bad[241, 149] = np.nan, np.inf
    dx, dw, _ = bl.bitlinear_grouped_backward(_t(torch, bad), *args)
    rows, cols = np.ones(m, bool), np.ones((4, n), bool)
    rows[[50, 241]] = False
    cols[2, 7] = cols[3, 149] = False
    assert np.array_equal(_np(dx)[rows], _np(clean[0])[rows]) and np.array_equal(_np(dw)[cols], _np(clean[1])[cols])
    assert not np.isfinite(_np(dx)[~rows]).any() and not np.isfinite(_np(dw)[~cols]).any()


def test_gradients_over_a_hundred_binades(dev):
    """Elements of any size beside each other keep their accuracy: every sum is of terms of one size."""
    torch, bl = dev
    rng = np.random.default_rng(17)
    counts, k, n = [33, 100], 192, 96
    offsets, _, m, _ = _layout(rng, counts, False)
    w, alpha, _ = _weights(rng, 2, n, k, False)
    # half of n has weights in half of k, and is 2^-100 of the other half
    w[:, : n // 2, : k // 2] = 0
    w[:, n // 2:, k // 2:] = 0
    x_q, beta = rng.integers(-127, 128, (m, k)).astype(np.int8), rng.uniform(0.5, 4, m).astype(F32)
    dy = rng.standard_normal((m, n)).astype(F32)
    dy[:, n // 2:] *= F32(2.0 ** -90)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((m, k), (2, n, k), (2, n)))
    bl.bitlinear_grouped_backward(*[_t(torch, a) for a in (dy, x_q, beta, offsets, _pack(w), alpha)], dx=dx, dW=dw, dbias=db)
    values, terms, lengths = experts_plain.gradients([dy.astype(np.float64)], [w], [alpha], x_q, beta, offsets, np.zeros((m, k)))
    _check_gradients([dx, dw, db], values, terms, lengths, "binades")


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(dev, act):
    """The gated block's gradients against central differences of the plain forward pass in 64 bits: the
    loss sum(dh h) as a function of the dequantized tokens and weights."""
    torch, bl = dev
    rng = np.random.default_rng(19)
    counts, k, f = [5, 0, 9, 20], 64, 24
    offsets, rows, m, t = _layout(rng, counts, True)
    w = [_weights(rng, 4, f, k, False) for _ in range(2)]
    x = rng.standard_normal((t, k)).astype(F32)
    xq, beta = plain.absmax(x)
    dh = rng.standard_normal((m, f)).astype(F32)
    g, u, h = (torch.empty(m, f, device="cuda") for _ in range(3))
    x_q, bt = torch.empty((t, k), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    wt = [v for (a, al, _) in w for v in (_t(torch, _pack(a)), _t(torch, al))]
    off, r = _t(torch, offsets), _t(torch, rows)
    bl.bitlinear_grouped_gated_forward(_t(torch, x), off, *wt, _code(bl, act), rows=r, h=h, g=g, u=u, x_q=x_q, beta=bt)
    dx, dwg, dwu, _, _ = bl.bitlinear_grouped_gated_backward(_t(torch, dh), g, u, x_q, bt, off, *wt, _code(bl, act), rows=r)
    xr, br = experts_plain.tokens(xq, beta, rows, m)
    real = xr.astype(np.float64) * br.astype(np.float64)[:, None] / 127
    ws = [a.astype(np.float64) * al.astype(np.float64)[:, None, None] for a, al, _ in w]
    group = np.searchsorted(offsets, np.arange(m), side="right") - 1

    def loss(xd, wg, wu):
        gg = np.einsum("mk,mfk->mf", xd, wg[group])
        uu = np.einsum("mk,mfk->mf", xd, wu[group])
        return float(np.sum(dh.astype(np.float64) * plain.activation(gg, act)[0] * uu))

    step = 1e-6
    for i, (grad, at) in enumerate(((dx, real), (dwg, ws[0]), (dwu, ws[1]))):
        for _ in range(3):
            v = rng.standard_normal(at.shape)
            args = [real, ws[0], ws[1]]
            up, down = list(args), list(args)
            up[i], down[i] = at + step * v, at - step * v
            slope = (loss(*up) - loss(*down)) / (2 * step)
            mine = float(np.sum(_np(grad).astype(np.float64) * v))
            # differences: step^2 times the third derivative, and cancellation of 2^-53 of the loss over the
            # step; the gradient's own 2^-18 of the root sum of squares of its products with v
            scale = float(np.sqrt(np.sum((_np(grad).astype(np.float64) * v) ** 2)))
            assert abs(mine - slope) <= 2.0 ** -18 * scale + 1e-6 * abs(slope) + 1e-5, (act, i)


@pytest.mark.parametrize("t,top,k,f", [(1, 2, 256, 200), (24, 3, 320, 256), (300, 2, 512, 640)])
def test_a_layer_in_a_graph(dev, t, top, k, f):
    """An fp8 projection, the experts' gated block, its quantizer and the experts' down projection, then
    both gradients, captured once and replayed with other tokens and other routes; every replay against
    the eager calls, which are against the plain forms above."""
    torch, bl = dev
    e = 6
    rng = np.random.default_rng([23, t])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t)
    m = t * top
    wg_, ag_, bg_ = _weights(rng, e, f, k, True)
    wu_, au_, _ = _weights(rng, e, f, k, False)
    wd_, ad_, _ = _weights(rng, e, k, f, False)
    wg_p, ag, bg = _t(torch, _pack(wg_)), _t(torch, ag_), _t(torch, bg_)
    wu_p, au = _t(torch, _pack(wu_)), _t(torch, au_)
    wd_p, ad = _t(torch, _pack(wd_)), _t(torch, ad_)
    p_q, ps = bl.bitlinear_quantize_weights_fp8(torch.randn(k, k, device="cuda", generator=gen) * 0.05)
    x = torch.empty(t, k, device="cuda")
    rows = torch.empty(m, dtype=torch.int64, device="cuda")
    offsets = torch.empty(e + 1, dtype=torch.int64, device="cuda")
    dy = torch.empty(m, k, device="cuda")

    def buffers():
        fl = lambda *s: torch.full(s, float("nan"), device="cuda")
        return dict(x_q8=torch.empty(t, k, dtype=torch.float8_e4m3fn, device="cuda"), xs=fl(-(-k // 128), t), z=fl(t, k),
                    h=fl(m, f), g=fl(m, f), u=fl(m, f), x_q=torch.empty(t, k, dtype=torch.int8, device="cuda"), beta=fl(t),
                    h_q=torch.empty(m, f, dtype=torch.int8, device="cuda"), hb=fl(m), y=fl(m, k), dh=fl(m, f), dwd=fl(e, k, f),
                    dx=fl(m, k), dwg=fl(e, f, k), dwu=fl(e, f, k), dbg=fl(e, f),
                    ws1=torch.empty(bl.bitlinear_grouped_backward_workspace_size(m, f, k, e), dtype=torch.uint8, device="cuda"),
                    ws2=torch.empty(bl.bitlinear_grouped_gated_backward_workspace_size(m, k, f, e), dtype=torch.uint8, device="cuda"))

    def step(o):
        bl.bitlinear_quantize_act_fp8(x, x_q=o["x_q8"], x_scale=o["xs"])
        bl.bitlinear_forward_fp8(o["x_q8"], o["xs"], p_q, ps, y=o["z"])
        bl.bitlinear_grouped_gated_forward(o["z"], offsets, wg_p, ag, wu_p, au, bl.BITLINEAR_ACT_SILU, rows=rows, bias_g=bg,
                                           h=o["h"], g=o["g"], u=o["u"], x_q=o["x_q"], beta=o["beta"])
        bl.bitlinear_quantize_act(o["h"], x_q=o["h_q"], beta=o["hb"])
        bl.bitlinear_grouped_forward(o["h_q"], o["hb"], offsets, wd_p, ad, y=o["y"])
        bl.bitlinear_grouped_backward(dy, o["h_q"], o["hb"], offsets, wd_p, ad, dx=o["dh"], dW=o["dwd"], workspace=o["ws1"])
        bl.bitlinear_grouped_gated_backward(o["dh"], o["g"], o["u"], o["x_q"], o["beta"], offsets, wg_p, ag, wu_p, au,
                                            bl.BITLINEAR_ACT_SILU, rows=rows, dx=o["dx"], dWg=o["dwg"], dWu=o["dwu"],
                                            dbias_g=o["dbg"], workspace=o["ws2"])

    def inputs():
        x.copy_(torch.randn(t, k, device="cuda", generator=gen))
        dy.copy_(torch.randn(m, k, device="cuda", generator=gen))
        chosen = torch.rand(t, e, device="cuda", generator=gen).topk(top, dim=1).indices.reshape(-1)
        rows.copy_(torch.argsort(chosen, stable=True) // top)
        counts = torch.bincount(chosen, minlength=e)
        offsets.copy_(torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]))

    a, b = buffers(), buffers()
    inputs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(4):
        inputs()
        graph.replay()
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        for name in ("z", "h", "y", "dh", "dwd", "dx", "dwg", "dwu", "dbg"):
            assert torch.equal(a[name], b[name]) and bool(torch.isfinite(a[name]).all()), (i, name)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = bl.bitlinear_grouped_forward(a["h_q"], a["hb"], offsets, wd_p, ad, stream=side)
    dx, dw, _ = bl.bitlinear_grouped_backward(dy, a["h_q"], a["hb"], offsets, wd_p, ad, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, a["y"]) and torch.equal(dx, a["dh"]) and torch.equal(dw, a["dwd"])


@pytest.mark.parametrize("m", [6, 900])
def test_weights_past_32_bit_offsets(dev, m):
    """Experts' weights past 2^32 bytes: the last expert's rows are read where they lie."""
    torch, bl = dev
    e, n, k = 36, 16384, 32768
    w = torch.full((e, n, k // 4), 0x55, dtype=torch.uint8, device="cuda")            # zeros
    w[-1, -2:, :3] = 0xAA                                                             # twelve ones
    alpha = torch.full((e,), 2.0, device="cuda")
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[-1] = m
    offsets[-2] = 1
    x_q, beta = torch.full((m, k), 3, dtype=torch.int8, device="cuda"), torch.full((m,), 127.0, device="cuda")
    _say(f"grouped_forward past 2^32 bytes, M={m}")
    y = bl.bitlinear_grouped_forward(x_q, beta, offsets, w, alpha)
    assert bool((y[1:, -2:] == 72).all()) and bool((y[:, :-2] == 0).all()) and bool((y[0] == 0).all())
    dx, _, _ = bl.bitlinear_grouped_backward(torch.ones(m, n, device="cuda"), x_q, beta, offsets, w, alpha,
                                             dx=torch.empty(m, k, device="cuda"))
    assert bool((dx[1:, :12] == 4).all()) and bool((dx[1:, 12:] == 0).all()) and bool((dx[0] == 0).all())


def test_outputs_past_32_bit_offsets(dev):
    torch, bl = dev
    m, n, k, e = 40000, 32768, 64, 2
    w = torch.full((e, n, k // 4), 0x55, dtype=torch.uint8, device="cuda")
    w[1, -1] = 0xAA
    alpha = torch.ones(e, device="cuda")
    offsets = torch.tensor([0, 7, m], dtype=torch.int64, device="cuda")
    x_q, beta = torch.ones((m, k), dtype=torch.int8, device="cuda"), torch.full((m,), 127.0, device="cuda")
    _say("grouped_forward with outputs past 2^32 bytes")
    y = bl.bitlinear_grouped_forward(x_q, beta, offsets, w, alpha)
    assert bool((y[7:, -1] == k).all()) and bool((y[:7] == 0).all()) and bool((y[:, :-1] == 0).all())
    dx, dw, _ = bl.bitlinear_grouped_backward(y, x_q, beta, offsets, w, alpha)
    # dy is k in the last column of group 1
    assert bool((dx[7:] == k).all()) and bool((dx[:7] == 0).all())
    assert bool((dw[1, -1] == float((m - 7) * k)).all()) and bool((dw[0] == 0).all()) and bool((dw[1, :-1] == 0).all())


@pytest.mark.parametrize("m", [6, 900])
def test_tokens_past_32_bit_offsets(dev, m):
    """Tokens' codes past 2^32 bytes, gathered: forward, gated forward's rows and dW of short and long groups."""
    torch, bl = dev
    t, k, n, e = 140000, 32768, 1088, 2
    x_q, beta = torch.zeros(t, k, dtype=torch.int8, device="cuda"), torch.full((t,), 127.0, device="cuda")
    x_q[-1] = 3
    x_q[1, 5] = 7
    rows = torch.full((m,), t - 1, dtype=torch.int64, device="cuda")
    rows[0] = 1
    w = torch.full((e, n, k // 4), 0x55, dtype=torch.uint8, device="cuda")
    w[1, :, 0] = 0xAA                                                                 # four ones
    alpha = torch.full((e,), 2.0, device="cuda")
    offsets = torch.tensor([0, 2, m], dtype=torch.int64, device="cuda")
    _say(f"grouped calls with tokens past 2^32 bytes, M={m}")
    y = bl.bitlinear_grouped_forward(x_q, beta, offsets, w, alpha, rows=rows)
    assert bool((y[:2] == 0).all()) and bool((y[2:] == 24).all())
    dy = torch.ones(m, n, device="cuda")
    dx, dw, _ = bl.bitlinear_grouped_backward(dy, x_q, beta, offsets, w, alpha, rows=rows)
    assert bool((dx[2:, :4] == 2 * n).all()) and bool((dx[:, 4:] == 0).all()) and bool((dx[:2] == 0).all())
    want = torch.full((k,), 3.0, device="cuda")
    want[5] += 7
    assert bool((dw[0] == want).all()) and bool((dw[1] == 3.0 * (m - 2)).all())


def test_gradients_past_32_bit_offsets(dev):
    """dW of short groups past 2^32 elements."""
    torch, bl = dev
    m, n, k, e = 40, 16384, 16384, 18
    w = torch.full((e, n, k // 4), 0x55, dtype=torch.uint8, device="cuda")
    w[-1, :, -1] = 0xAA
    offsets = torch.full((e + 1,), m, dtype=torch.int64, device="cuda")
    offsets[:-1] = 0
    offsets[1:-1] = 1
    x_q, beta = torch.ones((m, k), dtype=torch.int8, device="cuda"), torch.full((m,), 127.0, device="cuda")
    _say("grouped_backward with dW past 2^32 elements")
    dy = torch.zeros(m, n, device="cuda")
    dy[:, -1] = 2
    dx, dw, _ = bl.bitlinear_grouped_backward(dy, x_q, beta, offsets, w, torch.ones(e, device="cuda"))
    assert bool((dw[-1, -1] == 2.0 * (m - 1)).all()) and bool((dw[-1, :-1] == 0).all()) and bool((dw[1:-1] == 0).all())
    assert bool((dw[0, -1] == 2).all()) and bool((dw[0, :-1] == 0).all())
    assert bool((dx[1:, -4:] == 2).all()) and bool((dx[:, :-4] == 0).all()) and bool((dx[0] == 0).all())


@pytest.mark.parametrize("each", [1, 36])
def test_most_experts(dev, each):
    """4096 experts, every third without rows, of few rows and of many."""
    torch, bl = dev
    rng = np.random.default_rng([31, each])
    e, k, n = 4096, 64, 24
    counts = rng.integers(0, 2 * each + 1, e)
    counts[::3] = 0
    if each > 1:
        counts[1::3] += 33
    offsets, rows, m, t = _layout(rng, counts, True, 0, 2)
    w, alpha, _ = _weights(rng, e, n, k, False)
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    dy = _gradient_inputs(rng, m, n)
    args = [_t(torch, a) for a in (x_q, beta, offsets, _pack(w), alpha)]
    kw = dict(rows=_t(torch, rows))
    _say(f"4096 experts, M={m}")
    y = torch.full((m, n), 7.0, device="cuda")
    bl.bitlinear_grouped_forward(*args, y=y, **kw)
    xr, br = experts_plain.tokens(x_q, beta, rows, m)
    assert np.array_equal(_np(y), experts_plain.forward(xr, br, offsets, w, alpha, None, np.full((m, n), 7, F32)))
    dx, dw, db = (torch.zeros(s, device="cuda") for s in ((m, k), (e, n, k), (e, n)))
    bl.bitlinear_grouped_backward(_t(torch, dy), *args, dx=dx, dW=dw, dbias=db, **kw)
    values, terms, lengths = experts_plain.gradients([dy.astype(np.float64)], [w], [alpha], xr, br, offsets, np.zeros((m, k)))
    _check_gradients([dx, dw, db], values, terms, lengths, "4096")


@pytest.mark.parametrize("counts,k,n", [([20, 3, 40], 1024, 600), ([300, 90], 512, 1024)])
def test_two_calls_at_once(dev, counts, k, n):
    """Calls on two streams, each with its workspace and outputs, over and over: as the calls one after the other."""
    torch, bl = dev
    rng = np.random.default_rng([37, k])
    e = len(counts)
    offsets, rows, m, t = _layout(rng, counts, True)
    sides = []
    for _ in range(2):
        wg, ag, _ = _weights(rng, e, n, k, False)
        wu, au, _ = _weights(rng, e, n, k, False)
        x = rng.standard_normal((t, k)).astype(F32)
        dh = _gradient_inputs(rng, m, n)
        sides.append([_t(torch, a) for a in (x, offsets, _pack(wg), ag, _pack(wu), au, rows, dh)])

    def call(x, offsets, wg, ag, wu, au, rows, dh, stream):
        act = bl.BITLINEAR_ACT_SILU
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
        o = dict(h=new(m, n), g=new(m, n), u=new(m, n), x_q=new(t, k, dtype=torch.int8), beta=new(t), dx=new(m, k), dg=new(e, n, k), du=new(e, n, k))
        ws = new(bl.bitlinear_grouped_gated_backward_workspace_size(m, k, n, e), dtype=torch.uint8)
        stream.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            bl.bitlinear_grouped_gated_forward(x, offsets, wg, ag, wu, au, act, rows=rows, h=o["h"], g=o["g"], u=o["u"], x_q=o["x_q"],
                                               beta=o["beta"], stream=stream)
            bl.bitlinear_grouped_gated_backward(dh, o["g"], o["u"], o["x_q"], o["beta"], offsets, wg, ag, wu, au, act, rows=rows, dx=o["dx"],
                                                dWg=o["dg"], dWu=o["du"], workspace=ws, stream=stream)
        return o, ws

    streams = [torch.cuda.Stream() for _ in range(2)]
    at_once = [call(*s, stream) for s, stream in zip(sides, streams)]
    torch.cuda.synchronize()
    for s, (o, _) in zip(sides, at_once):
        alone, _ = call(*s, streams[0])
        torch.cuda.synchronize()
        for name in ("h", "g", "u", "dx", "dg", "du"):
            assert torch.equal(o[name], alone[name]), name
