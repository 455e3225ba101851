"""GPU tests of the gated feed-forward block, the BitLinear gradients and the W8A8 product against
plain 64-bit forms: integer sums and documented 32-bit steps bit for bit, activations and gradients
within bounds counted in roundings."""
import numpy as np
import pytest

import ffn_plain as plain
from ffn_plain import U

pytestmark = pytest.mark.gpu

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


def _f32(a):
    return np.asarray(a, dtype=np.float32)


def _bits(a):
    return np.ascontiguousarray(a).view(np.uint32)


def _layer(rng, n, k, bias):
    w = plain.ternary(rng, n, k)
    alpha = _f32(rng.uniform(0.01, 0.02, 1))
    return w, alpha, (_f32(rng.standard_normal(n) * 0.1) if bias else None)


# ------------------------------------------------------------------------------ gated forward
GATED = [(1, 4, 1), (1, 64, 3), (1, 4096, 200), (1, 1088, 77), (1, 8192, 33), (1, 11008, 64), (1, 100, 130),
         (2, 256, 16), (3, 4096, 100), (5, 68, 33), (8, 512, 17), (16, 2048, 300), (16, 320, 65), (17, 1024, 48),
         (31, 192, 40), (33, 768, 129), (48, 256, 31), (64, 4096, 96), (64, 4100, 20), (65, 512, 200), (128, 64, 128),
         (129, 1028, 257), (200, 640, 130), (300, 4096, 260)]


@pytest.mark.parametrize("m,k,f", GATED)
def test_gated_forward(dev, m, k, f):
    torch, bl = dev
    act = ACTS[(m + k // 4 + f) % 3]
    bias = (m + f) % 2 == 0
    _say(f"gated_forward M={m} K={k} F={f} {act} bias={bias}")
    rng = np.random.default_rng([7, m, k, f])
    x = _f32(rng.standard_normal((m, k)))
    wg, ag, bg = _layer(rng, f, k, bias)
    wu, au, bu = _layer(rng, f, k, bias)
    g, u = (torch.full((m, f), float("nan"), device="cuda") for _ in range(2))
    x_q = torch.empty((m, k), dtype=torch.int8, device="cuda")
    beta = torch.empty(m, device="cuda")
    args = (_t(torch, x), _t(torch, plain.pack(wg)), _t(torch, ag), _t(torch, plain.pack(wu)), _t(torch, au), _code(bl, act))
    kw = dict(bias_g=_t(torch, bg), bias_u=_t(torch, bu))
    h = bl.bitlinear_gated_forward(*args, g=g, u=u, x_q=x_q, beta=beta, **kw)
    h2 = bl.bitlinear_gated_forward(*args, **kw)
    torch.cuda.synchronize()
    xq_p, beta_p = plain.absmax(x)
    assert np.array_equal(_np(x_q), xq_p) and np.array_equal(_bits(_np(beta)), _bits(beta_p))
    g_p = plain.project(xq_p, beta_p, wg, ag[0], bg)
    u_p = plain.project(xq_p, beta_p, wu, au[0], bu)
    assert np.array_equal(_np(g), g_p) and np.array_equal(_np(u), u_p)
    # roundings of a(g): SiLU 7, GELU and squared ReLU 1, and the product's, to first order
    ref = plain.activation(g_p, act)[0] * u_p.astype(np.float64)
    n = {"silu": 8, "gelu": 2, "relu2": 2}[act]
    assert np.all(np.abs(_np(h) - ref) <= 1.01 * n * U * np.abs(ref) + 1e-37)
    # without g and u the same h
    assert np.array_equal(_bits(_np(h2)), _bits(_np(h)))


@pytest.mark.parametrize("act", ACTS)
def test_gated_forward_extremes(dev, act):
    """Zero rows, gates far out on both sides, alpha 0: finite, and the limits of a(g)."""
    torch, bl = dev
    rng = np.random.default_rng(5)
    m, k, f = 6, 256, 40
    x = _f32(rng.standard_normal((m, k)))
    x[1] = 0
    x[3] *= 1e-30
    x[4] *= 300
    wg, _, _ = _layer(rng, f, k, False)
    wu, _, _ = _layer(rng, f, k, False)
    for ag in (0.0, 0.015, 2.0):
        a1, a2 = _f32([ag]), _f32([0.5])
        h = bl.bitlinear_gated_forward(_t(torch, x), _t(torch, plain.pack(wg)), _t(torch, a1), _t(torch, plain.pack(wu)),
                                       _t(torch, a2), _code(bl, act))
        xq_p, beta_p = plain.absmax(x)
        g_p = plain.project(xq_p, beta_p, wg, a1[0], None)
        u_p = plain.project(xq_p, beta_p, wu, a2[0], None)
        ref = plain.activation(g_p, act)[0] * u_p.astype(np.float64)
        n = {"silu": 8, "gelu": 2, "relu2": 2}[act]
        h = _np(h)
        assert np.all(np.isfinite(h)) and np.all(h[1] == 0)
        # below 2^-100 a(g) may have lost bits to underflow (its absolute value is what is left)
        assert np.all(np.abs(h - ref) <= 1.01 * n * U * np.abs(ref) + 2.0 ** -120 * (1 + np.abs(u_p)))


def test_gated_forward_unaligned_views(dev):
    """Every tensor a contiguous view that starts off any vector alignment."""
    torch, bl = dev
    rng = np.random.default_rng(9)

    def off(a, n):
        t = _t(torch, a)
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        v = buf[n:].view(t.shape)
        v.copy_(t)
        return v

    for m, k, f in [(1, 256, 20), (9, 512, 33), (70, 256, 140)]:
        _say(f"gated_forward unaligned M={m} K={k} F={f}")
        x = _f32(rng.standard_normal((m, k)))
        wg, ag, bg = _layer(rng, f, k, True)
        wu, au, bu = _layer(rng, f, k, True)
        h = torch.full((m * f + 64,), 7.0, device="cuda")
        x_q = torch.empty(m * k + 3, dtype=torch.int8, device="cuda")[3:].view(m, k)
        bl.bitlinear_gated_forward(off(x, 1), off(plain.pack(wg), 1), off(ag, 1), off(plain.pack(wu), 3), off(au, 3),
                                   bl.BITLINEAR_ACT_RELU2, bias_g=off(bg, 1), bias_u=off(bu, 1),
                                   h=h[1:1 + m * f].view(m, f), x_q=x_q)
        xq_p, beta_p = plain.absmax(x)
        r = np.maximum(plain.project(xq_p, beta_p, wg, ag[0], bg), np.float32(0))
        ref = (r * r) * plain.project(xq_p, beta_p, wu, au[0], bu)
        hn = _np(h)
        assert np.array_equal(hn[1:1 + m * f].reshape(m, f), ref)
        assert hn[0] == 7.0 and np.all(hn[1 + m * f:] == 7.0)


# ---------------------------------------------------------------------------------- gradients
GRADS = [(1, 4, 1), (1, 256, 33), (2, 64, 130), (7, 100, 31), (16, 512, 64), (33, 132, 70), (61, 1024, 171),
         (64, 64, 64), (100, 260, 300), (129, 516, 129), (257, 320, 65), (300, 128, 520), (700, 68, 40)]
# few tokens: rows past one, two and three times 64 a workgroup, in one chunk and in many, columns past a tile
GRADS += [(3, 4, 1), (4, 8, 17), (5, 1028, 70), (8, 4096, 2501), (9, 4100, 4700), (15, 260, 515), (16, 12, 9000),
          (16, 2052, 1111), (17, 2052, 111)]
# up to 64 tokens: short rows of codes, rows and columns past a tile, and more tiles than go in one pass
GRADS += [(17, 4, 1), (20, 8, 70), (33, 12, 64), (64, 16, 65), (32, 1028, 129), (40, 260, 700), (64, 2052, 190),
          (24, 4100, 4200), (61, 8200, 2100)]
# more tokens, in too many tiles for one pass: every size of tile of the maxima
GRADS += [(100, 2100, 2100), (129, 4100, 700), (257, 2052, 1030), (300, 260, 4100), (700, 68, 3100)]


def _check(got, want, terms, lengths, names):
    for t, w, s, n, name in zip(got, want, terms, lengths, names):
        err = np.abs(_np(t).astype(np.float64) - w)
        tol = plain.gradient_tolerance(s, n)
        assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("m,k,n", GRADS)
def test_backward(dev, m, k, n):
    torch, bl = dev
    _say(f"backward M={m} K={k} N={n}")
    rng = np.random.default_rng([8, m, k, n])
    dy = _f32(rng.standard_normal((m, n)) * np.exp(rng.standard_normal((m, 1))) / m)
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    w, al, _ = _layer(rng, n, k, False)
    args = (_t(torch, dy), _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    out = bl.bitlinear_backward(*args, dx=nan(m, k), dW=nan(n, k), dbias=nan(n))
    torch.cuda.synchronize()
    want, terms = plain.linear_gradients(dy, x_q, beta, w, al[0])
    _check(out, want, terms, [n, m, m], ["dx", "dW", "dbias"])
    # each output alone, and a second call: the same bits
    for i, name in enumerate(["dx", "dW", "dbias"]):
        alone = bl.bitlinear_backward(*args, **{name: torch.empty_like(out[i])})
        assert torch.equal(alone[i], out[i]), name
        assert all(o is None for j, o in enumerate(alone) if j != i)


@pytest.mark.parametrize("m,k,f", GRADS)
def test_gated_backward(dev, m, k, f):
    torch, bl = dev
    act = ACTS[(m + k // 4 + f) % 3]
    _say(f"gated_backward M={m} K={k} F={f} {act}")
    rng = np.random.default_rng([9, m, k, f])
    dh = _f32(rng.standard_normal((m, f)) / m)
    g, u = (_f32(rng.standard_normal((m, f)) * 2) for _ in range(2))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    wg, ag, _ = _layer(rng, f, k, False)
    wu, au, _ = _layer(rng, f, k, False)
    args = (_t(torch, dh), _t(torch, g), _t(torch, u), _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(wg)),
            _t(torch, ag), _t(torch, plain.pack(wu)), _t(torch, au), _code(bl, act))
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    names = ["dx", "dWg", "dWu", "dbias_g", "dbias_u"]
    out = bl.bitlinear_gated_backward(*args, dx=nan(m, k), dWg=nan(f, k), dWu=nan(f, k), dbias_g=nan(f), dbias_u=nan(f))
    torch.cuda.synchronize()
    want, terms = plain.gated_gradients(dh, g, u, x_q, beta, wg, ag[0], wu, au[0], act)
    # a'(g) of SiLU and GELU passes through zero, where its error is 2^-24 of its parts, at most 2
    # in size: counted as roundings of dh u
    if act != "relu2":
        d0 = np.abs(dh.astype(np.float64) * u)
        xd = np.abs(x_q.astype(np.float64)) * beta[:, None] / 127
        extra = 24 * U * np.stack([0 * d0, d0])
        slack = [extra[1] @ np.abs(wg).astype(np.float64) * ag[0], extra[1].T @ xd, 0, extra[1].sum(0), 0]
    else:
        slack = [0, 0, 0, 0, 0]
    for t, w, s, n, sl, name in zip(out, want, terms, [2 * f, m, m, m, m], slack, names):
        err = np.abs(_np(t).astype(np.float64) - w)
        assert np.all(err <= plain.gradient_tolerance(s, n) + sl), name
    for keep in (["dx"], ["dWg", "dWu"], ["dbias_g"], ["dbias_u", "dx"]):
        alone = dict(zip(names, bl.bitlinear_gated_backward(*args, **{q: torch.empty_like(out[names.index(q)]) for q in keep})))
        for q in names:
            assert alone[q] is None if q not in keep else torch.equal(alone[q], out[names.index(q)]), (keep, q)


def _wide_range(dev, m, k=132, n=90):
    torch, bl = dev
    rng = np.random.default_rng(3)
    dy = _f32(rng.standard_normal((m, n)))
    dy[0] = 0
    dy[:, 1] = 0
    dy[2] *= _f32(1e-30)
    dy[3] *= _f32(1e30)
    dy[:, 4] *= _f32(2.0 ** -30)
    dy[5] *= _f32(np.exp2(-rng.integers(0, 16, n)))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    w, al, _ = _layer(rng, n, k, False)
    out = bl.bitlinear_backward(_t(torch, dy), _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    want, terms = plain.linear_gradients(dy, x_q, beta, w, al[0])
    dx, dw = _np(out[0]).astype(np.float64), _np(out[1]).astype(np.float64)
    # elements below 2^-17 of their row's largest are held to 2^-40 of it
    row = np.abs(dy.astype(np.float64)).max(1)[:, None] * al[0] * 2.0 ** -40 * n
    assert np.all(np.abs(dx - want[0]) <= plain.gradient_tolerance(terms[0], n) + row)
    v = np.abs(dy.astype(np.float64) * beta[:, None] / 127)
    col = v.max(0)[:, None] * 2.0 ** -40 * m * 127
    assert np.all(np.abs(dw - want[1]) <= plain.gradient_tolerance(terms[1], m) + col)
    assert np.all(dx[0] == 0) and np.all(dw[1] == 0)


def test_backward_wide_range(dev):
    """Gradients of very different sizes in one row and one column, zero rows and columns, and rows
    at the ends of the fp32 range: every row of dx and of dW keeps its own accuracy."""
    _wide_range(dev, 70)


@pytest.mark.parametrize("m", [6, 12, 40])
def test_backward_wide_range_few_tokens(dev, m):
    _wide_range(dev, m)


def test_backward_wide_range_many_tiles(dev):
    _wide_range(dev, 70, 2100, 2300)


@pytest.mark.parametrize("m,k,n", [(5, 268, 131), (13, 268, 131), (40, 268, 131), (100, 268, 131), (100, 2100, 2107)])
def test_backward_unaligned_views(dev, m, k, n):
    """Every tensor off its alignment; what lies around the outputs stays."""
    torch, bl = dev
    _say(f"backward unaligned M={m}")
    rng = np.random.default_rng([13, m])
    dy = _f32(rng.standard_normal((m, n)))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    w, al, _ = _layer(rng, n, k, False)

    def off(a, s):
        t = _t(torch, np.ascontiguousarray(a))
        v = torch.empty(t.numel() + s, dtype=t.dtype, device="cuda")[s:].view(t.shape)
        v.copy_(t)
        return v

    room = [torch.full((a * b + 64,), 3.0, device="cuda") for a, b in ((m, k), (n, k), (n, 1))]
    out = [r[1:1 + a * b].view(a, b) for r, (a, b) in zip(room, ((m, k), (n, k), (n, 1)))]
    bl.bitlinear_backward(off(dy, 1), off(x_q, 1), off(beta, 3), off(plain.pack(w), 3), off(al, 1), dx=out[0], dW=out[1],
                          dbias=out[2].view(n))
    want, terms = plain.linear_gradients(dy, x_q, beta, w, al[0])
    _check([out[0], out[1], out[2].view(n)], want, terms, [n, m, m], ["dx", "dW", "dbias"])
    for r, o in zip(room, out):
        assert float(r[0]) == 3.0 and bool((r[1 + o.numel():] == 3.0).all())


@pytest.mark.parametrize("m,k,f", [(1, 512, 300), (9, 260, 1100), (16, 1024, 640), (50, 520, 200)])
def test_backward_in_a_graph(dev, m, k, f):
    """Captured once and replayed with other inputs and eager work between: the eager call's bits."""
    torch, bl = dev
    _say(f"backward in a graph M={m} K={k} F={f}")
    s = _step_state(torch, bl, m, k, f, [14, m])
    _step(torch, bl, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(torch, bl, s)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        s["x"].copy_(torch.randn(m, k, device="cuda", generator=gen))
        s["dy"].copy_(torch.randn(m, k, device="cuda", generator=gen) / m)
        eager = [t.clone() for t in _step(torch, bl, s)]
        for t in ("dh", "dWd", "dx", "dWg", "dWu"):
            s[t].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, [s[q] for q in ("h", "y", "dh", "dWd", "dx", "dWg", "dWu")]):
            assert torch.equal(a, b)


def test_backward_against_differences(dev):
    """dW and dx against differences of the layer's own value: with the codes fixed the output is
    linear in the latent values, so a difference over a unit step is the derivative."""
    torch, bl = dev
    rng = np.random.default_rng(4)
    m, k, n = 5, 16, 6
    dy = _f32(rng.standard_normal((m, n)))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    w, al, _ = _layer(rng, n, k, False)
    dx, dw, _ = bl.bitlinear_backward(_t(torch, dy), _t(torch, x_q), _t(torch, beta), _t(torch, plain.pack(w)), _t(torch, al))
    xd = x_q.astype(np.float64) * beta[:, None] / 127
    wd = w.astype(np.float64) * float(al[0])
    loss = lambda a, b: float((dy.astype(np.float64) * (a @ b.T)).sum())
    base = loss(xd, wd)
    for i in range(n):
        for j in range(k):
            step = wd.copy()
            step[i, j] += 1
            assert abs(loss(xd, step) - base - float(dw[i, j])) <= 64 * U * (abs(base) + np.abs(dy[:, i] * xd[:, j]).sum())
    for i in range(m):
        for j in range(k):
            step = xd.copy()
            step[i, j] += 1
            assert abs(loss(step, wd) - base - float(dx[i, j])) <= 64 * U * (abs(base) + np.abs(dy[i] * wd[:, j]).sum())


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_against_differences(dev, act):
    """Every gradient of the block against central differences of its value in 64 bits, the codes
    fixed.  Steps of 2^-12: the third derivative's part is below 2^-24 times a few of its size."""
    torch, bl = dev
    rng = np.random.default_rng(6)
    m, k, f = 3, 8, 5
    dh = _f32(rng.standard_normal((m, f)))
    x_q, beta = plain.absmax(rng.standard_normal((m, k)))
    wg, ag, _ = _layer(rng, f, k, False)
    wu, au, _ = _layer(rng, f, k, False)
    ag, au = _f32([0.4]), _f32([0.3])
    xd = x_q.astype(np.float64) * beta[:, None] / 127
    mats = [xd, wg * float(ag[0]), wu * float(au[0])]
    bias = [_f32(rng.standard_normal(f) * 0.5) for _ in range(2)]

    def value(x, a, b, ba, bb):
        return float((dh * plain.activation(x @ a.T + ba, act)[0] * (x @ b.T + bb)).sum())

    g = _f32(xd @ mats[1].T + bias[0])
    u = _f32(xd @ mats[2].T + bias[1])
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    out = bl.bitlinear_gated_backward(_t(torch, dh), _t(torch, g), _t(torch, u), _t(torch, x_q), _t(torch, beta),
                                      _t(torch, plain.pack(wg)), _t(torch, ag), _t(torch, plain.pack(wu)), _t(torch, au),
                                      _code(bl, act), dx=nan(m, k), dWg=nan(f, k), dWu=nan(f, k), dbias_g=nan(f),
                                      dbias_u=nan(f))
    point = [mats[0], mats[1], mats[2], bias[0].astype(np.float64), bias[1].astype(np.float64)]
    e = 2.0 ** -12
    for i, t in enumerate(out):
        t = _np(t).astype(np.float64)
        for idx in np.ndindex(*point[i].shape):
            up, dn = [p.copy() for p in point], [p.copy() for p in point]
            up[i][idx] += e
            dn[i][idx] -= e
            diff = (value(*up) - value(*dn)) / (2 * e)
            assert abs(diff - t[idx]) <= 2e-5 * (1 + np.abs(t).max()), (act, i, idx)


# ------------------------------------------------------------------------------------ W8A8
I8 = [(1, 1, 1), (1, 16, 5), (1, 4096, 300), (1, 1001, 77), (1, 11008, 40), (2, 64, 16), (3, 4097, 33), (7, 256, 100),
      (16, 1024, 48), (16, 100, 515), (17, 640, 64), (33, 333, 65), (48, 2048, 129), (64, 512, 256), (64, 8192, 40),
      (65, 128, 130), (100, 65, 200), (128, 64, 256), (129, 1040, 257), (257, 96, 300), (301, 1001, 140), (512, 4096, 256)]


@pytest.mark.parametrize("m,k,n", I8)
def test_forward_i8(dev, m, k, n):
    torch, bl = dev
    bias = (m + n) % 2 == 1
    _say(f"forward_i8 M={m} K={k} N={n} bias={bias}")
    rng = np.random.default_rng([10, m, k, n])
    x, w = _f32(rng.standard_normal((m, k))), _f32(rng.standard_normal((n, k)) * 0.02)
    b = _f32(rng.standard_normal(n)) if bias else None
    xq_p, beta_p = plain.absmax(x)
    wq_p, gamma_p = plain.absmax(w)
    w_q, gamma = bl.bitlinear_quantize_weights_i8(_t(torch, w))
    assert np.array_equal(_np(w_q), wq_p) and np.array_equal(_bits(_np(gamma)), _bits(gamma_p))
    x_q, beta = _t(torch, xq_p), _t(torch, beta_p)
    y, acc = bl.bitlinear_forward_i8(x_q, beta, w_q, gamma, bias=_t(torch, b), acc=True)
    y2 = bl.bitlinear_forward_i8(x_q, beta, w_q, gamma, bias=_t(torch, b))
    ref = plain.int_product(xq_p, wq_p)
    assert np.array_equal(_np(acc), ref)
    f = np.float32
    yr = (ref.astype(f) * (beta_p / f(127))[:, None]) * (gamma_p / f(127))
    yr = yr if b is None else yr + b
    assert yr.dtype == np.float32 and np.array_equal(_np(y), yr)
    assert torch.equal(y, y2)


# (M, N): 36, 144 and 288 tiles of 64 x 256, the last of a row and of a column partial
@pytest.mark.parametrize("m,n", [(515, 901), (1089, 2017), (1473, 2950)])
@pytest.mark.parametrize("k", [1, 15, 16, 127, 128, 129, 130, 132, 260, 384, 400, 1001])
def test_forward_i8_many_tiles(dev, m, n, k):
    """K below, at and past the steps of 128, in rows on 16-byte and dword boundaries and off them."""
    torch, bl = dev
    _say(f"forward_i8 many tiles M={m} K={k} N={n}")
    rng = np.random.default_rng([12, m, k, n])
    xq = rng.integers(-127, 128, (m, k)).astype(np.int8)
    wq = rng.integers(-127, 128, (n, k)).astype(np.int8)
    beta, gamma = _f32(rng.random(m) + 0.5), _f32(rng.random(n) + 0.5)
    b = _f32(rng.standard_normal(n)) if k % 2 else None
    out = torch.full((m + 2, n), 3.0, device="cuda")
    _, acc = bl.bitlinear_forward_i8(_t(torch, xq), _t(torch, beta), _t(torch, wq), _t(torch, gamma), bias=_t(torch, b),
                                     y=out[1:m + 1], acc=True)
    ref = (xq.astype(np.float64) @ wq.astype(np.float64).T).astype(np.int32)     # exact: below 2^53
    assert np.array_equal(_np(acc), ref)
    f = np.float32
    yr = (ref.astype(f) * (beta / f(127))[:, None]) * (gamma / f(127))[None]
    assert np.array_equal(_np(out[1:m + 1]), yr if b is None else yr + b)
    assert bool((out[0] == 3).all()) and bool((out[m + 1] == 3).all())


def test_forward_i8_largest_sums(dev):
    """Codes of +-127 at the largest K: sums at the end of int32, on every path."""
    torch, bl = dev
    k = 133144
    for m, n in [(1, 5), (20, 33), (70, 40)]:
        _say(f"forward_i8 largest sums M={m} N={n}")
        x_q = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
        w_q = torch.full((n, k), -127, dtype=torch.int8, device="cuda")
        w_q[1::2] = 127
        one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
        _, acc = bl.bitlinear_forward_i8(x_q, one_m, w_q, one_n, acc=True)
        want = np.where(np.arange(n) % 2 == 1, 127 * 127 * k, -127 * 127 * k)
        assert np.array_equal(_np(acc), np.broadcast_to(want, (m, n)))


def test_forward_i8_unaligned_views(dev):
    torch, bl = dev
    rng = np.random.default_rng(11)
    for m, k, n in [(1, 128, 30), (20, 512, 33), (150, 256, 70)]:
        _say(f"forward_i8 unaligned M={m} K={k} N={n}")
        xq = rng.integers(-127, 128, (m, k)).astype(np.int8)
        wq = rng.integers(-127, 128, (n, k)).astype(np.int8)

        def off(a, s):
            t = _t(torch, a)
            v = torch.empty(t.numel() + s, dtype=t.dtype, device="cuda")[s:].view(t.shape)
            v.copy_(t)
            return v

        y = torch.full((m * n + 64,), 3.0, device="cuda")
        one = lambda q: torch.ones(q + 1, device="cuda")[1:]
        bl.bitlinear_forward_i8(off(xq, 1), one(m), off(wq, 5), one(n), y=y[1:1 + m * n].view(m, n))
        f = np.float32
        s = f(1) / f(127)
        ref = plain.int_product(xq, wq).astype(f) * s * s
        yn = _np(y)
        assert np.array_equal(yn[1:1 + m * n].reshape(m, n), ref)
        assert yn[0] == 3.0 and np.all(yn[1 + m * n:] == 3.0)


# ------------------------------------------------------------------- the operators together
def _step(torch, bl, s):
    """One training step of the block with a ternary down projection, through given buffers."""
    bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], h=s["h"], g=s["g"], u=s["u"],
                               x_q=s["x_q"], beta=s["beta"])
    bl.bitlinear_quantize_act(s["h"], s["h_q"], s["hbeta"])
    bl.bitlinear_forward(s["h_q"], s["hbeta"], s["Wd"], s["ad"], y=s["y"])
    bl.bitlinear_backward(s["dy"], s["h_q"], s["hbeta"], s["Wd"], s["ad"], dx=s["dh"], dW=s["dWd"], workspace=s["ws1"])
    bl.bitlinear_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"],
                                dx=s["dx"], dWg=s["dWg"], dWu=s["dWu"], workspace=s["ws2"])
    return [s[q] for q in ("h", "y", "dh", "dWd", "dx", "dWg", "dWu")]


def _step_state(torch, bl, m, k, f, seed):
    rng = np.random.default_rng(seed)
    e = lambda *sh, dt=torch.float32: torch.empty(sh, dtype=dt, device="cuda")
    s = dict(x=_t(torch, _f32(rng.standard_normal((m, k)))), dy=_t(torch, _f32(rng.standard_normal((m, k)) / m)),
             act=bl.BITLINEAR_ACT_SILU, h=e(m, f), g=e(m, f), u=e(m, f), x_q=e(m, k, dt=torch.int8), beta=e(m),
             h_q=e(m, f, dt=torch.int8), hbeta=e(m), y=e(m, k), dh=e(m, f), dWd=e(k, f), dx=e(m, k), dWg=e(f, k), dWu=e(f, k),
             ws1=e(bl.bitlinear_backward_workspace_size(m, f, k), dt=torch.uint8),
             ws2=e(bl.bitlinear_gated_backward_workspace_size(m, k, f), dt=torch.uint8))
    for w, al, n, c in (("Wg", "ag", f, k), ("Wu", "au", f, k), ("Wd", "ad", k, f)):
        s[w], s[al] = bl.bitlinear_quantize_weights(_t(torch, _f32(rng.standard_normal((n, c)) * 0.02)))
    return s


@pytest.mark.parametrize("m,k,f", [(1, 128, 192), (40, 256, 344), (130, 192, 260)])
def test_training_step(dev, m, k, f):
    """Forward and backward of the whole block against the plain forms chained the same way."""
    torch, bl = dev
    _say(f"training step M={m} K={k} F={f}")
    s = _step_state(torch, bl, m, k, f, [12, m])
    out = dict(zip(("h", "y", "dh", "dWd", "dx", "dWg", "dWu"), (_np(t) for t in _step(torch, bl, s))))
    unpack = lambda p: (((_np(p)[:, :, None] >> np.array([0, 2, 4, 6])) & 3).astype(np.int8) - 1).reshape(p.shape[0], -1)
    wg, wu, wd = unpack(s["Wg"]), unpack(s["Wu"]), unpack(s["Wd"])
    ag, au, ad = (float(s[q]) for q in ("ag", "au", "ad"))
    hq, hb = plain.absmax(out["h"])
    assert np.array_equal(out["y"], plain.project(hq, hb, wd, np.float32(ad), None))
    want, terms = plain.linear_gradients(_np(s["dy"]), hq, hb, wd, ad)
    for name, w, t, n in (("dh", want[0], terms[0], k), ("dWd", want[1], terms[1], m)):
        assert np.all(np.abs(out[name] - w) <= plain.gradient_tolerance(t, n)), name
    xq, xb = plain.absmax(_np(s["x"]))
    want, terms = plain.gated_gradients(out["dh"], _np(s["g"]), _np(s["u"]), xq, xb, wg, ag, wu, au, "silu")
    d0 = 24 * U * np.abs(out["dh"].astype(np.float64) * _np(s["u"]))      # a' near its zero
    slack = [d0 @ np.abs(wg) * ag, d0.T @ (np.abs(xq) * xb[:, None].astype(np.float64) / 127), 0]
    for name, w, t, n, sl in zip(("dx", "dWg", "dWu"), want, terms, (2 * f, m, m), slack):
        assert np.all(np.abs(out[name] - w) <= plain.gradient_tolerance(t, n) + sl), name


def test_training_step_in_a_graph_and_on_streams(dev):
    """The step captured and replayed, with eager work between the replays, and two steps at once on
    two streams with a workspace each: the eager bits every time."""
    torch, bl = dev
    a = _step_state(torch, bl, 70, 256, 344, 21)
    b = _step_state(torch, bl, 33, 192, 260, 22)
    want_a = [t.clone() for t in _step(torch, bl, a)]
    want_b = [t.clone() for t in _step(torch, bl, b)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(torch, bl, a)
    for rep in range(4):
        _say(f"replay {rep}")
        for t in outs + [a["ws1"], a["ws2"]]:
            t.fill_(77 if t.dtype == torch.uint8 else float("nan"))
        _step(torch, bl, b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want_a))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        for t in [a[q] for q in ("h", "y", "dh", "dWd", "dx", "dWg", "dWu")] + [b[q] for q in ("h", "dx", "dWg")]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            oa = _step(torch, bl, a)
        with torch.cuda.stream(s2):
            ob = _step(torch, bl, b)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(oa, want_a))
        assert all(torch.equal(o, w) for o, w in zip(ob, want_b))


def test_served_block_with_an_8bit_down_projection(dev):
    """Gated block, then quantize_act and the W8A8 product: one token and a small batch, each row's
    result the same whatever batch it came in."""
    torch, bl = dev
    rng = np.random.default_rng(30)
    k, f = 256, 344
    st = _step_state(torch, bl, 20, k, f, 31)
    wq, gamma = bl.bitlinear_quantize_weights_i8(_t(torch, _f32(rng.standard_normal((k, f)) * 0.02)))

    def serve(x):
        h = bl.bitlinear_gated_forward(x, st["Wg"], st["ag"], st["Wu"], st["au"], bl.BITLINEAR_ACT_SILU)
        h_q, hb = bl.bitlinear_quantize_act(h)
        return bl.bitlinear_forward_i8(h_q, hb, wq, gamma)

    y = serve(st["x"])
    hq, hb = plain.absmax(_np(bl.bitlinear_gated_forward(st["x"], st["Wg"], st["ag"], st["Wu"], st["au"], bl.BITLINEAR_ACT_SILU)))
    fl = np.float32
    ref = plain.int_product(hq, _np(wq)).astype(fl) * (hb / fl(127))[:, None] * (_np(gamma) / fl(127))
    assert np.array_equal(_np(y), ref)
    for i in (0, 7, 19):
        assert torch.equal(serve(st["x"][i:i + 1].contiguous())[0], y[i])


def test_explicit_stream_and_the_bindings_own_buffers(dev):
    """Calls on a given stream that is not the current one, codes, scales and workspace left to the
    binding, while the current stream allocates and overwrites memory all the time."""
    torch, bl = dev
    s = _step_state(torch, bl, 96, 512, 700, 41)
    want = [t.clone() for t in _step(torch, bl, s)]
    h_want, dx_want, dwd_want = want[0], want[4], want[3]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(5):
        h = bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], stream=side)
        dx, dwg, dwu, _, _ = bl.bitlinear_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["Wg"], s["ag"],
                                                         s["Wu"], s["au"], s["act"], stream=side)
        _, dwd, _ = bl.bitlinear_backward(s["dy"], s["h_q"], s["hbeta"], s["Wd"], s["ad"], stream=side)
        for _ in range(8):
            torch.full((3 << 20,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(h, h_want) and torch.equal(dx, dx_want) and torch.equal(dwd, dwd_want)
        assert torch.equal(dwg, want[5]) and torch.equal(dwu, want[6])


def test_arguments_are_checked(dev):
    """Wrong dtypes, shapes, layouts and buffers are refused in Python, before any launch."""
    torch, bl = dev
    s = _step_state(torch, bl, 4, 64, 32, 42)
    fwd = lambda **kw: bl.bitlinear_gated_forward(**{**dict(x=s["x"], Wg_packed=s["Wg"], alpha_g=s["ag"], Wu_packed=s["Wu"],
                                                            alpha_u=s["au"], act=s["act"]), **kw})
    for kw in (dict(x=s["x"].double()), dict(x=s["x"].t()), dict(x=s["x"][0]), dict(Wu_packed=s["Wd"]), dict(h=s["y"]),
               dict(alpha_g=s["beta"]), dict(bias_g=s["beta"]), dict(x_q=s["h_q"]), dict(x=s["x"].cpu()),
               dict(Wg_packed=s["Wg"].cpu())):
        with pytest.raises(ValueError):
            fwd(**kw)
    for kw in (dict(act=0), dict(g=s["g"])):
        with pytest.raises(bl.BitLinearError):
            fwd(**kw)
    bwd = lambda **kw: bl.bitlinear_backward(**{**dict(dy=s["dy"], x_q=s["h_q"], beta=s["hbeta"], W_packed=s["Wd"],
                                                       alpha=s["ad"]), **kw})
    for kw in (dict(x_q=s["x_q"]), dict(dx=s["dx"]), dict(dW=s["dWg"]), dict(dbias=s["hbeta"]), dict(beta=s["ad"]),
               dict(workspace=s["y"]), dict(dy=s["dy"].to(torch.bfloat16))):
        with pytest.raises(ValueError):
            bwd(**kw)
    with pytest.raises(bl.BitLinearError):
        bwd(workspace=s["ws1"][:256])
    i8 = dict(x_q=s["x_q"], beta=s["beta"], W_q=s["x_q"], gamma=s["beta"])
    for kw in (dict(W_q=s["h_q"]), dict(gamma=s["ad"]), dict(y=s["dy"]), dict(acc=s["dy"]), dict(bias=s["ad"])):
        with pytest.raises(ValueError):
            bl.bitlinear_forward_i8(**{**i8, **kw})


def test_outputs_past_32_bit_offsets(dev):
    """Outputs and gradients of more than 2^31 elements: the last rows equal those of a small call, the
    first ones too, and dW over all the tokens agrees with a 64-bit sum."""
    torch, bl = dev
    rng = np.random.default_rng(50)
    m, k, f = 196000, 64, 11008
    _say(f"gated_forward M={m} K={k} F={f}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(50)
    x = torch.randn(m, k, device="cuda", generator=gen)
    wg, wu = (_t(torch, plain.pack(plain.ternary(rng, f, k))) for _ in range(2))
    al = _t(torch, _f32([0.05]))
    h = bl.bitlinear_gated_forward(x, wg, al, wu, al, bl.BITLINEAR_ACT_SILU)
    assert h.numel() > 1 << 31
    for rows in (slice(0, 5), slice(m - 5, m)):
        assert torch.equal(h[rows], bl.bitlinear_gated_forward(x[rows].contiguous(), wg, al, wu, al, bl.BITLINEAR_ACT_SILU))
    _say("forward_i8")
    x_q, beta = bl.bitlinear_quantize_act(x)
    w_q, gamma = bl.bitlinear_quantize_weights_i8(torch.randn(f, k, device="cuda", generator=gen))
    y = bl.bitlinear_forward_i8(x_q, beta, w_q, gamma, y=h)
    for rows in (slice(0, 5), slice(m - 5, m)):
        assert torch.equal(y[rows], bl.bitlinear_forward_i8(x_q[rows].contiguous(), beta[rows].contiguous(), w_q, gamma))
    _say("backward")
    dx, dw, _ = bl.bitlinear_backward(y, x_q, beta, wg, al)
    w = (((_np(wg)[:, :, None] >> np.array([0, 2, 4, 6])) & 3).astype(np.int8) - 1).reshape(f, -1)
    for rows in (slice(0, 3), slice(m - 3, m)):
        want, terms = plain.linear_gradients(_np(y[rows]), _np(x_q[rows]), _np(beta[rows]), w, float(al[0]))
        assert np.all(np.abs(_np(dx[rows]) - want[0]) <= plain.gradient_tolerance(terms[0], f))
    xd = x_q.double() * (beta.double() / 127)[:, None]
    for n in (0, f - 1):
        d = y[:, n].double()
        want, terms = _np(d @ xd), np.sqrt(_np((d * d) @ (xd * xd)))
        # y follows x: the sums are a hundred root sums of squares
        assert np.all(np.abs(_np(dw[n]) - want) <= plain.gradient_tolerance(terms, m, want))
