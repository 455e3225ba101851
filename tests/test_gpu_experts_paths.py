"""GPU tests of the products grouped by expert, kernel by kernel: each case names the kernel that it is for, and
the call is seen to launch it."""
import numpy as np
import pytest

import experts_plain
import ffn_plain as plain
from graph_kernels import kernels
from test_gpu_experts import F32, _bits, _code, _np, _off, _pack, _say, _t, _weights, dev  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu
ACT_NUMBER = {"gelu": 1, "silu": 2, "relu2": 3}


def _counts(rng, m, e):
    """Rows of each of e experts, m in all: uneven, some without."""
    share = rng.random(e) ** 2 + 0.05
    share[:: 7] = 0 if e > 7 else share[:: 7]
    counts = np.floor(m * share / share.sum()).astype(np.int64)
    counts[-1] += m - counts.sum()
    return counts


def _case(rng, m, e, k, gone):
    """offsets of m rows, of which the last two are of no expert; the rows' tokens, a part `gone` of them not there; x_q, beta."""
    counts = _counts(rng, m - 2, e)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    t = m // 2 + 1
    rows = rng.integers(0, t, m).astype(np.int64)
    missing = rng.random(m) < gone
    rows[missing] = rng.choice(np.array([-1, t, 1 << 40, -(1 << 62)]), int(missing.sum()))
    x_q, beta = rng.integers(-127, 128, (t, k)).astype(np.int8), rng.uniform(0.5, 4, t).astype(F32)
    return offsets, rows, x_q, beta, t


def _check_forward(torch, bl, m, e, k, n, bias, gone, names):
    """bitlinear_grouped_forward bit for bit, on aligned tensors and on views that are not; `names`: the kernels of both."""
    rng = np.random.default_rng([41, m, e, k, n])
    offsets, rows, x_q, beta, t = _case(rng, m, e, k, gone)
    w, alpha, b = _weights(rng, e, n, k, bias)
    if bias:
        b[:, ::7] = -0.0
    want = experts_plain.forward(*experts_plain.tokens(x_q, beta, rows, m), offsets, w, alpha, b, np.full((m, n), 7, F32))
    args = [x_q, beta, offsets, _pack(w), alpha]
    for name, off in zip(names, (0, 1)):
        _say(f"grouped_forward M={m} E={e} K={k} N={n} bias={bias} views={off}: {name}")
        buf = torch.full((m * n + 8,), 7.0, device="cuda")
        y = buf[off:off + m * n].view(m, n)
        dev_args = [_off(torch, a, off) for a in args]
        kw = dict(rows=_off(torch, rows, off), bias=_off(torch, b, off), y=y)
        call = lambda: bl.bitlinear_grouped_forward(*dev_args, **kw)  # noqa: B023
        assert kernels(torch, call) == [name]
        call()
        torch.cuda.synchronize()
        assert np.array_equal(_bits(_np(y)), _bits(want)), name
        assert bool((buf[:off] == 7).all()) and bool((buf[off + m * n:] == 7).all())


def _check_gated(torch, bl, m, e, k, f, act, bias, gone, names):
    """The same of bitlinear_grouped_gated_forward: g and u bit for bit, h within its roundings."""
    rng = np.random.default_rng([43, m, e, k, f])
    offsets, rows, _, _, t = _case(rng, m, e, k, gone)
    wg, ag, bg = _weights(rng, e, f, k, bias)
    wu, au, bu = _weights(rng, e, f, k, bias)
    x = rng.standard_normal((t, k)).astype(F32)
    xr, br = experts_plain.tokens(*plain.absmax(x), rows, m)
    seven = np.full((m, f), 7, F32)
    g_p = experts_plain.forward(xr, br, offsets, wg, ag, bg, seven)
    u_p = experts_plain.forward(xr, br, offsets, wu, au, bu, seven)
    live = slice(0, int(offsets[-1]))
    ref = plain.activation(g_p, act)[0] * u_p.astype(np.float64)
    # roundings of a(g): SiLU 7, GELU and squared ReLU 1, and the product's, to first order
    tol = 1.01 * {"silu": 8, "gelu": 2, "relu2": 2}[act] * plain.U * np.abs(ref) + 1e-37
    args, first = [x, offsets, _pack(wg), ag, _pack(wu), au], None
    for name, off in zip(names, (0, 1)):
        _say(f"grouped_gated_forward M={m} E={e} K={k} F={f} {act} bias={bias} views={off}: {name}")
        bufs = [torch.full((m * f + 8,), 7.0, device="cuda") for _ in range(3)]
        h, g, u = (v[off:off + m * f].view(m, f) for v in bufs)
        dev_args = [_off(torch, a, off) for a in args]
        kw = dict(rows=_off(torch, rows, off), bias_g=_off(torch, bg, off), bias_u=_off(torch, bu, off), h=h,
                  x_q=_off(torch, np.zeros((t, k), np.int8), off), beta=torch.empty(t, device="cuda"))
        call = lambda **more: bl.bitlinear_grouped_gated_forward(*dev_args, _code(bl, act), **kw, **more)  # noqa: B023
        assert kernels(torch, call)[1:] == [name]
        call(g=g, u=u)
        torch.cuda.synchronize()
        assert np.array_equal(_bits(_np(g)), _bits(g_p)) and np.array_equal(_bits(_np(u)), _bits(u_p)), name
        got = _np(h)
        assert np.all(np.abs(got - ref)[live] <= tol[live]) and np.all(got[live.stop:] == 7), name
        # a row without a token and without biases: zeros, none of them negative
        if not bias:
            assert not _bits(got)[live][~(rows >= 0)[live] | (rows >= t)[live]].any(), name
        first = got if first is None else first
        assert np.array_equal(_bits(got), _bits(first)), name
        for v in bufs:
            assert bool((v[:off] == 7).all()) and bool((v[off + m * f:] == 7).all())
        h.fill_(7)
        call()
        assert np.array_equal(_bits(_np(h)), _bits(first)), name


def _id(v):
    return f"M{v[0]}_E{v[1]}_K{v[2]}_N{v[3]}" if isinstance(v, tuple) else v[0] if isinstance(v, list) else str(v)


def _gemm(act, aligned, fm):
    return f"k_grouped_gemm<{act}, {int(aligned)}, {fm}>"


# M, experts, K, columns, and the kernels of aligned tensors and of views
GONE = [(42, 3, 256, 160, ["k_grouped_dec<0, 8>"] * 2), (300, 9, 320, 1000, ["k_grouped_dec<0, 4>"] * 2),
        (403, 3, 320, 3300, [_gemm(0, 1, 1), _gemm(0, 0, 1)]), (700, 5, 192, 3100, [_gemm(0, 1, 2), _gemm(0, 0, 2)])]


@pytest.mark.parametrize("m,e,k,n,names", GONE, ids=_id)
def test_rows_without_a_token_are_of_zeros(dev, m, e, k, n, names):  # noqa: F811
    """A row whose index is no token reads x_q = 0 and beta = 0: +0 in every column, not the sign of another
    token's sum."""
    torch, bl = dev
    for bias in (False, True):
        _check_forward(torch, bl, m, e, k, n, bias, 0.4, names)


GONE_GATED = [(42, 3, 256, 160, ["k_grouped_dec<1, 8>"] * 2), (300, 9, 320, 500, ["k_grouped_dec<1, 4>"] * 2),
              (403, 3, 320, 1700, [_gemm(2, 1, 1), _gemm(2, 0, 1)]), (700, 5, 192, 1550, [_gemm(2, 1, 2), _gemm(2, 0, 2)])]


@pytest.mark.parametrize("m,e,k,f,names", GONE_GATED, ids=_id)
def test_gated_rows_without_a_token_are_of_zeros(dev, m, e, k, f, names):  # noqa: F811
    torch, bl = dev
    for bias in (False, True):
        _check_gated(torch, bl, m, e, k, f, "silu", bias, 0.4, names)


# M, experts, K, columns of every height of the GEMM's tiles: no whole step of 128, one to seven, with and without a rest,
# rows of codes that are not whole pieces of 16 bytes
TILES_32 = [(1990, 100, 60, 1801), (1990, 100, 64, 1700), (1990, 100, 100, 1160), (1990, 100, 128, 930), (403, 3, 192, 4700),
            (403, 3, 256, 3801), (403, 3, 260, 3750), (403, 3, 384, 2950), (403, 3, 512, 2513), (403, 3, 576, 2400), (403, 3, 640, 2250),
            (403, 3, 768, 2111), (403, 3, 896, 1985), (403, 3, 960, 1953), (403, 3, 1028, 1900)]
TILES_64 = [(700, 5, 60, 7001), (700, 5, 64, 6600), (700, 5, 100, 4500), (700, 5, 128, 3700), (700, 5, 192, 3073), (700, 5, 256, 3100),
            (700, 5, 260, 3201), (700, 5, 384, 3100), (700, 5, 512, 3329), (700, 5, 576, 3100), (700, 5, 640, 3077), (700, 5, 768, 3100),
            (700, 5, 896, 3263), (700, 5, 960, 3100)]
TILES_128 = [(1500, 4, 4096, 6700), (1500, 4, 4160, 6657), (1500, 4, 4100, 6721), (1500, 4, 4224, 6801), (1500, 4, 4352, 6657)]


@pytest.mark.parametrize("fm,size", [(1, s) for s in TILES_32] + [(2, s) for s in TILES_64] + [(4, s) for s in TILES_128], ids=_id)
def test_tiles(dev, fm, size):  # noqa: F811
    torch, bl = dev
    m, e, k, n = size
    _check_forward(torch, bl, m, e, k, n, k % 128 != 0, 0.05, [_gemm(0, k % 64 == 0, fm), _gemm(0, 0, fm)])


GATED_32 = [(1990, 100, 64, 850), (1990, 100, 100, 577), (1990, 100, 128, 470), (403, 3, 192, 2350), (403, 3, 256, 1900),
            (403, 3, 260, 1901), (403, 3, 384, 1500), (403, 3, 576, 1200), (403, 3, 896, 1001)]
GATED_64 = [(700, 5, 64, 3300), (700, 5, 128, 1900), (700, 5, 192, 1537), (700, 5, 256, 1600), (700, 5, 260, 1577), (700, 5, 384, 1555),
            (700, 5, 512, 1600), (700, 5, 576, 1537), (700, 5, 960, 1600)]
GATED_128 = [(1500, 4, 4096, 3400), (1500, 4, 4160, 3329), (1500, 4, 4100, 3401)]


@pytest.mark.parametrize("fm,size,act", [(fm, s, act) for fm, sizes in ((1, GATED_32), (2, GATED_64), (4, GATED_128))
                                         for i, s in enumerate(sizes) for act in (["silu", "gelu", "relu2"][(i + fm) % 3:][:1] if fm != 4
                                                                                  else ["silu", "gelu", "relu2"])], ids=_id)
def test_gated_tiles(dev, fm, size, act):  # noqa: F811
    """Every height with every activation; of 128 rows every activation at every size."""
    torch, bl = dev
    m, e, k, f = size
    number = ACT_NUMBER[act]
    _check_gated(torch, bl, m, e, k, f, act, f % 2 == 1, 0.05, [_gemm(number, k % 64 == 0, fm), _gemm(number, 0, fm)])


def test_tiles_of_tokens_past_2_gib(dev):  # noqa: F811
    """Tokens' codes between 2^31 and 2^32 bytes: the offsets of the aligned tiles are unsigned."""
    torch, bl = dev
    t, k, m, e, n = 125000, 32768, 900, 2, 1088
    gen = torch.Generator(device="cuda")
    gen.manual_seed(47)
    x_q = torch.zeros(t, k, dtype=torch.int8, device="cuda")
    rows = torch.randint(0, t, (m,), device="cuda", generator=gen)
    rows[:4] = torch.tensor([t - 1, 65535, 65536, 0], device="cuda")
    x_q[rows] = torch.randint(-127, 128, (m, k), device="cuda", generator=gen).to(torch.int8)
    beta = torch.rand(t, device="cuda", generator=gen) + 0.5
    w = torch.randint(0, 256, (e, n, k // 4), device="cuda", generator=gen).to(torch.uint8)
    w &= ~(w >> 1) | 0xAA                                           # no code of three
    alpha, offsets = torch.tensor([0.5, 0.25], device="cuda"), torch.tensor([0, 333, m], dtype=torch.int64, device="cuda")
    _say(f"grouped_forward of {t * k} bytes of tokens")
    call = lambda: bl.bitlinear_grouped_forward(x_q, beta, offsets, w, alpha, rows=rows, y=y)
    y = torch.empty(m, n, device="cuda")
    assert kernels(torch, call) == [_gemm(0, 1, 1)]
    call()
    shifts = torch.tensor([0, 2, 4, 6], device="cuda", dtype=torch.uint8)
    for i, j, g in ((0, 333, 0), (333, m, 1)):
        codes = ((w[g][:, :, None] >> shifts) & 3).reshape(n, k).double() - 1
        acc = (x_q[rows[i:j]].double() @ codes.t().contiguous()).float()           # exact: below 2^53
        s = (alpha[g].double() * beta[rows[i:j]].double() / 127.0).float()
        assert torch.equal(y[i:j], acc * s[:, None])


@pytest.mark.parametrize("m,e,k,n,name", [(1990, 100, 256, 600, _gemm(0, 1, 1)), (700, 5, 192, 3100, _gemm(0, 1, 2)),
                                          (1500, 4, 4096, 6657, _gemm(0, 1, 4))], ids=str)
def test_offsets_that_decrease_make_no_more_tiles(dev, m, e, k, n, name):  # noqa: F811
    """Groups that share rows make more tiles than were launched.  The tiles and the gradients of long groups stop at
    those that were: outputs are unspecified, what lies around them is not touched, and the next call is right."""
    torch, bl = dev
    rng = np.random.default_rng([53, m])
    bad = np.where(np.arange(e + 1) % 2 == 0, 0, m).astype(np.int64)
    offsets, rows, x_q, beta, t = _case(rng, m, e, k, 0.0)
    w, alpha, _ = _weights(rng, e, n, k, False)
    dy = rng.standard_normal((m, n)).astype(F32)
    xt, bt, wt, at, rt, dyt = (_t(torch, a) for a in (x_q, beta, _pack(w), alpha, rows, dy))

    def between(*shape):
        size = int(np.prod(shape))
        buf = torch.full((size + 512,), 7.0, device="cuda")
        return buf, buf[256:256 + size].view(shape)

    bufs, (y, dx, dw, db) = zip(*[between(*s) for s in ((m, n), (m, k), (e, n, k), (e, n))])
    ws = torch.empty(bl.bitlinear_grouped_backward_workspace_size(m, k, n, e), dtype=torch.uint8, device="cuda")
    for off in (bad, offsets):
        ot = _t(torch, off)
        forward = lambda: bl.bitlinear_grouped_forward(xt, bt, ot, wt, at, rows=rt, y=y)  # noqa: B023
        assert kernels(torch, forward) == [name]
        forward()
        if m > 32 * e:
            backward = lambda: bl.bitlinear_grouped_backward(dyt, xt, bt, ot, wt, at, rows=rt, dx=dx, dW=dw, dbias=db,  # noqa: B023
                                                             workspace=ws)
            assert kernels(torch, backward)[0] == "k_grouped_gradients"
            backward()
        torch.cuda.synchronize()
        for b in bufs:
            assert bool((b[:256] == 7).all()) and bool((b[-256:] == 7).all())
    want = experts_plain.forward(*experts_plain.tokens(x_q, beta, rows, m), offsets, w, alpha, None, np.zeros((m, n), F32))
    live = int(offsets[-1])
    assert np.array_equal(_bits(_np(y))[:live], _bits(want)[:live])
