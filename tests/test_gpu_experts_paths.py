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


def _gemm(act, aligned, fm):
    return f"k_grouped_gemm<{act}, {int(aligned)}, {fm}>"


# M, experts, K, columns, and the kernels of aligned tensors and of views
GONE = [(42, 3, 256, 160, ["k_grouped_dec<0, 8>"] * 2), (300, 9, 320, 1000, ["k_grouped_dec<0, 4>"] * 2),
        (403, 3, 320, 3300, [_gemm(0, 1, 1), _gemm(0, 0, 1)]), (700, 5, 192, 3100, [_gemm(0, 1, 2), _gemm(0, 0, 2)])]


@pytest.mark.parametrize("m,e,k,n,names", GONE, ids=lambda v: v[0] if isinstance(v, list) else str(v))
def test_rows_without_a_token_are_of_zeros(dev, m, e, k, n, names):  # noqa: F811
    """A row whose index is no token reads x_q = 0 and beta = 0: +0 in every column, not the sign of another
    token's sum."""
    torch, bl = dev
    for bias in (False, True):
        _check_forward(torch, bl, m, e, k, n, bias, 0.4, names)


GONE_GATED = [(42, 3, 256, 160, ["k_grouped_dec<1, 8>"] * 2), (300, 9, 320, 500, ["k_grouped_dec<1, 4>"] * 2),
              (403, 3, 320, 1700, [_gemm(2, 1, 1), _gemm(2, 0, 1)]), (700, 5, 192, 1550, [_gemm(2, 1, 2), _gemm(2, 0, 2)])]


@pytest.mark.parametrize("m,e,k,f,names", GONE_GATED, ids=lambda v: v[0] if isinstance(v, list) else str(v))
def test_gated_rows_without_a_token_are_of_zeros(dev, m, e, k, f, names):  # noqa: F811
    torch, bl = dev
    for bias in (False, True):
        _check_gated(torch, bl, m, e, k, f, "silu", bias, 0.4, names)
