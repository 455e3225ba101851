"""GPU tests of the fp8 product, kernel by kernel, with data whose sums are exact: each case names the kernels of
16-byte aligned rows, of rows on dwords and of rows anywhere, and the calls are seen to launch them."""
import numpy as np
import pytest

import fp8_plain
from graph_kernels import kernels
from test_gpu_fp8 import _off, _t, dev  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu


def _names(kind, k, *numbers):
    """Of views 0, 4 and 1 or 3 bytes off, by the rows' length; the largest tile has no form for bytes."""
    rows = [16 if k % 16 == 0 else 4 if k % 4 == 0 else 1, 4 if k % 4 == 0 else 1, 1]
    if kind == "k_fp8_gemm" and numbers == (2, 2):
        rows = [max(r, 4) for r in rows]
    return [f"{kind}<{', '.join(map(str, (r, *numbers)))}>" for r in rows]


def _check(torch, bl, m, k, n, data, names):
    x, xs, w, ws, want = data
    want = want.astype(np.float32)
    x_q, w_q = (_t(torch, a).to(torch.float8_e4m3fn).view(torch.uint8) for a in (x, w))
    e4m3 = torch.float8_e4m3fn
    for name, a, b in zip(names, (0, 4, 3), (0, 4, 1)):
        print(f"forward_fp8 M={m} K={k} N={n} views {a} {b}: {name}", flush=True)
        args = [_off(torch, x_q, a).view(e4m3), _off(torch, _t(torch, xs), b), _off(torch, w_q, b).view(e4m3), _off(torch, _t(torch, ws), a)]
        out = torch.full((m * n + 8,), 7.0, device="cuda")
        y = out[b:b + m * n].view(m, n)
        call = lambda: bl.bitlinear_forward_fp8(*args, y=y)  # noqa: B023
        assert kernels(torch, call) == [name]
        call()
        got = y.cpu().numpy()
        assert np.array_equal(got, want), (name, int(np.count_nonzero(got != want)))
        assert bool((out[:b] == 7).all()) and bool((out[b + m * n:] == 7).all())


# M, K, N and the kernel with its sizes
DEC = [(1, 1024, 300, 1), (3, 4097, 200, 1), (16, 2064, 130, 1), (17, 1300, 77, 2), (40, 1040, 150, 3), (64, 900, 140, 4), (100, 1153, 90, 4)]
# one to eight whole blocks of 128 in every tile, with and without a rest
TILES = [(140, 256 + 128 * i + r, 300 + i, 1, 1) for i, r in enumerate((0, 16, 4, 0, 1, 64, 0))] + \
        [(200, 128 + 128 * i + r, 8400 + i, 1, 2) for i, r in enumerate((16, 0, 4, 0, 64, 1, 0, 0))] + \
        [(640, 128 + 128 * i + r, 8200 + i, 2, 2) for i, r in enumerate((0, 0, 16, 0, 4, 0, 105, 0))] + [(1030, 1001, 4100, 2, 2)]


@pytest.mark.parametrize("m,k,n,mt", DEC)
def test_streaming_kernel(dev, m, k, n, mt):  # noqa: F811
    torch, bl = dev
    _check(torch, bl, m, k, n, fp8_plain.integers(np.random.default_rng([1, m, k, n]), m, k, n), _names("k_fp8_dec", k, mt))


@pytest.mark.parametrize("m,k,n,mi,fn", TILES)
def test_tiles(dev, m, k, n, mi, fn):  # noqa: F811
    torch, bl = dev
    _check(torch, bl, m, k, n, fp8_plain.integers(np.random.default_rng([2, m, k, n]), m, k, n), _names("k_fp8_gemm", k, mi, fn))


WIDE = [(1, 1032, 200, "k_fp8_dec", 1), (20, 520, 100, "k_fp8_dec", 2), (64, 256, 64, "k_fp8_dec", 4), (140, 384, 300, "k_fp8_gemm", 1, 1),
        (200, 520, 8400, "k_fp8_gemm", 1, 2), (640, 648, 8200, "k_fp8_gemm", 2, 2)]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_small_products_beside_large_ones(dev, case):  # noqa: F811
    """Products 2^14 to 2^18 times smaller than those beside them, which cancel: the small ones are the sum, exactly.
    (The e4m3 matrix instructions lose what lies below 2^-13 of the largest of eight products.)"""
    torch, bl = dev
    m, k, n, kind, *numbers = case
    _check(torch, bl, m, k, n, fp8_plain.wide(np.random.default_rng([3, m, k, n]), m, k, n), _names(kind, k, *numbers))
