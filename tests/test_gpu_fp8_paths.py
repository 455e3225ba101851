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


WIDE = [(1, 1032, 200, "k_fp8_dec", 1), (20, 520, 100, "k_fp8_dec", 2), (64, 256, 64, "k_fp8_dec", 4), (140, 384, 300, "k_fp8_gemm", 1, 1),
        (200, 520, 8400, "k_fp8_gemm", 1, 2), (640, 648, 8200, "k_fp8_gemm", 2, 2)]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_small_products_beside_large_ones(dev, case):  # noqa: F811
    """Products 2^14 to 2^18 times smaller than those beside them, which cancel: the small ones are the sum, exactly.
    (The e4m3 matrix instructions lose what lies below 2^-13 of the largest of eight products.)"""
    torch, bl = dev
    m, k, n, kind, *numbers = case
    _check(torch, bl, m, k, n, fp8_plain.wide(np.random.default_rng([3, m, k, n]), m, k, n), _names(kind, k, *numbers))
