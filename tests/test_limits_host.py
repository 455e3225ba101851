"""The limits of sizes that the header states, against what the library refuses; no call here gets as far as a launch."""
import random
import re

from test_abi_host import A, HEADER, bl  # noqa: F401  (fixture)


def _comment(name):
    """The comment above the first declaration of `name`."""
    src = open(HEADER).read()
    at = re.search(r"^\w[\w ]*\b" + name + r"\(", src, re.M).start()
    return re.sub(r"\s*\n \*\s*", " ", src[src.rindex("/*", 0, at):at])


def _power(text, what):
    m = re.search(re.escape(what) + r" <= 2\^(\d+)", text)
    assert m, f"the header states no limit of {what}"
    return 1 << int(m.group(1))


def test_fp8_limits(bl):  # noqa: F811
    shape = bl.BITLINEAR_ERR_SHAPE
    for name, call in (("bitlinear_quantize_act_fp8", bl.lib.bitlinear_quantize_act_fp8),
                       ("bitlinear_quantize_weights_fp8", bl.lib.bitlinear_quantize_weights_fp8)):
        most = _power(_comment("bitlinear_quantize_act_fp8"), "M K and N K")
        assert call(A, (1 << 26), most // (1 << 26) + 1, A, A, None) == shape, name
        assert call(A, most // (1 << 22) + 1, 1 << 22, A, A, None) == shape, name
    text = _comment("bitlinear_forward_fp8")
    most, outputs = _power(text, "M K and N K"), _power(text, "M N")
    f = bl.lib.bitlinear_forward_fp8
    assert f(A, A, 1, 1 << 22, A, A, most // (1 << 22) + 1, None, A, None) == shape
    assert f(A, A, most // (1 << 22) + 1, 1 << 22, A, A, 1, None, A, None) == shape
    assert f(A, A, 1 << 20, 8, A, A, outputs // (1 << 20) + 1, None, A, None) == shape


def _padded(v, to):
    return -(-v // to) * to


def test_grouped_limits(bl):  # noqa: F811
    """What the header says always fits has a workspace size, and what it rules out has none."""
    text = _comment("bitlinear_grouped_forward")
    back = _comment("bitlinear_grouped_backward_workspace_size")
    mn, en, enk = _power(text, "M N"), _power(text, "min(E, M) N"), _power(text, "E N K")
    b_enk, b_en, b_ek, b_mk = (_power(back, w) for w in ("E N K", "E N", "E K", "M K"))
    tk = _power(text, "T K and T N")
    rng = random.Random(5)
    fits = 0
    for _ in range(20000):
        m, e, n = (int(2 ** rng.uniform(0, b)) for b in (24, 12, 20))
        k = 4 * int(2 ** rng.uniform(0, 22))
        k = min(k, bl.BITLINEAR_MAX_K)
        np_, kp = _padded(n, 128), _padded(k, 256)
        if max(m * k, m * n) > tk or m * np_ > mn or min(e, m) * np_ > en or e * n * k > enk:
            continue
        if e * np_ * kp > b_enk or e * np_ > b_en or e * kp > b_ek or m * kp > b_mk:
            continue
        fits += 1
        for size in (bl.bitlinear_grouped_backward_workspace_size, bl.bitlinear_grouped_gated_backward_workspace_size):
            assert size(m, k, n, e) > 0, (m, k, n, e)
    assert fits > 5000
    # and beyond: refused, with nothing launched
    for m, k, n, e in ((64, 16384, 16384, 513), (1 << 24, 32768, 128, 1), (1 << 24, 1024, 4096, 8), (64, 64, 1 << 20, 4096)):
        assert bl.bitlinear_grouped_backward_workspace_size(m, k, n, e) == 0, (m, k, n, e)
        assert bl.lib.bitlinear_grouped_backward(A, m, n, A, A, 3, k, A, A, e, A, A, A, A, None, A, 1 << 62,
                                                 None) == bl.BITLINEAR_ERR_SHAPE
    f = bl.lib.bitlinear_grouped_forward
    for m, k, n, e in ((1 << 24, 64, 4097 * 2, 1), (4096, 4, 1 << 20, 4096), (8, 1 << 20, 1 << 20, 5)):
        assert f(A, A, 3, k, A, m, A, e, A, A, n, None, A, None) == bl.BITLINEAR_ERR_SHAPE, (m, k, n, e)
    assert f(A, A, tk // 64 + 1, 64, A, 6, A, 4, A, A, 8, None, A, None) == bl.BITLINEAR_ERR_SHAPE
    assert f(A, A, 1 << 31, 4, A, 6, A, 4, A, A, 8, None, A, None) == bl.BITLINEAR_ERR_SHAPE
