"""Refusals of the gated block, the gradients and the W8A8 product that need no GPU: every call is
invalid on purpose and is turned down on the host before anything is enqueued."""
import pytest

from test_abi_host import A, bl  # noqa: F401  (fixture)

B = 1 << 50


def _call(f, order, ok, **kw):
    d = dict(ok)
    d.update(kw)
    return f(*[d[k] for k in order])


GATED = ["x", "M", "K", "wg", "ag", "bg", "wu", "au", "bu", "F", "act", "h", "g", "u", "xq", "beta", "s"]


def test_gated_forward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_gated_forward
    ok = dict(x=A, M=2, K=64, wg=A, ag=A, bg=None, wu=A, au=A, bu=None, F=8, act=bl.BITLINEAR_ACT_SILU, h=A, g=None,
              u=None, xq=A, beta=A, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("x", "wg", "ag", "wu", "au", "h", "xq", "beta"):
        assert _call(f, GATED, ok, **{k: None}) == bad, k
    for k in ("M", "K", "F"):
        assert _call(f, GATED, ok, **{k: 0}) == bad and _call(f, GATED, ok, **{k: -4}) == bad
    assert _call(f, GATED, ok, g=A) == bad and _call(f, GATED, ok, u=A) == bad
    for act in (0, 4, -1):
        assert _call(f, GATED, ok, act=act) == bad
    for kw in (dict(K=66), dict(K=bl.BITLINEAR_MAX_K + 4), dict(M=1 << 31), dict(F=1 << 31), dict(M=1 << 30, F=1 << 30)):
        assert _call(f, GATED, ok, **kw) == bl.BITLINEAR_ERR_SHAPE, kw
    assert bl.lib.bitlinear_last_hip_error() == 0


BWD = ["dy", "M", "N", "xq", "beta", "K", "w", "al", "dx", "dw", "db", "ws", "bytes", "s"]


def test_backward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_backward
    ok = dict(dy=A, M=2, N=8, xq=A, beta=A, K=64, w=A, al=A, dx=A, dw=A, db=None, ws=A, bytes=B, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("dy", "xq", "beta", "w", "al"):
        assert _call(f, BWD, ok, **{k: None}) == bad, k
    for k in ("M", "K", "N"):
        assert _call(f, BWD, ok, **{k: 0}) == bad and _call(f, BWD, ok, **{k: -4}) == bad
    assert _call(f, BWD, ok, dx=None, dw=None) == bad
    for kw in (dict(K=62), dict(K=bl.BITLINEAR_MAX_K + 4), dict(M=(1 << 21) + 1), dict(N=(1 << 21) + 1), dict(M=1 << 21, N=1 << 21)):
        assert _call(f, BWD, ok, **kw) == bl.BITLINEAR_ERR_SHAPE, kw
    need = bl.bitlinear_backward_workspace_size(2, 64, 8)
    assert need > 0
    assert _call(f, BWD, ok, ws=None) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, BWD, ok, bytes=need - 1) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, BWD, ok, ws=A + 16) == bl.BITLINEAR_ERR_ALIGNMENT
    for size in ((0, 64, 8), (2, 66, 8), (2, 64, -1), ((1 << 21) + 1, 64, 8)):
        assert bl.bitlinear_backward_workspace_size(*size) == 0
        assert bl.bitlinear_gated_backward_workspace_size(*size) == 0


GBWD = ["dh", "g", "u", "M", "F", "xq", "beta", "K", "wg", "ag", "wu", "au", "act", "dx", "dwg", "dwu", "dbg", "dbu", "ws",
        "bytes", "s"]


def test_gated_backward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_gated_backward
    ok = dict(dh=A, g=A, u=A, M=2, F=8, xq=A, beta=A, K=64, wg=A, ag=A, wu=A, au=A, act=bl.BITLINEAR_ACT_GELU, dx=A, dwg=A,
              dwu=A, dbg=None, dbu=None, ws=A, bytes=B, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("dh", "g", "u", "xq", "beta", "wg", "ag", "wu", "au", "dwg", "dwu"):
        assert _call(f, GBWD, ok, **{k: None}) == bad, k
    for k in ("M", "K", "F"):
        assert _call(f, GBWD, ok, **{k: 0}) == bad
    assert _call(f, GBWD, ok, dx=None, dwg=None, dwu=None) == bad
    assert _call(f, GBWD, ok, act=0) == bad
    assert _call(f, GBWD, ok, K=66) == bl.BITLINEAR_ERR_SHAPE
    assert _call(f, GBWD, ok, F=(1 << 21) + 1) == bl.BITLINEAR_ERR_SHAPE
    need = bl.bitlinear_gated_backward_workspace_size(2, 64, 8)
    assert _call(f, GBWD, ok, ws=None) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, GBWD, ok, bytes=need - 1) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, GBWD, ok, ws=A + 128) == bl.BITLINEAR_ERR_ALIGNMENT


I8 = ["xq", "beta", "M", "K", "wq", "gamma", "N", "bias", "y", "acc", "s"]


def test_i8_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_forward_i8
    ok = dict(xq=A, beta=A, M=2, K=65, wq=A, gamma=A, N=8, bias=None, y=A, acc=None, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("xq", "beta", "wq", "gamma", "y"):
        assert _call(f, I8, ok, **{k: None}) == bad, k
    for k in ("M", "K", "N"):
        assert _call(f, I8, ok, **{k: 0}) == bad and _call(f, I8, ok, **{k: -1}) == bad
    for kw in (dict(K=133145), dict(M=1 << 31), dict(N=1 << 31), dict(M=1 << 30, N=1 << 30)):
        assert _call(f, I8, ok, **kw) == bl.BITLINEAR_ERR_SHAPE, kw
    q = bl.lib.bitlinear_quantize_weights_i8
    assert q(None, 4, 8, A, A, None) == bad and q(A, 4, 8, None, A, None) == bad and q(A, 4, 8, A, None, None) == bad
    assert q(A, 0, 8, A, A, None) == bad and q(A, 1 << 31, 1, A, A, None) == bl.BITLINEAR_ERR_SHAPE


def test_binding_refuses_host_tensors(bl):  # noqa: F811
    import torch
    m = torch.zeros(4, 8)
    for call in (lambda: bl.bitlinear_gated_forward(m, m, m, m, m, bl.BITLINEAR_ACT_SILU),
                 lambda: bl.bitlinear_backward(m, m, m, m, m),
                 lambda: bl.bitlinear_gated_backward(m, m, m, m, m, m, m, m, m, bl.BITLINEAR_ACT_SILU),
                 lambda: bl.bitlinear_quantize_weights_i8(m), lambda: bl.bitlinear_forward_i8(m, m, m, m)):
        with pytest.raises(ValueError):
            call()
