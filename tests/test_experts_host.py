"""Refusals of the grouped and the fp8 calls that need no GPU, and where the binding allocates for them."""
import pytest

import test_binding_streams as streams
from test_abi_host import A, bl  # noqa: F401  (fixture)

B = 1 << 50


def _call(f, order, ok, **kw):
    d = dict(ok)
    d.update(kw)
    return f(*[d[k] for k in order])


def _sizes(f, order, ok, n, bl):  # noqa: F811
    """What every grouped call refuses of its sizes; `n` is the name of its N."""
    bad, shape = bl.BITLINEAR_ERR_INVALID_ARG, bl.BITLINEAR_ERR_SHAPE
    for k in ("K", "E", n):
        assert _call(f, order, ok, **{k: 0}) == bad and _call(f, order, ok, **{k: -4}) == bad, k
    assert _call(f, order, ok, M=-1) == bad and _call(f, order, ok, T=-1) == bad and _call(f, order, ok, T=0) == bad
    assert _call(f, order, ok, rows=None) == shape                 # T != M
    for kw in (dict(K=62), dict(K=bl.BITLINEAR_MAX_K + 4), dict(M=(1 << 24) + 1), {n: (1 << 21) + 1}, dict(E=65536),
               dict(T=1 << 31), dict(K=1 << 20, **{n: 1 << 21}), dict(E=65535, K=65536, **{n: 65536})):
        assert _call(f, order, ok, **kw) == shape, kw


FWD = ["xq", "beta", "T", "K", "rows", "M", "off", "E", "w", "al", "N", "bias", "y", "s"]


def test_grouped_forward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_grouped_forward
    ok = dict(xq=A, beta=A, T=3, K=64, rows=A, M=6, off=A, E=4, w=A, al=A, N=8, bias=None, y=A, s=None)
    for k in ("xq", "beta", "off", "w", "al", "y"):
        assert _call(f, FWD, ok, **{k: None}) == bl.BITLINEAR_ERR_INVALID_ARG, k
    _sizes(f, FWD, ok, "N", bl)
    # no rows: nothing to do, and nothing to read but what a layer has in hand
    none = dict(ok, M=0, xq=None, beta=None, y=None, rows=None)
    assert _call(f, FWD, none) == bl.BITLINEAR_OK and _call(f, FWD, none, T=0) == bl.BITLINEAR_OK
    assert _call(f, FWD, none, w=None) == bl.BITLINEAR_ERR_INVALID_ARG
    assert bl.lib.bitlinear_last_hip_error() == 0


GATED = ["x", "T", "K", "rows", "M", "off", "E", "wg", "ag", "bg", "wu", "au", "bu", "F", "act", "h", "g", "u", "xq", "beta", "s"]


def test_grouped_gated_forward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_grouped_gated_forward
    ok = dict(x=A, T=3, K=64, rows=A, M=6, off=A, E=4, wg=A, ag=A, bg=None, wu=A, au=A, bu=None, F=8,
              act=bl.BITLINEAR_ACT_SILU, h=A, g=None, u=None, xq=A, beta=A, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("x", "off", "wg", "ag", "wu", "au", "h", "xq", "beta"):
        assert _call(f, GATED, ok, **{k: None}) == bad, k
    assert _call(f, GATED, ok, g=A) == bad and _call(f, GATED, ok, u=A) == bad
    for act in (0, 4, -1):
        assert _call(f, GATED, ok, act=act) == bad
    _sizes(f, GATED, ok, "F", bl)
    assert _call(f, GATED, ok, T=0, M=0, x=None, xq=None, beta=None, h=None, rows=None) == bl.BITLINEAR_OK


BWD = ["dy", "M", "N", "xq", "beta", "T", "K", "rows", "off", "E", "w", "al", "dx", "dw", "db", "ws", "bytes", "s"]


def test_grouped_backward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_grouped_backward
    ok = dict(dy=A, M=6, N=8, xq=A, beta=A, T=3, K=64, rows=A, off=A, E=4, w=A, al=A, dx=A, dw=A, db=None, ws=A, bytes=B, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("dy", "xq", "beta", "off", "w", "al"):
        assert _call(f, BWD, ok, **{k: None}) == bad, k
    assert _call(f, BWD, ok, dx=None, dw=None) == bad
    _sizes(f, BWD, ok, "N", bl)
    need = bl.bitlinear_grouped_backward_workspace_size(6, 64, 8, 4)
    assert need > 0
    assert _call(f, BWD, ok, ws=None) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, BWD, ok, bytes=need - 1) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, BWD, ok, ws=A + 16) == bl.BITLINEAR_ERR_ALIGNMENT
    for size in ((-1, 64, 8, 4), (6, 66, 8, 4), (6, 64, 0, 4), (6, 64, 8, 65536), ((1 << 24) + 1, 64, 8, 4)):
        assert bl.bitlinear_grouped_backward_workspace_size(*size) == 0
        assert bl.bitlinear_grouped_gated_backward_workspace_size(*size) == 0
    assert bl.bitlinear_grouped_backward_workspace_size(0, 64, 8, 4) > 0


GBWD = ["dh", "g", "u", "M", "F", "xq", "beta", "T", "K", "rows", "off", "E", "wg", "ag", "wu", "au", "act", "dx", "dwg", "dwu",
        "dbg", "dbu", "ws", "bytes", "s"]


def test_grouped_gated_backward_refusals(bl):  # noqa: F811
    f = bl.lib.bitlinear_grouped_gated_backward
    ok = dict(dh=A, g=A, u=A, M=6, F=8, xq=A, beta=A, T=3, K=64, rows=A, off=A, E=4, wg=A, ag=A, wu=A, au=A,
              act=bl.BITLINEAR_ACT_GELU, dx=A, dwg=A, dwu=A, dbg=None, dbu=None, ws=A, bytes=B, s=None)
    bad = bl.BITLINEAR_ERR_INVALID_ARG
    for k in ("dh", "g", "u", "xq", "beta", "off", "wg", "ag", "wu", "au", "dwg", "dwu"):
        assert _call(f, GBWD, ok, **{k: None}) == bad, k
    assert _call(f, GBWD, ok, dx=None, dwg=None, dwu=None) == bad
    assert _call(f, GBWD, ok, act=0) == bad
    _sizes(f, GBWD, ok, "F", bl)
    need = bl.bitlinear_grouped_gated_backward_workspace_size(6, 64, 8, 4)
    assert _call(f, GBWD, ok, ws=None) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, GBWD, ok, bytes=need - 1) == bl.BITLINEAR_ERR_WORKSPACE
    assert _call(f, GBWD, ok, ws=A + 128) == bl.BITLINEAR_ERR_ALIGNMENT


def test_fp8_refusals(bl):  # noqa: F811
    bad, shape = bl.BITLINEAR_ERR_INVALID_ARG, bl.BITLINEAR_ERR_SHAPE
    for q in (bl.lib.bitlinear_quantize_act_fp8, bl.lib.bitlinear_quantize_weights_fp8):
        for i in (0, 3, 4):
            args = [A, 4, 8, A, A, None]
            args[i] = None
            assert q(*args) == bad
        assert q(A, 0, 8, A, A, None) == bad and q(A, 4, -1, A, A, None) == bad
        assert q(A, 1 << 31, 1, A, A, None) == shape and q(A, 1, (1 << 24) + 1, A, A, None) == shape
        assert q(A, 1 << 20, 1 << 21, A, A, None) == shape
    order = ["xq", "xs", "M", "K", "wq", "ws", "N", "bias", "y", "s"]
    ok = dict(xq=A, xs=A, M=2, K=65, wq=A, ws=A, N=8, bias=None, y=A, s=None)
    f = bl.lib.bitlinear_forward_fp8
    for k in ("xq", "xs", "wq", "ws", "y"):
        assert _call(f, order, ok, **{k: None}) == bad, k
    for k in ("M", "K", "N"):
        assert _call(f, order, ok, **{k: 0}) == bad and _call(f, order, ok, **{k: -1}) == bad
    for kw in (dict(K=(1 << 24) + 1), dict(M=1 << 31), dict(N=1 << 31), dict(M=1 << 30, N=1 << 30), dict(M=1 << 25, K=1 << 16)):
        assert _call(f, order, ok, **kw) == shape, kw


def test_binding_refuses_host_tensors(bl):  # noqa: F811
    import torch
    m, w, v = torch.zeros(4, 8), torch.zeros(2, 8, 2), torch.zeros(3, dtype=torch.int64)
    act = bl.BITLINEAR_ACT_SILU
    for call in (lambda: bl.bitlinear_grouped_forward(m, m, v, w, m), lambda: bl.bitlinear_quantize_act_fp8(m),
                 lambda: bl.bitlinear_grouped_gated_forward(m, v, w, m, w, m, act),
                 lambda: bl.bitlinear_grouped_backward(m, m, m, v, w, m),
                 lambda: bl.bitlinear_grouped_gated_backward(m, m, m, m, m, v, w, m, w, m, act),
                 lambda: bl.bitlinear_quantize_weights_fp8(m), lambda: bl.bitlinear_forward_fp8(m, m, m, m)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------- what the binding allocates, and where
class _Torch(streams.Torch):
    def __init__(self):
        super().__init__()
        self.float8_e4m3fn, self.int64 = "float8_e4m3fn", "int64"


T, M, K, N, E = 3, 5, 128, 64, 2


def _calls(bl):  # noqa: F811
    t = streams.Tensor
    f = lambda *s: t(s, "float32")
    xq, rows, off, w, al = t((T, K), "int8"), t(M, "int64"), t(E + 1, "int64"), t((E, N, K // 4), "uint8"), f(E)
    act = bl.BITLINEAR_ACT_SILU
    return {
        "grouped_forward": lambda s: bl.bitlinear_grouped_forward(xq, f(T), off, w, al, rows=rows, stream=s),
        "grouped_gated_forward": lambda s: bl.bitlinear_grouped_gated_forward(f(T, K), off, w, al, w, al, act, rows=rows, stream=s),
        "grouped_backward": lambda s: bl.bitlinear_grouped_backward(f(M, N), xq, f(T), off, w, al, rows=rows, stream=s),
        "grouped_gated_backward": lambda s: bl.bitlinear_grouped_gated_backward(
            f(M, N), f(M, N), f(M, N), xq, f(T), off, w, al, w, al, act, rows=rows, stream=s),
        "quantize_act_fp8": lambda s: bl.bitlinear_quantize_act_fp8(f(T, K), stream=s),
        "quantize_weights_fp8": lambda s: bl.bitlinear_quantize_weights_fp8(f(N, K), stream=s),
        "forward_fp8": lambda s: bl.bitlinear_forward_fp8(t((T, K), "float8_e4m3fn"), f(1, T), t((N, K), "float8_e4m3fn"), f(1, 1),
                                                          stream=s),
    }


NAMES = ["grouped_forward", "grouped_gated_forward", "grouped_backward", "grouped_gated_backward", "quantize_act_fp8",
         "quantize_weights_fp8", "forward_fp8"]


@pytest.mark.parametrize("name", NAMES)
def test_buffers_belong_to_the_stream_of_the_call(bl, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(streams, "Torch", _Torch)
    streams._given_stream(bl, monkeypatch, _calls(bl)[name])
    streams._current_stream(bl, monkeypatch, _calls(bl)[name])


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(bl, monkeypatch, name):  # noqa: F811
    library = streams.Library()
    monkeypatch.setattr(bl, "_torch", _Torch)
    monkeypatch.setattr(bl, "lib", library)
    with pytest.raises(ValueError, match="stream"):
        _calls(bl)[name](streams.Stream(77, device_index=1))
    assert library.streams == []


def test_binding_refuses_shapes(bl, monkeypatch):  # noqa: F811
    """Tensors that do not fit each other, each refused by its name before the library is called."""
    library = streams.Library()
    monkeypatch.setattr(bl, "_torch", _Torch)
    monkeypatch.setattr(bl, "lib", library)
    t = streams.Tensor
    f = lambda *s: t(s, "float32")
    ok = dict(x_q=t((T, K), "int8"), beta=f(T), offsets=t(E + 1, "int64"), W_packed=t((E, N, K // 4), "uint8"), alpha=f(E),
              rows=t(M, "int64"), bias=f(E, N), y=f(M, N))
    bl.bitlinear_grouped_forward(**ok)
    assert len(library.streams) == 1
    for name, wrong in (("beta", f(T + 1)), ("offsets", t(E, "int64")), ("offsets", t(E + 1, "int32")), ("rows", t(M, "int32")),
                        ("W_packed", t((E, N, K // 2), "uint8")), ("alpha", f(1)), ("bias", f(N)), ("y", f(T, N))):
        with pytest.raises(ValueError, match=name):
            bl.bitlinear_grouped_forward(**dict(ok, **{name: wrong}))
    for wrong in (t((N, K // 4), "uint8"), f(E)):
        with pytest.raises(ValueError, match="W_packed"):
            bl.bitlinear_grouped_forward(**dict(ok, W_packed=wrong))
    with pytest.raises(ValueError, match="rows"):
        bl.bitlinear_grouped_forward(**dict(ok, rows=t((M, 1), "int64")))
    e4 = lambda *s: t(s, "float8_e4m3fn")
    ok = dict(x_q=e4(T, K), x_scale=f(1, T), W_q=e4(N, K), W_scale=f(1, 1), bias=f(N), y=f(T, N))
    for name, wrong in (("x_scale", f(T, 1)), ("W_q", e4(N, K + 1)), ("W_q", t((N, K), "int8")), ("W_scale", f(1, 2)),
                        ("bias", f(1)), ("y", f(N, T))):
        with pytest.raises(ValueError, match=name):
            bl.bitlinear_forward_fp8(**dict(ok, **{name: wrong}))
    assert len(library.streams) == 1
