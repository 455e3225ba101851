"""Where the binding takes the tensors that it allocates from, shown without a GPU: torch's allocator
keeps a pool for each stream, and a block of the current stream's pool may still be in use by work
queued there, which a call on another stream does not wait for.  A stand-in for torch notes the
stream that is current at each allocation; the library's calls are stand-ins that enqueue nothing."""
import contextlib
import types

import pytest

from test_abi_host import bl  # noqa: F401  (fixture)


class Stream:
    def __init__(self, handle, device_index=0):
        self.cuda_stream = handle
        self.device_index = device_index


class Tensor:
    is_cuda = True
    device = "cuda:0"

    def __init__(self, shape, dtype, pool=None):
        self.shape = (shape,) if isinstance(shape, int) else tuple(shape)
        self.dtype = dtype
        self.pool = pool                       # the stream that was current when it was allocated
        self.recorded = []

    @property
    def ndim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        self.recorded.append(stream)


class Torch(types.SimpleNamespace):
    """The parts of torch that the binding uses."""

    def __init__(self):
        super().__init__(Tensor=Tensor, float32="float32", uint8="uint8", int8="int8", int32="int32")
        self.home = self.now = Stream(0)
        self.allocated = []
        self._C = types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda i: self.now.cuda_stream)
        self.cuda = types.SimpleNamespace(Stream=Stream, ExternalStream=lambda handle, device: Stream(handle),
                                          stream=self._on, current_stream=lambda device=None: self.now,
                                          current_device=lambda: 0)

    @contextlib.contextmanager
    def _on(self, stream):
        before, self.now = self.now, stream
        try:
            yield
        finally:
            self.now = before

    def empty(self, shape, dtype, device):
        self.allocated.append(Tensor(shape, dtype, self.now))
        return self.allocated[-1]


class Library:
    """Every call returns OK; sizes are 64."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size") or name.endswith("_bytes"):
                return 64
            self.streams.append(args[-1])
            return 0
        return call


M, K, N = 3, 64, 64


def _operands():
    f = lambda *s: Tensor(s, "float32")
    i8 = lambda *s: Tensor(s, "int8")
    u8 = lambda *s: Tensor(s, "uint8")
    return f, i8, u8


def _new_calls(bl):  # noqa: F811
    f, i8, u8 = _operands()
    one, w = f(1), u8(N, K // 4)
    act = bl.BITLINEAR_ACT_SILU
    return {
        "gated_forward": lambda s: bl.bitlinear_gated_forward(f(M, K), w, one, w, one, act, stream=s),
        "backward": lambda s: bl.bitlinear_backward(f(M, N), i8(M, K), f(M), w, one, stream=s),
        "gated_backward": lambda s: bl.bitlinear_gated_backward(f(M, N), f(M, N), f(M, N), i8(M, K), f(M), w, one, w, one,
                                                                act, stream=s),
        "quantize_weights_i8": lambda s: bl.bitlinear_quantize_weights_i8(f(N, K), stream=s),
        "forward_i8": lambda s: bl.bitlinear_forward_i8(i8(M, K), f(M), i8(N, K), f(N), acc=True, stream=s),
    }


def _old_calls(bl):  # noqa: F811
    f, i8, u8 = _operands()
    one, w = f(1), u8(N, K // 4)
    return {
        "quantize_weights": lambda s: bl.bitlinear_quantize_weights(f(N, K), stream=s),
        "quantize_weights_rows": lambda s: bl.bitlinear_quantize_weights_rows(f(N, K), stream=s),
        "quantize_act": lambda s: bl.bitlinear_quantize_act(f(M, K), stream=s),
        "quantize_weights_t5": lambda s: bl.bitlinear_quantize_weights_t5(f(N, K), stream=s),
        "repack_t5": lambda s: bl.bitlinear_repack_t5(w, K, stream=s),
        "forward_t5": lambda s: bl.bitlinear_forward_t5(i8(M, K), f(M), u8(N, 64), one, stream=s),
        "quantize_weights_blocks": lambda s: bl.bitlinear_quantize_weights_blocks(f(N, 2 * K), stream=s),
        "forward_blocks": lambda s: bl.bitlinear_forward_blocks(i8(M, K), f(M), w, f(N), stream=s),
        "mlp_forward": lambda s: bl.bitlinear_mlp_forward(f(M, K), w, one, w, one, stream=s),
        "hadamard_rows": lambda s: bl.bitlinear_hadamard_rows(f(M, K), 64, stream=s),
        "quantize_act_hadamard": lambda s: bl.bitlinear_quantize_act_hadamard(f(M, K), 64, stream=s),
        "forward_fused_hadamard": lambda s: bl.bitlinear_forward_fused_hadamard(f(M, K), 64, None, w, one, stream=s),
        "forward": lambda s: bl.bitlinear_forward(i8(M, K), f(M), w, one, acc=True, stream=s),
        "forward_rows": lambda s: bl.bitlinear_forward_rows(i8(M, K), f(M), w, f(N), acc=True, stream=s),
        "forward_fused": lambda s: bl.bitlinear_forward_fused(f(M, K), w, one, acc=True, stream=s),
        "forward_fused_rows": lambda s: bl.bitlinear_forward_fused_rows(f(M, K), w, f(N), acc=True, stream=s),
    }


OLD = ["quantize_weights", "quantize_weights_rows", "quantize_act", "quantize_weights_t5", "repack_t5", "forward_t5",
       "quantize_weights_blocks", "forward_blocks", "mlp_forward", "hadamard_rows", "quantize_act_hadamard",
       "forward_fused_hadamard", "forward", "forward_rows", "forward_fused", "forward_fused_rows"]
NEW = ["gated_forward", "backward", "gated_backward", "quantize_weights_i8", "forward_i8"]


def _run(bl, monkeypatch, call, stream):  # noqa: F811
    torch, library = Torch(), Library()
    monkeypatch.setattr(bl, "_torch", lambda: torch)
    monkeypatch.setattr(bl, "lib", library)
    out = call(stream)
    assert torch.now is torch.home and torch.allocated
    out = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    return torch, library, out


def _given_stream(bl, monkeypatch, call):  # noqa: F811
    side = Stream(77)
    torch, library, out = _run(bl, monkeypatch, call, side)
    assert library.streams == [77]
    for t in torch.allocated:
        assert t.pool is side, t.shape
        # the caller uses on its own stream what it gets back, and sees nothing of the rest
        assert t.recorded == ([torch.home] if any(t is o for o in out) else []), t.shape


def _current_stream(bl, monkeypatch, call):  # noqa: F811
    torch, library, _ = _run(bl, monkeypatch, call, None)
    assert library.streams == [0]
    assert all(t.pool is torch.home and not t.recorded for t in torch.allocated)


@pytest.mark.parametrize("name", NEW)
def test_buffers_of_a_call_on_a_given_stream(bl, monkeypatch, name):  # noqa: F811
    _given_stream(bl, monkeypatch, _new_calls(bl)[name])


@pytest.mark.parametrize("name", NEW)
def test_buffers_of_a_call_on_the_current_stream(bl, monkeypatch, name):  # noqa: F811
    _current_stream(bl, monkeypatch, _new_calls(bl)[name])


@pytest.mark.parametrize("name", OLD)
def test_buffers_of_a_single_layer_call_on_a_given_stream(bl, monkeypatch, name):  # noqa: F811
    _given_stream(bl, monkeypatch, _old_calls(bl)[name])


@pytest.mark.parametrize("name", OLD)
def test_buffers_of_a_single_layer_call_on_the_current_stream(bl, monkeypatch, name):  # noqa: F811
    _current_stream(bl, monkeypatch, _old_calls(bl)[name])


@pytest.mark.parametrize("name", NEW)
def test_a_stream_of_another_device_is_refused(bl, monkeypatch, name):  # noqa: F811
    library = Library()
    monkeypatch.setattr(bl, "_torch", Torch)
    monkeypatch.setattr(bl, "lib", library)
    with pytest.raises(ValueError, match="stream"):
        _new_calls(bl)[name](Stream(77, device_index=1))
    assert library.streams == []
