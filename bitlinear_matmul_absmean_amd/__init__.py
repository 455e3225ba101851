"""Python binding of the MI355X BitNet b1.58 BitLinear library (W1.58A8).

Argument marshalling only: every step of the computation runs in the HIP kernels of
``libbitlinear.so`` behind the C ABI of ``include/bitlinear.h``.  PyTorch provides device
memory (tensors) and the current HIP stream; nothing here computes on the host.  If the
library has not been built, importing this package raises -- there is no fallback.

A call runs on ``stream`` if one is given, else on the current stream; what it allocates belongs
to the stream it runs on.  Ordering it with the work that made its arguments and that uses its
results is up to the caller.

The functions carry the C names.  ``lib`` exposes the raw C entry points (ctypes) for
callers that manage pointers themselves.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbitlinear.so")

BITLINEAR_OK = 0
BITLINEAR_ERR_INVALID_ARG = -1
BITLINEAR_ERR_SHAPE = -2
BITLINEAR_ERR_ALIGNMENT = -3
BITLINEAR_ERR_WORKSPACE = -4
BITLINEAR_ERR_HIP = -5
BITLINEAR_ERR_SCRATCH = -6
BITLINEAR_MAX_K = 16909320

# bitlinear_activation
BITLINEAR_ACT_GELU = 1
BITLINEAR_ACT_SILU = 2
BITLINEAR_ACT_RELU2 = 3

# Every symbol the header declares, with (restype, argtypes).
_P, _I64, _SZ, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "bitlinear_abi_version": (_INT, []),
    "bitlinear_status_string": (ctypes.c_char_p, [_INT]),
    "bitlinear_last_hip_error": (_INT, []),
    "bitlinear_quantize_weights_workspace_size": (_SZ, [_I64, _I64]),
    "bitlinear_quantize_weights": (_INT, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitlinear_quantize_weights_noalloc": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "bitlinear_quantize_weights_noalloc_max_rows": (_SZ, []),
    "bitlinear_quantize_weights_rows": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "bitlinear_quantize_act": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "bitlinear_forward": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P]),
    "bitlinear_forward_rows": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P]),
    "bitlinear_forward_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _P, _P]),
    "bitlinear_forward_fused": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "bitlinear_forward_fused_rows": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "bitlinear_forward_fused_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _P, _P, _P]),
    "bitlinear_t5_row_bytes": (_SZ, [_I64]),
    "bitlinear_quantize_weights_t5": (_INT, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitlinear_forward_t5": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P]),
    "bitlinear_repack_t5": (_INT, [_P, _I64, _I64, _P, _P]),
    "bitlinear_quantize_weights_blocks": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "bitlinear_forward_blocks": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P]),
    "bitlinear_mlp_forward": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "bitlinear_hadamard_rows": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "bitlinear_quantize_act_hadamard": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P, _P]),
    "bitlinear_forward_fused_hadamard": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, _P]),
    "bitlinear_gated_forward": (_INT, [_P, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _INT, _P, _P, _P, _P, _P, _P]),
    "bitlinear_backward_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitlinear_backward": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bitlinear_gated_backward_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitlinear_gated_backward": (_INT, [_P, _P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _INT, _P, _P, _P, _P, _P,
                                        _P, _SZ, _P]),
    "bitlinear_quantize_weights_i8": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "bitlinear_forward_i8": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m bitlinear_matmul_absmean_amd.build` "
            "(hipcc --offload-arch=gfx950). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class BitLinearError(RuntimeError):
    def __init__(self, what: str, status: int):
        msg = lib.bitlinear_status_string(status).decode()
        if status == BITLINEAR_ERR_HIP:
            msg += f" (hipError {lib.bitlinear_last_hip_error()})"
        super().__init__(f"{what}: {msg} [status {status}]")
        self.status = status


def _check(what: str, status: int):
    if status != BITLINEAR_OK:
        raise BitLinearError(what, status)


def abi_version() -> int:
    return lib.bitlinear_abi_version()


# ------------------------------------------------------------------ torch marshalling
def _torch():
    import torch  # imported lazily: the C entry points above need no torch
    return torch


def _dev(t, dtype, name, numel=None):
    """Device pointer of t after checking device, dtype, layout and (numel) the minimum number of
    elements the library reads or writes through it."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} must hold at least {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _stream(stream):
    """Raw HIP stream handle: `stream`, else torch's current stream on the current device (the
    capture stream inside torch.cuda.graph).  The raw accessor skips building a Stream object,
    a few microseconds of host time per call."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream, scratch=False):
    """A tensor that the binding allocates for a call on `stream` (None: the current stream).

    The block comes from the pool of the stream that the call runs on: one from the current stream's
    pool may still be in use by work queued there before the call, which a given stream does not
    wait for.  What is handed back is recorded on the caller's stream as well, so that the block is
    not handed out again before the caller's work on it is done; scratch nobody else sees."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def bitlinear_quantize_weights(W, W_packed=None, alpha=None, workspace=None, stream=None):
    """W [N, K] fp32 -> (W_packed uint8 [N, K/4], alpha fp32 [1]) on the device."""
    torch = _torch()
    N, K = W.shape
    if W_packed is None:
        W_packed = _empty((N, K // 4), torch.uint8, W.device, stream)
    if alpha is None:
        alpha = _empty(1, torch.float32, W.device, stream)
    need = lib.bitlinear_quantize_weights_workspace_size(N, K)
    if workspace is None:
        workspace = _empty(max(need, 8), torch.uint8, W.device, stream, scratch=True)
    _check("bitlinear_quantize_weights", lib.bitlinear_quantize_weights(
        _dev(W, torch.float32, "W", N * K), N, K, _dev(W_packed, torch.uint8, "W_packed", N * (K // 4)),
        _dev(alpha, torch.float32, "alpha", 1), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)))
    return W_packed, alpha


def bitlinear_quantize_weights_noalloc(W, W_packed, alpha, stream=None):
    """bitlinear_quantize_weights into caller buffers W_packed uint8 [N, K/4] and alpha fp32 [1],
    without a workspace: the library uses its fixed per-device scratch and allocates nothing
    (neither does this wrapper).  Calls that overlap on one device race."""
    torch = _torch()
    N, K = W.shape
    _check("bitlinear_quantize_weights_noalloc", lib.bitlinear_quantize_weights_noalloc(
        _dev(W, torch.float32, "W", N * K), N, K, _dev(W_packed, torch.uint8, "W_packed", N * (K // 4)),
        _dev(alpha, torch.float32, "alpha", 1), _stream(stream)))
    return W_packed, alpha


def bitlinear_quantize_weights_rows(W, W_packed=None, alpha_rows=None, stream=None):
    """W [N, K] fp32 -> (W_packed uint8 [N, K/4], alpha_rows fp32 [N])."""
    torch = _torch()
    N, K = W.shape
    if W_packed is None:
        W_packed = _empty((N, K // 4), torch.uint8, W.device, stream)
    if alpha_rows is None:
        alpha_rows = _empty(N, torch.float32, W.device, stream)
    _check("bitlinear_quantize_weights_rows", lib.bitlinear_quantize_weights_rows(
        _dev(W, torch.float32, "W", N * K), N, K, _dev(W_packed, torch.uint8, "W_packed", N * (K // 4)),
        _dev(alpha_rows, torch.float32, "alpha_rows", N), _stream(stream)))
    return W_packed, alpha_rows


def bitlinear_quantize_act(x, x_q=None, beta=None, stream=None):
    """x [M, K] fp32 -> (x_q int8 [M, K], beta fp32 [M])."""
    torch = _torch()
    M, K = x.shape
    if x_q is None:
        x_q = _empty((M, K), torch.int8, x.device, stream)
    if beta is None:
        beta = _empty(M, torch.float32, x.device, stream)
    _check("bitlinear_quantize_act", lib.bitlinear_quantize_act(
        _dev(x, torch.float32, "x", M * K), M, K, _dev(x_q, torch.int8, "x_q", M * K),
        _dev(beta, torch.float32, "beta", M), _stream(stream)))
    return x_q, beta


def bitlinear_quantize_weights_t5(W, W_t5=None, alpha=None, workspace=None, stream=None):
    """W [N, K] fp32 -> (W_t5 uint8 [N, 16 ceil(K/80)], alpha fp32 [1]): five codes per byte."""
    torch = _torch()
    N, K = W.shape
    rb = lib.bitlinear_t5_row_bytes(K)
    if W_t5 is None:
        W_t5 = _empty((N, rb), torch.uint8, W.device, stream)
    if alpha is None:
        alpha = _empty(1, torch.float32, W.device, stream)
    need = lib.bitlinear_quantize_weights_workspace_size(N, K)
    if workspace is None:
        workspace = _empty(max(need, 8), torch.uint8, W.device, stream, scratch=True)
    _check("bitlinear_quantize_weights_t5", lib.bitlinear_quantize_weights_t5(
        _dev(W, torch.float32, "W", N * K), N, K, _dev(W_t5, torch.uint8, "W_t5", N * rb),
        _dev(alpha, torch.float32, "alpha", 1),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)))
    return W_t5, alpha


def bitlinear_repack_t5(W_packed, K, W_t5=None, stream=None):
    """2-bit packed [N, K/4] -> five codes per byte [N, 16 ceil(K/80)] (same codes)."""
    torch = _torch()
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    if W_t5 is None:
        W_t5 = _empty((N, lib.bitlinear_t5_row_bytes(K)), torch.uint8, W_packed.device, stream)
    _check("bitlinear_repack_t5", lib.bitlinear_repack_t5(
        _dev(W_packed, torch.uint8, "W_packed"), N, K,
        _dev(W_t5, torch.uint8, "W_t5", N * lib.bitlinear_t5_row_bytes(K)), _stream(stream)))
    return W_t5


def bitlinear_forward_t5(x_q, beta, W_t5, alpha, bias=None, y=None, stream=None):
    """y [M, N] from x_q, beta and 5-trit packed weights."""
    torch = _torch()
    M, K = x_q.shape
    N = W_t5.shape[0]
    if W_t5.shape[1] != lib.bitlinear_t5_row_bytes(K):
        raise ValueError("W_t5 must be [N, bitlinear_t5_row_bytes(K)]")
    if y is None:
        y = _empty((M, N), torch.float32, x_q.device, stream)
    _check("bitlinear_forward_t5", lib.bitlinear_forward_t5(
        _dev(x_q, torch.int8, "x_q"), _dev(beta, torch.float32, "beta", M), M, K, _dev(W_t5, torch.uint8, "W_t5"),
        _dev(alpha, torch.float32, "alpha", 1), N,
        _dev(bias, torch.float32, "bias", N) if bias is not None else None,
        _dev(y, torch.float32, "y", M * N), _stream(stream)))
    return y


def bitlinear_quantize_weights_blocks(W, W_packed=None, alpha_blocks=None, stream=None):
    """W [N, K] fp32 -> (W_packed uint8 [N, K/4], alpha_blocks fp32 [N, K/128])."""
    torch = _torch()
    N, K = W.shape
    if W_packed is None:
        W_packed = _empty((N, K // 4), torch.uint8, W.device, stream)
    if alpha_blocks is None:
        alpha_blocks = _empty((N, K // 128), torch.float32, W.device, stream)
    _check("bitlinear_quantize_weights_blocks", lib.bitlinear_quantize_weights_blocks(
        _dev(W, torch.float32, "W", N * K), N, K, _dev(W_packed, torch.uint8, "W_packed", N * (K // 4)),
        _dev(alpha_blocks, torch.float32, "alpha_blocks", N * (K // 128)), _stream(stream)))
    return W_packed, alpha_blocks


def bitlinear_forward_blocks(x_q, beta, W_packed, alpha_blocks, bias=None, y=None, stream=None):
    """y [M, N] from x_q, beta and block-scaled packed weights."""
    torch = _torch()
    M, K = x_q.shape
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    if y is None:
        y = _empty((M, N), torch.float32, x_q.device, stream)
    _check("bitlinear_forward_blocks", lib.bitlinear_forward_blocks(
        _dev(x_q, torch.int8, "x_q"), _dev(beta, torch.float32, "beta", M), M, K,
        _dev(W_packed, torch.uint8, "W_packed"), _dev(alpha_blocks, torch.float32, "alpha_blocks", N * (K // 128)),
        N, _dev(bias, torch.float32, "bias", N) if bias is not None else None, _dev(y, torch.float32, "y", M * N),
        _stream(stream)))
    return y


def bitlinear_mlp_forward(x, W1_packed, alpha1, W2_packed, alpha2, bias1=None, bias2=None, y=None, g=None,
                          x_q1=None, beta1=None, x_q2=None, beta2=None, stream=None):
    """BitMLP y = fc2(GELU(fc1(x))); returns (y, g).  x_q1/beta1/x_q2/beta2 are allocated
    when M > 1 and not given (the two-call path needs them beyond four tokens and is the
    faster one for most several-token shapes)."""
    torch = _torch()
    M, d_model = x.shape
    d_ff = W1_packed.shape[0]
    if W1_packed.shape[1] * 4 != d_model or W2_packed.shape != (d_model, d_ff // 4):
        raise ValueError("W1_packed must be [d_ff, d_model/4] and W2_packed [d_model, d_ff/4]")
    if y is None:
        y = _empty((M, d_model), torch.float32, x.device, stream)
    if g is None:
        g = _empty((M, d_ff), torch.float32, x.device, stream)
    if M > 1:
        if x_q1 is None:
            x_q1 = _empty((M, d_model), torch.int8, x.device, stream, scratch=True)
        if beta1 is None:
            beta1 = _empty(M, torch.float32, x.device, stream, scratch=True)
        if x_q2 is None:
            x_q2 = _empty((M, d_ff), torch.int8, x.device, stream, scratch=True)
        if beta2 is None:
            beta2 = _empty(M, torch.float32, x.device, stream, scratch=True)
    opt = lambda t, dt, n, k: _dev(t, dt, n, k) if t is not None else None
    _check("bitlinear_mlp_forward", lib.bitlinear_mlp_forward(
        _dev(x, torch.float32, "x", M * d_model), M, d_model, d_ff, _dev(W1_packed, torch.uint8, "W1_packed"),
        _dev(alpha1, torch.float32, "alpha1", 1), opt(bias1, torch.float32, "bias1", d_ff),
        _dev(W2_packed, torch.uint8, "W2_packed"), _dev(alpha2, torch.float32, "alpha2", 1),
        opt(bias2, torch.float32, "bias2", d_model), _dev(y, torch.float32, "y", M * d_model),
        _dev(g, torch.float32, "g", M * d_ff), opt(x_q1, torch.int8, "x_q1", M * d_model),
        opt(beta1, torch.float32, "beta1", M), opt(x_q2, torch.int8, "x_q2", M * d_ff),
        opt(beta2, torch.float32, "beta2", M), _stream(stream)))
    return y, g


def bitlinear_hadamard_rows(x, block, signs=None, out=None, stream=None):
    """x [M, K] fp32 -> rows rotated by diag(d) . blockdiag(H_block) / sqrt(block); out may be x."""
    torch = _torch()
    M, K = x.shape
    if out is None:
        out = _empty((M, K), torch.float32, x.device, stream)
    _check("bitlinear_hadamard_rows", lib.bitlinear_hadamard_rows(
        _dev(x, torch.float32, "x", M * K), M, K, int(block),
        _dev(signs, torch.int8, "signs", K) if signs is not None else None,
        _dev(out, torch.float32, "out", M * K), _stream(stream)))
    return out


def bitlinear_quantize_act_hadamard(x, block, signs=None, x_q=None, beta=None, stream=None):
    """x [M, K] fp32 -> (x_q int8 [M, K], beta fp32 [M]) of the rotated rows."""
    torch = _torch()
    M, K = x.shape
    if x_q is None:
        x_q = _empty((M, K), torch.int8, x.device, stream)
    if beta is None:
        beta = _empty(M, torch.float32, x.device, stream)
    _check("bitlinear_quantize_act_hadamard", lib.bitlinear_quantize_act_hadamard(
        _dev(x, torch.float32, "x", M * K), M, K, int(block),
        _dev(signs, torch.int8, "signs", K) if signs is not None else None,
        _dev(x_q, torch.int8, "x_q", M * K), _dev(beta, torch.float32, "beta", M), _stream(stream)))
    return x_q, beta


def bitlinear_forward_fused_hadamard(x, block, signs, W_packed, alpha, bias=None, y=None, x_q=None, beta=None,
                                     stream=None):
    """y [M, N] from fp32 x: rotation (block, signs), absmax int8 and the forward in one call."""
    torch = _torch()
    M, K = x.shape
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    if y is None:
        y = _empty((M, N), torch.float32, x.device, stream)
    opt = lambda t, dt, n, k: _dev(t, dt, n, k) if t is not None else None
    _check("bitlinear_forward_fused_hadamard", lib.bitlinear_forward_fused_hadamard(
        _dev(x, torch.float32, "x", M * K), M, K, int(block), opt(signs, torch.int8, "signs", K),
        _dev(W_packed, torch.uint8, "W_packed"), _dev(alpha, torch.float32, "alpha", 1), N,
        opt(bias, torch.float32, "bias", N), _dev(y, torch.float32, "y", M * N), opt(x_q, torch.int8, "x_q", M * K),
        opt(beta, torch.float32, "beta", M), _stream(stream)))
    return y


def _forward(fn, what, x_q, beta, W_packed, alpha, bias, y, acc, stream, alpha_n=1):
    torch = _torch()
    M, K = x_q.shape
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    if y is None:
        y = _empty((M, N), torch.float32, x_q.device, stream)
    if acc is True:
        acc = _empty((M, N), torch.int32, x_q.device, stream)
    acc_ptr = _dev(acc, torch.int32, "acc", M * N) if acc is not None and acc is not False else None
    bias_ptr = _dev(bias, torch.float32, "bias", N) if bias is not None else None
    _check(what, fn(
        _dev(x_q, torch.int8, "x_q"), _dev(beta, torch.float32, "beta", M), M, K,
        _dev(W_packed, torch.uint8, "W_packed"), _dev(alpha, torch.float32, "alpha", alpha_n), N,
        bias_ptr, _dev(y, torch.float32, "y", M * N), acc_ptr, _stream(stream)))
    return (y, acc) if acc_ptr is not None else y


def bitlinear_forward(x_q, beta, W_packed, alpha, bias=None, y=None, acc=None, stream=None):
    """y [M, N] = (x_q . W_hat^T) * alpha*beta/127 (+ bias).  acc=True (or an int32 [M, N]
    tensor) also returns the exact integer sums: (y, acc)."""
    return _forward(lib.bitlinear_forward, "bitlinear_forward", x_q, beta, W_packed, alpha,
                    bias, y, acc, stream)


def bitlinear_forward_rows(x_q, beta, W_packed, alpha_rows, bias=None, y=None, acc=None, stream=None):
    """bitlinear_forward with one alpha per output row."""
    return _forward(lib.bitlinear_forward_rows, "bitlinear_forward_rows", x_q, beta, W_packed,
                    alpha_rows, bias, y, acc, stream, alpha_n=W_packed.shape[0])


def _forward_fused(name, x, W_packed, alpha, bias, y, x_q, beta, acc, stream):
    torch = _torch()
    M, K = x.shape
    N = W_packed.shape[0]
    if W_packed.shape[1] * 4 != K:
        raise ValueError("W_packed must be [N, K/4]")
    if y is None:
        y = _empty((M, N), torch.float32, x.device, stream)
    if acc is True:
        acc = _empty((M, N), torch.int32, x.device, stream)
    acc_ptr = _dev(acc, torch.int32, "acc", M * N) if acc is not None and acc is not False else None
    _check(name, getattr(lib, name)(
        _dev(x, torch.float32, "x", M * K), M, K, _dev(W_packed, torch.uint8, "W_packed"),
        _dev(alpha, torch.float32, "alpha", N if name.endswith("_rows") else 1), N,
        _dev(bias, torch.float32, "bias", N) if bias is not None else None, _dev(y, torch.float32, "y", M * N),
        _dev(x_q, torch.int8, "x_q", M * K) if x_q is not None else None,
        _dev(beta, torch.float32, "beta", M) if beta is not None else None, acc_ptr, _stream(stream)))
    return (y, acc) if acc_ptr is not None else y


def bitlinear_forward_fused(x, W_packed, alpha, bias=None, y=None, x_q=None, beta=None, acc=None,
                            stream=None):
    """y [M, N] from fp32 x [M, K] in one call (activation quantization + forward).
    x_q / beta (tensors) receive the quantized activations if given; acc as bitlinear_forward.
    Returns y, or (y, acc) when acc is requested."""
    return _forward_fused("bitlinear_forward_fused", x, W_packed, alpha, bias, y, x_q, beta, acc, stream)


def bitlinear_forward_fused_rows(x, W_packed, alpha_rows, bias=None, y=None, x_q=None, beta=None, acc=None,
                                 stream=None):
    """bitlinear_forward_fused with alpha_rows [N] fp32 (one alpha per output row); also the
    call for grouped projections (stacked packed rows, each projection's alpha repeated)."""
    return _forward_fused("bitlinear_forward_fused_rows", x, W_packed, alpha_rows, bias, y, x_q, beta, acc, stream)


def _shaped(t, dtype, name, shape, index):
    """Device pointer of t (None for None) after checking that it is a contiguous tensor of exactly
    this dtype and shape on device `index`.  One test when all is well: a call marshals a dozen
    tensors, and single-token kernels take less time than their checks would."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on device {index}, got {t.device}")


def _rows(t, name):
    """Shape (rows, columns) and device index of a matrix argument, which has to lie on the current
    device (the library launches there)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, got {len(shape)} dimensions")
    index = t.get_device()
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current device")
    return shape[0], shape[1], index


def _stream_on(stream, index):
    """_stream for a call whose tensors are known to lie on the current device `index`, which a given
    stream has to be of too."""
    if stream is not None:
        if getattr(stream, "device_index", index) != index:
            raise ValueError(f"stream must be of device {index}")
        return stream.cuda_stream
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else _stream(None)


def _first(t, name):
    """Rows of a matrix argument."""
    if getattr(t, "ndim", 0) != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape[0]


def bitlinear_gated_forward(x, Wg_packed, alpha_g, Wu_packed, alpha_u, act, bias_g=None, bias_u=None, h=None, g=None,
                            u=None, x_q=None, beta=None, stream=None):
    """h [M, F] = a(g) * u with g, u the BitLinears of fp32 x [M, K] under Wg, Wu [F, K/4]; act is one
    of BITLINEAR_ACT_GELU / _SILU / _RELU2.  g and u (fp32 [M, F], both or neither), x_q and beta
    (tensors) receive what bitlinear_gated_backward needs; x_q and beta are allocated if not given.
    Returns h."""
    torch = _torch()
    M, K, dev = _rows(x, "x")
    F = _first(Wg_packed, "Wg_packed")
    if h is None:
        h = _empty((M, F), torch.float32, dev, stream)
    if x_q is None:
        x_q = _empty((M, K), torch.int8, dev, stream, scratch=True)
    if beta is None:
        beta = _empty(M, torch.float32, dev, stream, scratch=True)
    f32, u8 = torch.float32, torch.uint8
    _check("bitlinear_gated_forward", lib.bitlinear_gated_forward(
        _shaped(x, f32, "x", (M, K), dev), M, K, _shaped(Wg_packed, u8, "Wg_packed", (F, K // 4), dev),
        _shaped(alpha_g, f32, "alpha_g", (1,), dev), _shaped(bias_g, f32, "bias_g", (F,), dev),
        _shaped(Wu_packed, u8, "Wu_packed", (F, K // 4), dev), _shaped(alpha_u, f32, "alpha_u", (1,), dev),
        _shaped(bias_u, f32, "bias_u", (F,), dev), F, int(act), _shaped(h, f32, "h", (M, F), dev),
        _shaped(g, f32, "g", (M, F), dev), _shaped(u, f32, "u", (M, F), dev),
        _shaped(x_q, torch.int8, "x_q", (M, K), dev), _shaped(beta, f32, "beta", (M,), dev), _stream_on(stream, dev)))
    return h


def bitlinear_backward_workspace_size(M, K, N) -> int:
    """Bytes of workspace of bitlinear_backward (0 for invalid sizes)."""
    return lib.bitlinear_backward_workspace_size(M, K, N)


def bitlinear_gated_backward_workspace_size(M, K, F) -> int:
    """Bytes of workspace of bitlinear_gated_backward (0 for invalid sizes)."""
    return lib.bitlinear_gated_backward_workspace_size(M, K, F)


def _workspace(workspace, need, index, stream):
    """The given workspace, or a new one of the bytes needed, its pointer and its bytes."""
    if workspace is None:
        workspace = _empty(max(need, 256), _torch().uint8, index, stream, scratch=True)
    ptr = _dev(workspace, _torch().uint8, "workspace")
    if workspace.get_device() != index:
        raise ValueError(f"workspace must be on device {index}, got {workspace.device}")
    return workspace, ptr, workspace.numel()


def bitlinear_backward(dy, x_q, beta, W_packed, alpha, dx=None, dW=None, dbias=None, workspace=None, stream=None):
    """Gradients of y = bitlinear_forward(x_q, beta, W_packed, alpha, bias): dx [M, K], dW [N, K] and
    dbias [N], each written if its tensor is given; with none given, dx and dW are allocated.
    Returns (dx, dW, dbias), None for what was not asked for."""
    torch = _torch()
    M, N, dev = _rows(dy, "dy")
    _, K, _ = _rows(x_q, "x_q")
    f32 = torch.float32
    if dx is None and dW is None and dbias is None:
        dx = _empty((M, K), f32, dev, stream)
        dW = _empty((N, K), f32, dev, stream)
    workspace, ws, ws_bytes = _workspace(workspace, lib.bitlinear_backward_workspace_size(M, K, N), dev, stream)
    _check("bitlinear_backward", lib.bitlinear_backward(
        _shaped(dy, f32, "dy", (M, N), dev), M, N, _shaped(x_q, torch.int8, "x_q", (M, K), dev),
        _shaped(beta, f32, "beta", (M,), dev), K, _shaped(W_packed, torch.uint8, "W_packed", (N, K // 4), dev),
        _shaped(alpha, f32, "alpha", (1,), dev), _shaped(dx, f32, "dx", (M, K), dev),
        _shaped(dW, f32, "dW", (N, K), dev), _shaped(dbias, f32, "dbias", (N,), dev), ws, ws_bytes, _stream_on(stream, dev)))
    return dx, dW, dbias


def bitlinear_gated_backward(dh, g, u, x_q, beta, Wg_packed, alpha_g, Wu_packed, alpha_u, act, dx=None, dWg=None,
                             dWu=None, dbias_g=None, dbias_u=None, workspace=None, stream=None):
    """Gradients of bitlinear_gated_forward from dh [M, F] and the g, u, x_q, beta it left: dx [M, K],
    dWg and dWu [F, K] (both or neither), dbias_g and dbias_u [F], each written if its tensor is
    given; with none given, dx, dWg and dWu are allocated.  Returns (dx, dWg, dWu, dbias_g, dbias_u),
    None for what was not asked for."""
    torch = _torch()
    M, F, dev = _rows(dh, "dh")
    _, K, _ = _rows(x_q, "x_q")
    f32, u8 = torch.float32, torch.uint8
    if dx is None and dWg is None and dWu is None and dbias_g is None and dbias_u is None:
        dx = _empty((M, K), f32, dev, stream)
        dWg = _empty((F, K), f32, dev, stream)
        dWu = _empty((F, K), f32, dev, stream)
    workspace, ws, ws_bytes = _workspace(workspace, lib.bitlinear_gated_backward_workspace_size(M, K, F), dev, stream)
    _check("bitlinear_gated_backward", lib.bitlinear_gated_backward(
        _shaped(dh, f32, "dh", (M, F), dev), _shaped(g, f32, "g", (M, F), dev), _shaped(u, f32, "u", (M, F), dev), M, F,
        _shaped(x_q, torch.int8, "x_q", (M, K), dev), _shaped(beta, f32, "beta", (M,), dev), K,
        _shaped(Wg_packed, u8, "Wg_packed", (F, K // 4), dev), _shaped(alpha_g, f32, "alpha_g", (1,), dev),
        _shaped(Wu_packed, u8, "Wu_packed", (F, K // 4), dev), _shaped(alpha_u, f32, "alpha_u", (1,), dev), int(act),
        _shaped(dx, f32, "dx", (M, K), dev), _shaped(dWg, f32, "dWg", (F, K), dev), _shaped(dWu, f32, "dWu", (F, K), dev),
        _shaped(dbias_g, f32, "dbias_g", (F,), dev), _shaped(dbias_u, f32, "dbias_u", (F,), dev), ws, ws_bytes,
        _stream_on(stream, dev)))
    return dx, dWg, dWu, dbias_g, dbias_u


def bitlinear_quantize_weights_i8(W, W_q=None, gamma=None, stream=None):
    """W [N, K] fp32 -> (W_q int8 [N, K], gamma fp32 [N]): absmax int8 codes, one scale per row."""
    torch = _torch()
    N, K, dev = _rows(W, "W")
    if W_q is None:
        W_q = _empty((N, K), torch.int8, dev, stream)
    if gamma is None:
        gamma = _empty(N, torch.float32, dev, stream)
    _check("bitlinear_quantize_weights_i8", lib.bitlinear_quantize_weights_i8(
        _shaped(W, torch.float32, "W", (N, K), dev), N, K, _shaped(W_q, torch.int8, "W_q", (N, K), dev),
        _shaped(gamma, torch.float32, "gamma", (N,), dev), _stream_on(stream, dev)))
    return W_q, gamma


def bitlinear_forward_i8(x_q, beta, W_q, gamma, bias=None, y=None, acc=None, stream=None):
    """y [M, N] = (x_q . W_q^T) * (beta / 127) * (gamma / 127) (+ bias).  acc=True (or an int32
    [M, N] tensor) also returns the exact integer sums: (y, acc)."""
    torch = _torch()
    M, K, dev = _rows(x_q, "x_q")
    N = _first(W_q, "W_q")
    f32 = torch.float32
    if y is None:
        y = _empty((M, N), f32, dev, stream)
    if acc is True:
        acc = _empty((M, N), torch.int32, dev, stream)
    elif acc is False:
        acc = None
    _check("bitlinear_forward_i8", lib.bitlinear_forward_i8(
        _shaped(x_q, torch.int8, "x_q", (M, K), dev), _shaped(beta, f32, "beta", (M,), dev), M, K,
        _shaped(W_q, torch.int8, "W_q", (N, K), dev), _shaped(gamma, f32, "gamma", (N,), dev), N,
        _shaped(bias, f32, "bias", (N,), dev), _shaped(y, f32, "y", (M, N), dev),
        _shaped(acc, torch.int32, "acc", (M, N), dev), _stream_on(stream, dev)))
    return y if acc is None else (y, acc)


def bitlinear_forward_fused_kernel(M, K, N, x=None, W_packed=None, x_q=None) -> str:
    xp = x.data_ptr() if x is not None else 256
    wp = W_packed.data_ptr() if W_packed is not None else 256
    qp = x_q.data_ptr() if x_q is not None else None
    return lib.bitlinear_forward_fused_kernel(M, K, N, xp, wp, qp).decode()


def bitlinear_forward_kernel(M, K, N, x_q=None, W_packed=None) -> str:
    """Name of the kernel bitlinear_forward selects (pointers decide alignment; None
    stands for a 256-byte aligned allocation)."""
    xp = x_q.data_ptr() if x_q is not None else 256
    wp = W_packed.data_ptr() if W_packed is not None else 256
    return lib.bitlinear_forward_kernel(M, K, N, xp, wp).decode()
