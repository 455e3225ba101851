"""Workloads of the gated feed-forward block, the BitLinear gradients and the W8A8 product.

Three groups of operators of a ternary (W1.58A8) feed-forward layer, each with its plain form
in elementary torch operations and the call that a user makes of the library:

  gated      h = act(g) * u, g and u BitLinears of the same x (per-token absmax int8 codes,
             ternary weights); training calls also keep g, u, x_q and beta
  gated_bwd  its gradients: dx, dWg, dWu (straight through the quantizers), bias gradients
  linear_bwd the gradients of one BitLinear: dx, dW, dbias
  i8         y = x_q . W_q^T with a scale for each token and each output channel

Weights are N(0, 0.02) latent weights quantized as the layer defines it; activations are
N(0, 1) with one element in a thousand 20 times larger; incoming gradients are small and
differ in size from token to token.
"""
import math

import numpy as np
import torch

own = False

W_STD = 0.02
OUTLIER_FRACTION = 0.001
OUTLIER_GAIN = 20.0


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence generating: 7B-class layer, one token, latency counts
        dict(name="gated_decode_1", op="gated", M=1, K=4096, F=11008, act="silu", bias=False, train=False),
        # sixteen sequences generating on a 70B-class layer: the weights' bytes count
        dict(name="gated_decode_16", op="gated", M=16, K=8192, F=28672, act="relu2", bias=False, train=False),
        # a long prompt on the 7B-class layer: the integer products count
        dict(name="gated_prefill_2048", op="gated", M=2048, K=4096, F=11008, act="silu", bias=False, train=False),
        # a training forward of a small odd-sized layer with biases: g, u, x_q and beta are kept
        dict(name="gated_train_333", op="gated", M=333, K=1088, F=2729, act="gelu", bias=True, train=True),
        # the gradients of that prompt's length on the 7B-class layer, the largest case
        dict(name="gated_bwd_2048", op="gated_bwd", M=2048, K=4096, F=11008, act="silu", bias=False),
        # the gradients of a short ragged batch on a small layer with biases
        dict(name="gated_bwd_61", op="gated_bwd", M=61, K=1024, F=2731, act="relu2", bias=True),
        # the down projection's gradients at the training length
        dict(name="linear_bwd_2048", op="linear_bwd", M=2048, K=11008, N=4096, bias=False),
        # fine-tuning on a handful of tokens: few rows, all of dW to write
        dict(name="linear_bwd_7", op="linear_bwd", M=7, K=1000, N=1023, bias=True),
        # the output head kept in 8 bits, one token
        dict(name="i8_decode_1", op="i8", M=1, K=4096, N=32000, bias=False),
        # a small batch generating through an 8-bit projection
        dict(name="i8_decode_48", op="i8", M=48, K=8192, N=8192, bias=False),
        # a long prompt through an 8-bit down projection
        dict(name="i8_prefill_2048", op="i8", M=2048, K=11008, N=4096, bias=False),
        # sizes that fit no tile: odd rows that are not aligned, with a bias
        dict(name="i8_odd_501", op="i8", M=501, K=1001, N=1537, bias=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def ternary_k():
        # widths of real layers are multiples of 64; the packing asks for multiples of 4
        return 4 * log(32, 1024) if rng.random() < 0.25 else 64 * log(4, 64)

    op = rng.choice(["gated", "gated", "gated_bwd", "linear_bwd", "i8", "i8"])
    M = log(1, 2048)
    bias = rng.random() < 0.4
    if op == "gated":
        return dict(op=op, M=M, K=ternary_k(), F=log(200, 11008), act=rng.choice(["silu", "gelu", "relu2"]),
                    bias=bias, train=rng.random() < 0.4)
    if op == "gated_bwd":
        return dict(op=op, M=M, K=ternary_k(), F=log(200, 11008), act=rng.choice(["silu", "gelu", "relu2"]), bias=bias)
    if op == "linear_bwd":
        return dict(op=op, M=M, K=ternary_k(), N=log(200, 11008), bias=bias)
    K = log(200, 11008)
    if rng.random() < 0.6:
        K = max(64, K // 64 * 64)
    return dict(op=op, M=M, K=K, N=log(200, 32000 if M <= 64 else 8192), bias=bias)


# ----------------------------------------------------------------------------- the inputs
def _activations(gen, m, k):
    x = torch.randn(m, k, device="cuda", generator=gen)
    x[torch.rand(m, k, device="cuda", generator=gen) < OUTLIER_FRACTION] *= OUTLIER_GAIN
    return x


def _gradients(gen, m, n):
    # token gradients whose sizes differ by a factor of a few, as after a mean over tokens
    size = torch.exp(0.7 * torch.randn(m, 1, device="cuda", generator=gen)) / m
    return torch.randn(m, n, device="cuda", generator=gen) * size


def _absmax_codes(t):
    """Rows of t as int8 codes and their scales: absmax + 1e-8, one rounding per step (the
    quotient of two 32-bit numbers, formed in 64 bits and rounded, is the 32-bit quotient)."""
    scale = t.abs().amax(1) + 1e-8
    q = ((t * 127.0).double() / scale.double()[:, None]).float()
    return torch.round(q).clamp(-127, 127).to(torch.int8), scale


def _ternary(gen, n, k):
    """Packed codes [n, k/4] (code W + 1 at bits 2 (k % 4)) and alpha [1] of a latent weight."""
    w = torch.randn(n, k, device="cuda", generator=gen) * W_STD
    alpha = w.abs().mean(dtype=torch.float64).float().reshape(1)
    c = (torch.round(w / alpha).clamp(-1, 1) + 1).to(torch.uint8).reshape(n, k // 4, 4)
    packed = c[:, :, 0] | (c[:, :, 1] << 2) | (c[:, :, 2] << 4) | (c[:, :, 3] << 6)
    return packed.contiguous(), alpha


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = dict(case)
    if op in ("gated", "gated_bwd"):
        F = case["F"]
        s["Wg"], s["ag"] = _ternary(gen, F, K)
        s["Wu"], s["au"] = _ternary(gen, F, K)
        s["bg"] = s["bu"] = None
        if case["bias"]:
            s["bg"] = torch.randn(F, device="cuda", generator=gen) * 0.1
            s["bu"] = torch.randn(F, device="cuda", generator=gen) * 0.1
        s["x"] = _activations(gen, M, K)
        if op == "gated":
            s["h"] = _empty(M, F)
            s["x_q"], s["beta"] = _empty(M, K, dtype=torch.int8), _empty(M)
            s["g"], s["u"] = (_empty(M, F), _empty(M, F)) if case["train"] else (None, None)
        else:
            # g and u as a forward pass leaves them: about unit size, gate and up independent
            s["g"] = torch.randn(M, F, device="cuda", generator=gen) * (0.012 * math.sqrt(K))
            s["u"] = torch.randn(M, F, device="cuda", generator=gen) * (0.012 * math.sqrt(K))
            s["x_q"], s["beta"] = _absmax_codes(s.pop("x"))
            s["dh"] = _gradients(gen, M, F)
            s["dx"], s["dWg"], s["dWu"] = _empty(M, K), _empty(F, K), _empty(F, K)
            s["dbg"], s["dbu"] = (_empty(F), _empty(F)) if case["bias"] else (None, None)
    elif op == "linear_bwd":
        N = case["N"]
        s["W"], s["alpha"] = _ternary(gen, N, K)
        s["x_q"], s["beta"] = _absmax_codes(_activations(gen, M, K))
        s["dy"] = _gradients(gen, M, N)
        s["dx"], s["dW"] = _empty(M, K), _empty(N, K)
        s["db"] = _empty(N) if case["bias"] else None
    else:
        N = case["N"]
        s["W_q"], s["gamma"] = _absmax_codes(torch.randn(N, K, device="cuda", generator=gen) * W_STD)
        s["x_q"], s["beta"] = _absmax_codes(_activations(gen, M, K))
        s["b"] = torch.randn(N, device="cuda", generator=gen) * 0.1 if case["bias"] else None
        s["y"] = _empty(M, N)
    if own:
        import bitlinear_matmul_absmean_amd as bl
        if op in ("gated", "gated_bwd"):
            s["act_code"] = {"gelu": bl.BITLINEAR_ACT_GELU, "silu": bl.BITLINEAR_ACT_SILU,
                             "relu2": bl.BITLINEAR_ACT_RELU2}[case["act"]]
        if op == "gated_bwd":
            s["ws"] = _empty(bl.bitlinear_gated_backward_workspace_size(M, K, case["F"]), dtype=torch.uint8)
        if op == "linear_bwd":
            s["ws"] = _empty(bl.bitlinear_backward_workspace_size(M, K, case["N"]), dtype=torch.uint8)
        s["bl"] = bl
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    bl, op = s["bl"], s["op"]
    if op == "gated":
        bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act_code"], bias_g=s["bg"],
                                   bias_u=s["bu"], h=s["h"], g=s["g"], u=s["u"], x_q=s["x_q"], beta=s["beta"])
        return [s["h"], s["g"], s["u"], s["x_q"], s["beta"]] if s["train"] else [s["h"]]
    if op == "gated_bwd":
        bl.bitlinear_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["Wg"], s["ag"], s["Wu"], s["au"],
                                    s["act_code"], dx=s["dx"], dWg=s["dWg"], dWu=s["dWu"], dbias_g=s["dbg"],
                                    dbias_u=s["dbu"], workspace=s["ws"])
        return [s["dx"], s["dWg"], s["dWu"]] + ([s["dbg"], s["dbu"]] if s["bias"] else [])
    if op == "linear_bwd":
        bl.bitlinear_backward(s["dy"], s["x_q"], s["beta"], s["W"], s["alpha"], dx=s["dx"], dW=s["dW"],
                              dbias=s["db"], workspace=s["ws"])
        return [s["dx"], s["dW"]] + ([s["db"]] if s["bias"] else [])
    bl.bitlinear_forward_i8(s["x_q"], s["beta"], s["W_q"], s["gamma"], bias=s["b"], y=s["y"])
    return [s["y"]]


def _unpack(packed, k):
    """Ternary weights [N, K] in 32 bits from their packed codes."""
    shifts = torch.tensor([0, 2, 4, 6], device=packed.device, dtype=torch.uint8)
    return ((packed[:, :, None] >> shifts) & 3).reshape(-1, k).float() - 1.0


def _project(x_q, beta, packed, alpha, bias):
    acc = x_q.float() @ _unpack(packed, x_q.shape[1]).t()
    y = acc * (alpha.double() * beta.double() / 127.0).float()[:, None]
    return y if bias is None else y + bias


def _act_and_slope(g, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if act == "relu2":
        r = torch.where(g > 0, g, torch.zeros_like(g))
        return r * r, 2.0 * r
    # the normal distribution's tail loses its digits in 32 bits
    g = g.double()
    phi = 0.5 * torch.erfc(-g * math.sqrt(0.5))
    return (g * phi).float(), (phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)).float()


def _run_plain(s):
    op = s["op"]
    if op == "gated":
        x_q, beta = _absmax_codes(s["x"])
        g = _project(x_q, beta, s["Wg"], s["ag"], s["bg"])
        u = _project(x_q, beta, s["Wu"], s["au"], s["bu"])
        h = _act_and_slope(g, s["act"])[0] * u
        return [h, g, u, x_q, beta] if s["train"] else [h]
    x_q, beta = s["x_q"], s["beta"]
    if op == "gated_bwd":
        a, slope = _act_and_slope(s["g"], s["act"])
        dg, du = s["dh"] * s["u"] * slope, s["dh"] * a
        xd = x_q.float() * (beta / 127.0)[:, None]
        k = x_q.shape[1]
        dx = (dg * s["ag"]) @ _unpack(s["Wg"], k) + (du * s["au"]) @ _unpack(s["Wu"], k)
        out = [dx, dg.t() @ xd, du.t() @ xd]
        return out + ([dg.sum(0), du.sum(0)] if s["bias"] else [])
    if op == "linear_bwd":
        xd = x_q.float() * (beta / 127.0)[:, None]
        out = [(s["dy"] * s["alpha"]) @ _unpack(s["W"], x_q.shape[1]), s["dy"].t() @ xd]
        return out + ([s["dy"].sum(0)] if s["bias"] else [])
    acc = x_q.float() @ s["W_q"].float().t()
    y = acc * (beta / 127.0)[:, None] * (s["gamma"] / 127.0)
    return [y if s["b"] is None else y + s["b"]]


# ------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    f64 = lambda t: t.to(D)

    def weights(packed, alpha, k):
        b = packed.to(torch.int16)
        w = torch.empty(packed.shape[0], k, dtype=D, device=packed.device)
        for i in range(4):
            w[:, i::4] = f64((b // 4 ** i) % 4 - 1)
        return w.mul_(f64(alpha))

    def activation(g):
        if case["act"] == "relu2":
            return torch.clamp(g, min=0) ** 2, 2 * torch.clamp(g, min=0)
        if case["act"] == "silu":
            sg = torch.sigmoid(g)
            return g * sg, sg + g * sg * torch.sigmoid(-g)
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) * (0.5 / math.pi) ** 0.5

    k = case["K"]
    if case["op"] == "gated":
        # the codes are defined by 32-bit steps: absmax + 1e-8, 127 x and their quotient
        x = s["x"].cpu().numpy()
        top = np.abs(x).max(axis=1)
        beta32 = (top + np.float32(1e-8)).astype(np.float32)
        codes = np.rint((x * np.float32(127)) / beta32[:, None])
        x_q = torch.from_numpy(np.clip(codes, -127, 127).astype(np.int8)).cuda()
        beta = torch.from_numpy(beta32).cuda()
        xd = f64(x_q) * f64(beta)[:, None] / 127
        g, u = xd @ weights(s["Wg"], s["ag"], k).t(), xd @ weights(s["Wu"], s["au"], k).t()
        if case["bias"]:
            g, u = g + f64(s["bg"]), u + f64(s["bu"])
        h = activation(g)[0] * u
        return [h, g, u, x_q, beta] if case["train"] else [h]
    xd = f64(s["x_q"]) * f64(s["beta"])[:, None] / 127
    if case["op"] == "gated_bwd":
        a, slope = activation(f64(s["g"]))
        dh = f64(s["dh"])
        dg, du = dh * f64(s["u"]) * slope, dh * a
        dx = dg @ weights(s["Wg"], s["ag"], k)
        dx += du @ weights(s["Wu"], s["au"], k)
        out = [dx, dg.t().contiguous() @ xd, du.t().contiguous() @ xd]
        return out + ([dg.sum(0), du.sum(0)] if case["bias"] else [])
    if case["op"] == "linear_bwd":
        dy = f64(s["dy"])
        out = [dy @ weights(s["W"], s["alpha"], k), dy.t().contiguous() @ xd]
        return out + ([dy.sum(0)] if case["bias"] else [])
    y = xd @ (f64(s["W_q"]) * f64(s["gamma"])[:, None] / 127).t()
    return [y if s["b"] is None else y + f64(s["b"])]


# --------------------------------------------------------------------------- the least work
def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "gated":
        F = case["F"]
        by = 4 * M * K + 2 * F * K // 4 + 8 + 4 * M * F
        if case["bias"]:
            by += 8 * F
        if case["train"]:
            by += 8 * M * F + M * K + 4 * M
        return {"bytes": by, "flops": 2 * M * K * 2 * F}
    if case["op"] == "gated_bwd":
        F = case["F"]
        by = 12 * M * F + M * K + 4 * M + 2 * F * K // 4 + 8 + 4 * M * K + 8 * F * K
        if case["bias"]:
            by += 8 * F
        return {"bytes": by, "flops": 2 * (2 * M * K * 2 * F)}
    N = case["N"]
    if case["op"] == "linear_bwd":
        by = 4 * M * N + M * K + 4 * M + N * K // 4 + 4 + 4 * M * K + 4 * N * K + (4 * N if case["bias"] else 0)
        return {"bytes": by, "flops": 2 * (2 * M * K * N)}
    by = M * K + 4 * M + N * K + 4 * N + 4 * M * N + (4 * N if case["bias"] else 0)
    return {"bytes": by, "flops": 2 * M * K * N}
