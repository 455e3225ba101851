"""Workloads of the products grouped by expert and of the product in 8-bit floating point.

Operators of a layer of ternary experts and of the projections beside them, each with its plain
form in elementary torch operations and the call that a user makes of the library:

  grouped      y = BitLinear of the row's expert, rows sorted by expert, any number for each
  gated        h = act(g) * u of the row's expert, from fp32 tokens; training calls keep g, u, x_q, beta
  grouped_bwd  gradients of grouped: dx of every row, dW and dbias of every expert
  gated_bwd    gradients of gated
  fp8          x quantized to e4m3 in blocks of 128 and multiplied with e4m3 weights that have a
               scale for each block of 128 x 128
  fp8_weights  the quantizer of those weights

Tokens choose `top` of `E` experts by logits that favour some experts over others; a row is one
choice, `rows` holds its token.  Weights, activations and gradients are distributed as in
perf/operators.py: N(0, 0.02) latent weights, N(0, 1) activations with one element in a thousand
20 times larger, gradients whose size differs from token to token.
"""
import math

import numpy as np
import torch

own = False

W_STD = 0.02
OUTLIER_FRACTION = 0.001
OUTLIER_GAIN = 20.0
BLOCK = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence generating through a layer of 8 experts, 7B-class sizes: latency counts
        dict(name="gated_decode_1", op="gated", T=1, top=2, E=8, K=4096, F=11008, act="silu", bias=False, train=False),
        # a long prompt through 16 smaller experts: the integer products count
        dict(name="gated_prefill_2048", op="gated", T=2048, top=4, E=16, K=2048, F=2816, act="silu", bias=False, train=False),
        # the down projections while sixteen sequences generate: a few rows for each expert
        dict(name="grouped_decode_16", op="grouped", T=16, top=4, E=16, K=2816, N=2048, bias=False, gather=False),
        # a ragged batch at odd sizes with biases, rows gathered from their tokens
        dict(name="grouped_odd_501", op="grouped", T=501, top=3, E=7, K=1088, N=1537, bias=True, gather=True),
        # a training step of the gated experts, the largest case
        dict(name="gated_bwd_2048", op="gated_bwd", T=2048, top=2, E=8, K=2048, F=2816, act="silu", bias=False),
        # a short ragged batch with biases
        dict(name="gated_bwd_61", op="gated_bwd", T=61, top=2, E=5, K=1024, F=2731, act="relu2", bias=True),
        # the down projections' gradients of that step
        dict(name="grouped_bwd_2048", op="grouped_bwd", T=2048, top=2, E=8, K=2816, N=2048, bias=False, gather=False),
        # fine-tuning on a handful of tokens: few rows, all of dW to write
        dict(name="grouped_bwd_7", op="grouped_bwd", T=7, top=2, E=4, K=1000, N=1023, bias=True, gather=True),
        # the output head in fp8, one token
        dict(name="fp8_decode_1", op="fp8", M=1, K=4096, N=32000, bias=False),
        # a long prompt through a down projection in fp8
        dict(name="fp8_prefill_2048", op="fp8", M=2048, K=11008, N=4096, bias=False),
        # loading that projection: its weights quantized
        dict(name="fp8_weights_4096", op="fp8_weights", N=4096, K=11008),
        # a matrix whose last blocks are not whole
        dict(name="fp8_weights_odd", op="fp8_weights", N=1537, K=1001),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def ternary_k(hi):
        # widths of real layers are multiples of 64; the packing asks for multiples of 4
        return 4 * log(32, hi // 4) if rng.random() < 0.25 else 64 * log(4, hi // 64)

    op = rng.choice(["gated", "grouped", "gated_bwd", "grouped_bwd", "fp8", "fp8", "fp8_weights"])
    if op == "fp8":
        K = log(128, 11008)
        if rng.random() < 0.6:
            K = K // 128 * 128
        M = log(1, 2048)
        return dict(op=op, M=M, K=K, N=log(128, 32000 if M <= 64 else 4096), bias=rng.random() < 0.4)
    if op == "fp8_weights":
        return dict(op=op, N=log(100, 8192), K=log(100, 8192))
    E = log(2, 64)
    top = rng.randint(1, min(E, 8))
    T = log(1, max(1, 4096 // top))
    c = dict(op=op, T=T, top=top, E=E, K=ternary_k(2048), bias=rng.random() < 0.4)
    # all experts' weights within 2^26 elements a matrix
    width = log(200, max(201, min(2816, (1 << 26) // (E * c["K"]))))
    if op in ("gated", "gated_bwd"):
        c.update(F=width, act=rng.choice(["silu", "gelu", "relu2"]))
        if op == "gated":
            c["train"] = rng.random() < 0.4
    else:
        c.update(N=width, gather=rng.random() < 0.5)
    return c


# ----------------------------------------------------------------------------- the inputs
def _activations(gen, m, k):
    x = torch.randn(m, k, device="cuda", generator=gen)
    x[torch.rand(m, k, device="cuda", generator=gen) < OUTLIER_FRACTION] *= OUTLIER_GAIN
    return x


def _gradients(gen, m, n):
    size = torch.exp(0.7 * torch.randn(m, 1, device="cuda", generator=gen)) / m
    return torch.randn(m, n, device="cuda", generator=gen) * size


def _absmax_codes(t):
    """Rows of t as int8 codes and their scales: absmax + 1e-8, one rounding per step (the
    quotient of two 32-bit numbers, formed in 64 bits and rounded, is the 32-bit quotient)."""
    scale = t.abs().amax(1) + 1e-8
    q = ((t * 127.0).double() / scale.double()[:, None]).float()
    return torch.round(q).clamp(-127, 127).to(torch.int8), scale


def _experts(gen, e, n, k):
    """Packed codes [e, n, k/4] (code W + 1 at bits 2 (k % 4)) and alpha [e] of latent weights."""
    packed = torch.empty(e, n, k // 4, dtype=torch.uint8, device="cuda")
    alpha = torch.empty(e, device="cuda")
    for i in range(e):
        w = torch.randn(n, k, device="cuda", generator=gen) * W_STD
        alpha[i] = w.abs().mean(dtype=torch.float64).float()
        c = (torch.round(w / alpha[i]).clamp(-1, 1) + 1).to(torch.uint8).reshape(n, k // 4, 4)
        packed[i] = c[:, :, 0] | (c[:, :, 1] << 2) | (c[:, :, 2] << 4) | (c[:, :, 3] << 6)
    return packed, alpha


def _routes(gen, t, top, e):
    """rows [t top] and offsets [e + 1]: every token's choices, sorted by expert."""
    logits = torch.randn(t, e, device="cuda", generator=gen) + 0.5 * torch.randn(e, device="cuda", generator=gen)
    chosen = logits.topk(top, dim=1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(chosen, minlength=e), 0)
    return order // top, offsets


def _round_e4m3(v):
    """Values in [-448, 448] rounded to e4m3 (ties to even), as the 8-bit type."""
    return v.to(torch.float8_e4m3fn)


def _quantize_blocks(t, high):
    """t [R, K] in e4m3 with a scale absmax / 448 for each block of `high` x 128: codes [R, K] and
    scales [ceil(R / high), ceil(K / 128)].  A block of zeros has scale 0 and codes 0."""
    r, k = t.shape
    nr, nk = -(-r // high), -(-k // BLOCK)
    p = torch.zeros(nr * high, nk * BLOCK, device=t.device)
    p[:r, :k] = t
    p = p.reshape(nr, high, nk, BLOCK)
    scale = (p.abs().amax((1, 3)).double() / E4M3_MAX).float()
    s = scale[:, None, :, None]
    q = (p.double() / torch.where(s > 0, s, torch.ones_like(s)).double()).float().clamp(-E4M3_MAX, E4M3_MAX)
    codes = _round_e4m3(q.reshape(nr * high, nk * BLOCK)[:r, :k].contiguous())
    return codes, scale


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, K = case["op"], case["K"]
    s = dict(case)
    if op == "fp8_weights":
        N = case["N"]
        s["W"] = torch.randn(N, K, device="cuda", generator=gen) * W_STD
        s["W_q"], s["W_scale"] = _empty(N, K, dtype=torch.float8_e4m3fn), _empty(-(-N // BLOCK), -(-K // BLOCK))
    elif op == "fp8":
        M, N = case["M"], case["N"]
        s["x"] = _activations(gen, M, K)
        s["W_q"], s["W_scale"] = _quantize_blocks(torch.randn(N, K, device="cuda", generator=gen) * W_STD, BLOCK)
        s["b"] = torch.randn(N, device="cuda", generator=gen) * 0.1 if case["bias"] else None
        s["x_q"], s["x_scale"] = _empty(M, K, dtype=torch.float8_e4m3fn), _empty(-(-K // BLOCK), M)
        s["y"] = _empty(M, N)
    else:
        T, top, E = case["T"], case["top"], case["E"]
        M = T * top
        rows, s["offsets"] = _routes(gen, T, top, E)
        s["cuts"] = s["offsets"].tolist()          # the plain forms' loop over experts is on the host
        gather = op in ("gated", "gated_bwd") or case["gather"]
        s["rows"] = rows if gather else None
        x = _activations(gen, T if gather else M, K)
        if op in ("gated", "gated_bwd"):
            F = case["F"]
            s["Wg"], s["ag"] = _experts(gen, E, F, K)
            s["Wu"], s["au"] = _experts(gen, E, F, K)
            s["bg"] = s["bu"] = None
            if case["bias"]:
                s["bg"] = torch.randn(E, F, device="cuda", generator=gen) * 0.1
                s["bu"] = torch.randn(E, F, device="cuda", generator=gen) * 0.1
            if op == "gated":
                s["x"], s["h"] = x, _empty(M, F)
                s["x_q"], s["beta"] = _empty(T, K, dtype=torch.int8), _empty(T)
                s["g"], s["u"] = (_empty(M, F), _empty(M, F)) if case["train"] else (None, None)
            else:
                # g and u as a forward pass leaves them: about unit size, gate and up independent
                s["g"] = torch.randn(M, F, device="cuda", generator=gen) * (0.012 * math.sqrt(K))
                s["u"] = torch.randn(M, F, device="cuda", generator=gen) * (0.012 * math.sqrt(K))
                s["x_q"], s["beta"] = _absmax_codes(x)
                s["dh"] = _gradients(gen, M, F)
                s["dx"], s["dWg"], s["dWu"] = _empty(M, K), _empty(E, F, K), _empty(E, F, K)
                s["dbg"], s["dbu"] = (_empty(E, F), _empty(E, F)) if case["bias"] else (None, None)
        else:
            N = case["N"]
            s["W"], s["alpha"] = _experts(gen, E, N, K)
            s["x_q"], s["beta"] = _absmax_codes(x)
            if op == "grouped":
                s["b"] = torch.randn(E, N, device="cuda", generator=gen) * 0.1 if case["bias"] else None
                s["y"] = _empty(M, N)
            else:
                s["dy"] = _gradients(gen, M, N)
                s["dx"], s["dW"] = _empty(M, K), _empty(E, N, K)
                s["db"] = _empty(E, N) if case["bias"] else None
    if own:
        import bitlinear_matmul_absmean_amd as bl
        if op in ("gated", "gated_bwd"):
            s["act_code"] = {"gelu": bl.BITLINEAR_ACT_GELU, "silu": bl.BITLINEAR_ACT_SILU,
                             "relu2": bl.BITLINEAR_ACT_RELU2}[case["act"]]
        if op == "gated_bwd":
            s["ws"] = _empty(bl.bitlinear_grouped_gated_backward_workspace_size(case["T"] * case["top"], K, case["F"],
                                                                                case["E"]), dtype=torch.uint8)
        if op == "grouped_bwd":
            s["ws"] = _empty(bl.bitlinear_grouped_backward_workspace_size(case["T"] * case["top"], K, case["N"],
                                                                          case["E"]), dtype=torch.uint8)
        s["bl"] = bl
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    bl, op = s["bl"], s["op"]
    if op == "gated":
        bl.bitlinear_grouped_gated_forward(s["x"], s["offsets"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act_code"],
                                           rows=s["rows"], bias_g=s["bg"], bias_u=s["bu"], h=s["h"], g=s["g"], u=s["u"],
                                           x_q=s["x_q"], beta=s["beta"])
        return [s["h"], s["g"], s["u"], s["x_q"], s["beta"]] if s["train"] else [s["h"]]
    if op == "grouped":
        bl.bitlinear_grouped_forward(s["x_q"], s["beta"], s["offsets"], s["W"], s["alpha"], rows=s["rows"], bias=s["b"],
                                     y=s["y"])
        return [s["y"]]
    if op == "gated_bwd":
        bl.bitlinear_grouped_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["offsets"], s["Wg"], s["ag"],
                                            s["Wu"], s["au"], s["act_code"], rows=s["rows"], dx=s["dx"], dWg=s["dWg"],
                                            dWu=s["dWu"], dbias_g=s["dbg"], dbias_u=s["dbu"], workspace=s["ws"])
        return [s["dx"], s["dWg"], s["dWu"]] + ([s["dbg"], s["dbu"]] if s["bias"] else [])
    if op == "grouped_bwd":
        bl.bitlinear_grouped_backward(s["dy"], s["x_q"], s["beta"], s["offsets"], s["W"], s["alpha"], rows=s["rows"],
                                      dx=s["dx"], dW=s["dW"], dbias=s["db"], workspace=s["ws"])
        return [s["dx"], s["dW"]] + ([s["db"]] if s["bias"] else [])
    if op == "fp8":
        bl.bitlinear_quantize_act_fp8(s["x"], x_q=s["x_q"], x_scale=s["x_scale"])
        bl.bitlinear_forward_fp8(s["x_q"], s["x_scale"], s["W_q"], s["W_scale"], bias=s["b"], y=s["y"])
        return [s["y"]]
    bl.bitlinear_quantize_weights_fp8(s["W"], W_q=s["W_q"], W_scale=s["W_scale"])
    return [s["W_q"].float(), s["W_scale"]]


def _unpack(packed, k):
    """Ternary weights [N, K] in 32 bits from their packed codes."""
    shifts = torch.tensor([0, 2, 4, 6], device=packed.device, dtype=torch.uint8)
    return ((packed[:, :, None] >> shifts) & 3).reshape(-1, k).float() - 1.0


def _groups(s):
    """(expert, first row, end) of every expert that has rows."""
    c = s["cuts"]
    return [(e, c[e], c[e + 1]) for e in range(len(c) - 1) if c[e + 1] > c[e]]


def _project(s, x_q, beta, packed, alpha, bias):
    """Rows of x_q under their experts' weights."""
    y = _empty(x_q.shape[0], packed.shape[1])
    for e, i, j in _groups(s):
        acc = x_q[i:j].float() @ _unpack(packed[e], x_q.shape[1]).t()
        v = acc * (alpha[e].double() * beta[i:j].double() / 127.0).float()[:, None]
        y[i:j] = v if bias is None else v + bias[e]
    return y


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


def _gradients_of(s, pairs, x_q, beta):
    """dx, then dW and dbias of each (d, packed, alpha) of `pairs`, over the experts."""
    k = x_q.shape[1]
    dx = torch.zeros(x_q.shape[0], k, device=x_q.device)
    dws = [torch.zeros(p.shape[0], p.shape[1], k, device=x_q.device) for _, p, _ in pairs]
    dbs = [torch.zeros(p.shape[0], p.shape[1], device=x_q.device) for _, p, _ in pairs]
    xd = x_q.float() * (beta / 127.0)[:, None]
    for e, i, j in _groups(s):
        for n, (d, packed, alpha) in enumerate(pairs):
            dx[i:j] += (d[i:j] * alpha[e]) @ _unpack(packed[e], k)
            dws[n][e] = d[i:j].t() @ xd[i:j]
            if s["bias"]:
                dbs[n][e] = d[i:j].sum(0)
    return [dx] + dws + (dbs if s["bias"] else [])


def _run_plain(s):
    op = s["op"]
    if op == "fp8_weights":
        codes, scale = _quantize_blocks(s["W"], BLOCK)
        return [codes.float(), scale]
    if op == "fp8":
        x_q, x_scale = _quantize_blocks(s["x"], 1)
        k, n = x_q.shape[1], s["W_q"].shape[0]
        xd = x_q.float() * x_scale.repeat_interleave(BLOCK, 1)[:, :k]
        wd = s["W_q"].float() * s["W_scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
        y = xd @ wd.t()
        return [y if s["b"] is None else y + s["b"]]
    if op == "gated":
        codes, scales = _absmax_codes(s["x"])
        x_q, beta = codes[s["rows"]], scales[s["rows"]]
        g = _project(s, x_q, beta, s["Wg"], s["ag"], s["bg"])
        u = _project(s, x_q, beta, s["Wu"], s["au"], s["bu"])
        h = _act_and_slope(g, s["act"])[0] * u
        return [h, g, u, codes, scales] if s["train"] else [h]
    x_q, beta = (s["x_q"], s["beta"]) if s["rows"] is None else (s["x_q"][s["rows"]], s["beta"][s["rows"]])
    if op == "grouped":
        return [_project(s, x_q, beta, s["W"], s["alpha"], s["b"])]
    if op == "grouped_bwd":
        return _gradients_of(s, [(s["dy"], s["W"], s["alpha"])], x_q, beta)
    a, slope = _act_and_slope(s["g"], s["act"])
    return _gradients_of(s, [(s["dh"] * s["u"] * slope, s["Wg"], s["ag"]), (s["dh"] * a, s["Wu"], s["au"])], x_q, beta)


# ------------------------------------------------------------------------ 64-bit values
def _e4m3_values(q):
    """64-bit values of q in [-448, 448] rounded to a sign, four significant bits and exponents from -6 up."""
    m = np.abs(q)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(m, 2.0 ** -40))), -6) - 3)
    return np.copysign(np.rint(m / step) * step, q)


def _exact_blocks(t, high):
    """Codes' values and scales of t (64-bit arrays) by the definition: 32-bit scale, 32-bit quotient, e4m3."""
    t = t.cpu().numpy()
    r, k = t.shape
    values = np.zeros((r, k))
    scales = np.zeros((-(-r // high), -(-k // BLOCK)))
    for b in range(scales.shape[1]):
        part = t[:, b * BLOCK:(b + 1) * BLOCK]
        for i in ([0] if high == 1 else range(scales.shape[0])):
            blk = part if high == 1 else part[i * high:(i + 1) * high]
            s = np.abs(blk).max(1, keepdims=True) if high == 1 else np.abs(blk).max().reshape(1, 1)
            s = (s / np.float32(E4M3_MAX)).astype(np.float32)
            q = np.divide(blk, s, out=np.zeros_like(blk), where=s > 0)
            v = _e4m3_values(np.clip(q, -E4M3_MAX, E4M3_MAX).astype(np.float64))
            if high == 1:
                values[:, b * BLOCK:(b + 1) * BLOCK], scales[:, b] = v, s[:, 0]
            else:
                values[i * high:(i + 1) * high, b * BLOCK:(b + 1) * BLOCK], scales[i, b] = v, s[0, 0]
    return torch.from_numpy(values).cuda(), torch.from_numpy(scales).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    f64 = lambda t: t.to(D)
    op, k = case["op"], case["K"]
    if op == "fp8_weights":
        return list(_exact_blocks(s["W"], BLOCK))
    if op == "fp8":
        v, sc = _exact_blocks(s["x"], 1)
        y = torch.zeros(case["M"], case["N"], dtype=D, device="cuda")
        for b in range(sc.shape[1]):
            cut = slice(b * BLOCK, (b + 1) * BLOCK)
            ws = f64(s["W_scale"][:, b])[torch.arange(case["N"], device="cuda") // BLOCK]
            y += (v[:, cut] * sc[:, b:b + 1]) @ (f64(s["W_q"][:, cut].float()) * ws[:, None]).t()
        return [y if s["b"] is None else y + f64(s["b"])]

    def weights(packed, alpha):
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

    if op == "gated":
        # the codes are defined by 32-bit steps: absmax + 1e-8, 127 x and their quotient
        x = s["x"].cpu().numpy()
        beta32 = (np.abs(x).max(axis=1) + np.float32(1e-8)).astype(np.float32)
        codes = np.clip(np.rint((x * np.float32(127)) / beta32[:, None]), -127, 127).astype(np.int8)
        s["x_q"], s["beta"] = torch.from_numpy(codes).cuda(), torch.from_numpy(beta32).cuda()
    xd = f64(s["x_q"]) * f64(s["beta"])[:, None] / 127
    if s["rows"] is not None:
        xd = xd[s["rows"]]
    M, E = xd.shape[0], case["E"]
    of = torch.bucketize(torch.arange(M, device="cuda"), s["offsets"][1:], right=True)

    def forward(packed, alpha, bias):
        y = torch.empty(M, packed.shape[1], dtype=D, device="cuda")
        for e in range(E):
            y[of == e] = xd[of == e] @ weights(packed[e], alpha[e]).t()
        return y if bias is None else y + f64(bias)[of]

    if op == "grouped":
        return [forward(s["W"], s["alpha"], s["b"])]
    if op == "gated":
        g, u = forward(s["Wg"], s["ag"], s["bg"]), forward(s["Wu"], s["au"], s["bu"])
        h = activation(g)[0] * u
        return [h, g, u, s["x_q"], s["beta"]] if case["train"] else [h]
    if op == "grouped_bwd":
        parts = [(f64(s["dy"]), s["W"], s["alpha"])]
    else:
        a, slope = activation(f64(s["g"]))
        dh = f64(s["dh"])
        parts = [(dh * f64(s["u"]) * slope, s["Wg"], s["ag"]), (dh * a, s["Wu"], s["au"])]
    dx = torch.zeros(M, k, dtype=D, device="cuda")
    dws = [torch.zeros(p.shape[0], p.shape[1], k, dtype=D, device="cuda") for _, p, _ in parts]
    dbs = [torch.zeros(p.shape[0], p.shape[1], dtype=D, device="cuda") for _, p, _ in parts]
    for e in range(E):
        mine = of == e
        for n, (d, packed, alpha) in enumerate(parts):
            dx[mine] += d[mine] @ weights(packed[e], alpha[e])
            dws[n][e] = d[mine].t().contiguous() @ xd[mine]
            dbs[n][e] = d[mine].sum(0)
    return [dx] + dws + (dbs if case["bias"] else [])


# --------------------------------------------------------------------------- the least work
def work(case):
    op, K = case["op"], case["K"]
    if op == "fp8_weights":
        N = case["N"]
        return {"bytes": 5 * N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK), "flops": 2 * N * K}
    if op == "fp8":
        M, N = case["M"], case["N"]
        by = 4 * M * K + N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK) + 4 * M * N + (4 * N if case["bias"] else 0)
        return {"bytes": by, "flops": 2 * M * K * N}
    T, top, E = case["T"], case["top"], case["E"]
    M = T * top
    used = E * (1 - (1 - top / E) ** T)            # experts that some token chose, on average
    gather = op in ("gated", "gated_bwd") or case["gather"]
    tokens = T if gather else M
    by = 8 * (E + 1) + (8 * M if gather else 0)
    if op == "gated":
        F = case["F"]
        by += 4 * T * K + used * (2 * F * K // 4 + 8 + (8 * F if case["bias"] else 0)) + 4 * M * F
        if case["train"]:
            by += 8 * M * F + T * K + 4 * T
        return {"bytes": int(by), "flops": 2 * M * K * 2 * F}
    if op == "grouped":
        N = case["N"]
        by += tokens * (K + 4) + used * (N * K // 4 + 4 + (4 * N if case["bias"] else 0)) + 4 * M * N
        return {"bytes": int(by), "flops": 2 * M * K * N}
    if op == "gated_bwd":
        F = case["F"]
        by += 12 * M * F + T * (K + 4) + used * (2 * F * K // 4 + 8) + 4 * M * K + E * (8 * F * K + (8 * F if case["bias"] else 0))
        return {"bytes": int(by), "flops": 2 * (2 * M * K * 2 * F)}
    N = case["N"]
    by += 4 * M * N + tokens * (K + 4) + used * (N * K // 4 + 4) + 4 * M * K + E * (4 * N * K + (4 * N if case["bias"] else 0))
    return {"bytes": int(by), "flops": 2 * (2 * M * K * N)}
