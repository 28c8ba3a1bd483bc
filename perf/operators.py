"""Measured cases of the norm and 8-bit operators: RMS norm with the residual's
addition (its gradient, and its form with an int8 output), the int8 row
quantizers, and the int8 matrix product with a scale for each token and channel.

``own`` false computes them as elementary torch operations in 32 bits, ``own``
true calls this package. Int8 operands are [rows][pitch], the pitch being the
columns rounded up to a multiple of 128 with zero codes in between, as the
package's quantizers write them and its users keep their weights.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    """Hidden sizes and products are those of the benchmark (4096 hidden, 6144
    query-key-value rows, 14336 feed-forward rows, 28672 gate and up rows, 8192
    tokens); the odd ones are generic."""
    return [
        # one decoded token through a block's norm: latency
        dict(name="norm 1x4096", kind="norm", rows=1, cols=4096, type="bf16"),
        # the norm in front of a linear layer, prompt-sized
        dict(name="norm 8192x4096", kind="norm", rows=8192, cols=4096, type="bf16"),
        # a training step's norm, forward and backward
        dict(name="norm train 8192x4096", kind="norm_train", rows=8192, cols=4096, type="bf16"),
        # an odd width and token count held in 32 bits (16-byte loads do not fit the rows)
        dict(name="norm train 1541x1111", kind="norm_train", rows=1541, cols=1111, type="fp32"),
        # decoding four sequences: norm, codes, query-key-value product
        dict(name="norm linear 4x6144x4096", kind="norm_linear", T=4, N=6144, K=4096, type="bf16"),
        # the same for a prompt of 2048 tokens
        dict(name="norm linear 2048x6144x4096", kind="norm_linear", T=2048, N=6144, K=4096, type="bf16"),
        # one token's down projection: the weight's bytes are everything
        dict(name="linear 1x4096x14336", kind="linear", T=1, N=4096, K=14336, type="bf16", bias=False),
        # a ragged product with a bias in half precision
        dict(name="linear 333x1537x2777", kind="linear", T=333, N=1537, K=2777, type="fp16", bias=True),
        # gate and up rows for a batch of 64 decoded tokens
        dict(name="product 64x28672x4096", kind="product", T=64, N=28672, K=4096, type="bf16"),
        # the benchmark's largest product
        dict(name="product 8192x28672x4096", kind="product", T=8192, N=28672, K=4096, type="bf16"),
        # a feed-forward block for 16 decoded tokens, and for a prompt piece
        dict(name="mlp 16 tokens", kind="mlp", T=16, F=14336, K=4096, type="bf16"),
        dict(name="mlp 512 tokens", kind="mlp", T=512, F=14336, K=4096, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "norm_linear", "linear", "product", "mlp"])
    kinds = ["bf16", "bf16", "fp16", "fp32"]
    if kind in ("norm", "norm_train"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = max(64, cols // 64 * 64)
        rows = min(_log(rng, 1, 16384), max(1, 8192 * 4096 // cols))
        return dict(kind=kind, rows=rows, cols=cols, type=rng.choice(kinds))
    K, T = _log(rng, 256, 14336), _log(rng, 1, 8192)
    if rng.random() < 0.6:
        K = K // 128 * 128
    if kind == "mlp":
        F = _log(rng, 256, 14336)
        T = min(T, 2048)
        return dict(kind=kind, T=T, F=F, K=min(K, 8192), type=rng.choice(["bf16", "fp16"]))
    N = _log(rng, 128, 28672)
    if rng.random() < 0.6:
        N = N // 64 * 64
    T = max(1, min(T, 8192 * 28672 * 4096 // (N * K)))
    case = dict(kind=kind, T=T, N=N, K=K, type=rng.choice(kinds if kind == "product" else kinds[:3]))
    if kind == "linear":
        case["bias"] = rng.random() < 0.5
    return case


def _pitch(cols):
    return (cols + 127) // 128 * 128


def _weight(n, k, g):
    """Int8 weight codes [n][pitch] and their scales, made once."""
    w = torch.randn(n, k, device="cuda", generator=g)
    a = w.abs().amax(1)
    q = torch.zeros(n, _pitch(k), dtype=torch.int8, device="cuda")
    q[:, :k] = torch.round(w * (127.0 / a)[:, None]).to(torch.int8)
    return q, a * (k ** -0.5 / 127.0)


def _activations(t, k, dtype, g):
    """Tokens of unequal size, with a few channels that stand out."""
    x = torch.randn(t, k, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(t, 1, device="cuda", generator=g))
    x *= 1 + 9 * (torch.rand(k, device="cuda", generator=g) < 0.01)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, dtype = case["kind"], TYPES[case["type"]]
    s = dict(kind=kind, dtype=dtype)
    if kind in ("norm", "norm_train"):
        t, k = case["rows"], case["cols"]
    else:
        t, k = case["T"], case["K"]
    if kind == "product":
        s["a"], sa = _weight(t, k, g)
        s["a_scales"] = sa * k ** 0.5
    else:
        s["x"] = _activations(t, k, dtype, g)
    if kind != "linear" and kind != "product":
        s["res"] = _activations(t, k, dtype, g)
        s["norm_w"] = (1 + 0.2 * torch.randn(k, device="cuda", generator=g)).to(dtype)
    if kind == "norm_train":
        s["dy"] = torch.randn(t, k, device="cuda", generator=g).to(dtype)
        s["dh"] = torch.randn(t, k, device="cuda", generator=g).to(dtype)
        for n in ("x", "res", "norm_w"):
            s[n].requires_grad_(True)
    if kind in ("norm_linear", "linear", "product"):
        s["w"], s["w_scales"] = _weight(case["N"], k, g)
    s["bias"] = torch.randn(case["N"], device="cuda", generator=g) if case.get("bias") else None
    if kind == "mlp":
        s["gu"], s["gu_scales"] = _weight(2 * case["F"], k, g)
        s["down"], s["down_scales"] = _weight(k, case["F"], g)
    return s


# ------------------------------------------------------------ plain forms
def _norm(x, res, w):
    """(h in its type, the normalised row times the weight in 32 bits, the row's factor)."""
    h = (x.float() + res.float()).to(x.dtype)
    hf = h.float()
    r = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    return h, hf * r * w.float(), r


def _codes(y):
    """Int8 codes (as 32-bit numbers, zeros up to the pitch) and scales of the rows of y."""
    a = y.abs().amax(1, keepdim=True)
    q = torch.round(y * torch.where(a > 0, 127.0 / a, 0.0))
    return torch.nn.functional.pad(q, (0, _pitch(y.shape[1]) - y.shape[1])), a / 127.0


def _product(q, sq, w, sw, bias, dtype):
    c = (q @ w.float().t()) * sq * sw
    return (c if bias is None else c + bias).to(dtype)


def _plain(s):
    kind, dtype = s["kind"], s["dtype"]
    if kind == "product":
        return {"c": _product(s["a"].float(), s["a_scales"][:, None], s["w"], s["w_scales"], None, dtype)}
    if kind == "linear":
        q, sq = _codes(s["x"].float())
        return {"c": _product(q, sq, s["w"], s["w_scales"], s["bias"], dtype)}
    with torch.no_grad():
        h, y, r = _norm(s["x"], s["res"], s["norm_w"])
        if kind == "norm":
            return {"y": y.to(dtype), "h": h}
        if kind == "norm_train":
            dy, xh = s["dy"].float(), h.float() * r
            d = dy * s["norm_w"].float()
            dx = (r * (d - xh * (d * xh).mean(1, keepdim=True)) + s["dh"].float()).to(dtype)
            return {"y": y.to(dtype), "h": h, "dx": dx, "dres": dx, "dw": (dy * xh).sum(0).to(dtype)}
        q, sq = _codes(y)
        if kind == "norm_linear":
            return {"c": _product(q, sq, s["w"], s["w_scales"], None, dtype), "h": h}
        gu = _product(q, sq, s["gu"], s["gu_scales"], None, dtype).float()
        gate, up = gu.chunk(2, dim=1)
        q, sq = _codes(gate / (1 + torch.exp(-gate)) * up)
        return {"c": _product(q, sq, s["down"], s["down_scales"], None, dtype), "h": h}


# ------------------------------------------------------ this package's calls
def _own(s):
    from mxfp4_quantized_gemm_amd import int8, norm
    kind, dtype = s["kind"], s["dtype"]
    if kind == "norm":
        y, h = norm.rms_norm(s["x"], s["norm_w"], EPS, residual=s["res"])
        return {"y": y, "h": h}
    if kind == "norm_train":
        y, h = norm.rms_norm(s["x"], s["norm_w"], EPS, residual=s["res"])
        dx, dres, dw = torch.autograd.grad((y, h), (s["x"], s["res"], s["norm_w"]), (s["dy"], s["dh"]))
        return {"y": y, "h": h, "dx": dx, "dres": dres, "dw": dw}
    if kind == "norm_linear":
        q, sq, h = norm.rms_norm_int8(s["x"], s["norm_w"], EPS, residual=s["res"])
        return {"c": int8.int8_gemm(q, sq, s["w"], s["w_scales"], out_dtype=dtype), "h": h}
    if kind == "linear":
        return {"c": int8.int8_linear(s["x"], s["w"], s["w_scales"], bias=s["bias"])}
    if kind == "product":
        return {"c": int8.int8_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"], out_dtype=dtype)}
    c, h = int8.int8_mlp(s["x"], s["norm_w"], EPS, s["gu"], s["gu_scales"], s["down"], s["down_scales"],
                         residual=s["res"])
    return {"c": c, "h": h}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind, e = case["kind"], SIZE[case["type"]]
    if kind in ("norm", "norm_train"):
        n, k = case["rows"] * case["cols"], case["cols"]
        if kind == "norm":  # x, res, weight in; y, h out
            return {"bytes": 4 * n * e + k * e, "flops": 6 * n}
        # the gradients of y and h in too, one gradient of x and res and the weight's out
        return {"bytes": 7 * n * e + 2 * k * e, "flops": 18 * n}
    T, K = case["T"], case["K"]
    if kind == "mlp":
        F = case["F"]
        return {"bytes": 3 * F * K + 4 * (2 * F + K) + 4 * T * K * e + K * e, "flops": 6 * T * F * K}
    N = case["N"]
    b = N * K + 4 * N + T * N * e
    b += {"norm_linear": 3 * T * K * e + K * e, "linear": T * K * e, "product": T * K + 4 * T}[kind]
    return {"bytes": b + (4 * N if case.get("bias") else 0), "flops": 2 * T * N * K}


# ------------------------------------------------------------- 64 bits
def _exact_rows(v):
    """Codes and scales of rows given in 64 bits: the nearest multiple of a 127th of the row's largest magnitude."""
    top = v.abs().max(dim=1).values.unsqueeze(1)
    step = top / 127
    return torch.round(v / torch.where(step > 0, step, torch.ones_like(step))), step


def _exact_dot(q, step, w, ws):
    w64 = w.double()[:, : q.shape[1]]
    return torch.mm(q, w64.t()) * step * ws.double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, dtype = case["kind"], s["dtype"]
    with torch.no_grad():
        if kind == "product":
            return {"c": _exact_dot(s["a"].double(), s["a_scales"].double()[:, None], s["w"], s["w_scales"])}
        if kind == "linear":
            c = _exact_dot(*_exact_rows(s["x"].double()), s["w"], s["w_scales"])
            return {"c": c if s["bias"] is None else c + s["bias"].double()}
        # the residual stream is held in the inputs' type, and the norm reads it as held
        h = (s["x"].double() + s["res"].double()).to(dtype).double()
        w = s["norm_w"].double()
        size = torch.sqrt(torch.mean(h * h, dim=1, keepdim=True) + EPS)
        y = h / size * w
        if kind == "norm":
            return {"y": y, "h": h}
        if kind == "norm_train":
            dy = s["dy"].double()
            unit = h / size
            dunit = dy * w
            # d unit / d h = (I - unit unit^T / cols) / size
            dh = (dunit - unit * torch.sum(dunit * unit, dim=1, keepdim=True) / h.shape[1]) / size + s["dh"].double()
            return {"y": y, "h": h, "dx": dh, "dres": dh, "dw": torch.sum(dy * unit, dim=0)}
        q, step = _exact_rows(y)
        if kind == "norm_linear":
            return {"c": _exact_dot(q, step, s["w"], s["w_scales"]), "h": h}
        gu = _exact_dot(q, step, s["gu"], s["gu_scales"]).to(dtype).double()  # held in the inputs' type
        f = case["F"]
        q, step = _exact_rows(gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:])
        return {"c": _exact_dot(q, step, s["down"], s["down_scales"]), "h": h}
