"""Measured cases of attention's operators: the norm of each head of queries and
keys with their rotation (its gradient, several position axes), an int8 cache of
keys and values as it is written and read back, attention of one new token a
sequence over that cache in pages, and the 8-bit attention block that calls them.

``own`` false computes them as elementary torch operations in 32 bits, ``own``
true calls this package. A cache is (k, k_scales, v, v_scales): int8 codes
[pages][heads][page size][pitch], the pitch being the head's width rounded up to
a multiple of 64 with zero codes in between, and fp32 scales [pages][heads][page
size]. Int8 weights are [rows][pitch], padded to a multiple of 128.
"""
import math

import torch

own = False

EPS = 1e-5       # of the block's norm
QK_EPS = 1e-6    # of the heads' norms
BASE = 500000.0  # of the rotation's frequencies
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    """4096 hidden, 6144 query-key-value rows (32 + 8 + 8 heads of 128) and 8192
    tokens are the benchmark's; the others are generic."""
    return [
        # queries and keys of four decoded tokens: latency
        dict(name="qk 4 tokens", kind="qk", T=4, H=32, KV=8, D=128, rot=128, norm=True, axes=1, inter=False, type="bf16"),
        # a training step's queries and keys, forward and backward
        dict(name="qk train 8192 tokens", kind="qk_train", T=8192, H=32, KV=8, D=128, rot=128, norm=True, axes=1,
             inter=False, type="bf16"),
        # time, height and width of image patches, part of an 80-wide head rotated in neighbouring pairs, held in 32 bits
        dict(name="qk train 1541x9 of 80", kind="qk_train", T=1541, H=9, KV=3, D=80, rot=60, norm=True, axes=3,
             inter=True, type="fp32"),
        # 16 sequences' new tokens: norm, rotation and codes into the cache, read back
        dict(name="append 16 tokens", kind="append", T=16, H=32, KV=8, D=128, rot=128, norm=True, axes=1, inter=False,
             page=64, type="bf16"),
        # a prompt's
        dict(name="append 8192 tokens", kind="append", T=8192, H=32, KV=8, D=128, rot=128, norm=True, axes=1,
             inter=False, page=64, type="bf16"),
        # keys and values that are rotated already, an odd number of tokens, small pages
        dict(name="write 3001x5 of 96", kind="write", T=3001, KV=5, D=96, page=16, type="fp16"),
        # a cached prefix read back
        dict(name="read 32768 tokens", kind="read", T=32768, KV=8, D=128, page=64, type="bf16"),
        # one sequence of ordinary length: latency
        dict(name="attention 1x1000", kind="attention", B=1, L=1000, H=32, KV=8, D=128, page=64, ragged=False, window=0,
             type="bf16"),
        # a serving batch
        dict(name="attention 64x8192", kind="attention", B=64, L=8192, H=32, KV=8, D=128, page=64, ragged=False,
             window=0, type="bf16"),
        # one long document
        dict(name="attention 1x131072", kind="attention", B=1, L=131072, H=32, KV=8, D=128, page=64, ragged=False,
             window=0, type="bf16"),
        # sequences of all lengths (empty ones too) behind a sliding window, seven queries a key head
        dict(name="attention 37 ragged", kind="attention", B=37, L=20011, H=14, KV=2, D=64, page=16, ragged=True,
             window=4096, type="fp16"),
        # the attention block for 16 decoded tokens
        dict(name="block 16x2048", kind="block", B=16, L=2048, H=32, KV=8, D=128, K=4096, page=64, ragged=True,
             window=0, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    return kv, kv * rng.choice([g for g in (1, 2, 3, 4, 4, 5, 7, 8, 12, 16) if kv * g <= 64])


def draw(rng):
    kind = rng.choice(["qk", "qk_train", "append", "write", "read", "attention", "attention", "attention", "block"])
    kv, h = _heads(rng)
    d = rng.choice([64, 80, 96, 112, 128, 128, 128, 192, 256])
    case = dict(kind=kind, KV=kv, D=d)
    if kind in ("qk", "qk_train", "append"):
        axes = rng.choice([1, 1, 2, 3])
        rot = d if rng.random() < 0.6 else 2 * rng.randint(max(axes, d // 8), d // 2)
        case.update(H=h, rot=rot, axes=axes, norm=rng.random() < 0.7, inter=rng.random() < 0.3)
    if kind in ("qk", "qk_train"):
        case["T"] = max(1, min(_log(rng, 1, 32768), 8192 * 40 * 128 // ((h + kv) * d)))
        case["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return case
    case["page"] = rng.choice([16, 32, 48, 64, 128, 256])
    if kind in ("append", "write", "read"):
        most = 8192 * 40 * 128 // ((h + kv) * d) if kind == "append" else 32768 * 8 * 128 // (kv * d)
        case["T"] = max(1, min(_log(rng, 1, 32768), most))
        case["type"] = rng.choice(["bf16", "bf16", "fp16"])
        return case
    case.update(H=h, ragged=rng.random() < 0.6, window=rng.choice([0, 0, 0, rng.randint(1, 9000)]))
    if kind == "attention":
        case["L"] = _log(rng, 1, 131072)
        case["B"] = max(1, min(_log(rng, 1, 300), 64 * 8192 * 8 * 128 // (case["L"] * kv * d)))
        case["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return case
    case.update(L=_log(rng, 1, 8192), K=64 * rng.randint(8, 64), type=rng.choice(["bf16", "fp16"]))
    case["B"] = max(1, min(_log(rng, 1, 64), 64 * 2048 * 8 * 128 // (case["L"] * kv * d)))
    return case


# --------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens of each sequence: all L, or spread over their logarithm from 1 to L with every eighth sequence empty."""
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    n = [max(1, int(round(case["L"] ** ((i * 0.6180339887498949) % 1.0)))) for i in range(case["B"])]
    n[0] = case["L"]
    if case["kind"] == "attention":
        n[5::8] = [0] * len(n[5::8])
    return n


def _sections(case):
    """Pairs of each axis: an equal share, the rest to the first."""
    n, a = case["rot"] // 2, case["axes"]
    return [n - (a - 1) * (n // a)] + [n // a] * (a - 1)


def _pad(n, to):
    return (n + to - 1) // to * to


def _int8_rows(shape, pitch, g):
    """Codes [..., pitch] and scales of rows of normal values."""
    w = torch.randn(shape, device="cuda", generator=g)
    a = w.abs().amax(-1)
    q = torch.zeros(*shape[:-1], pitch, dtype=torch.int8, device="cuda")
    q[..., : shape[-1]] = w.mul_((127.0 / a)[..., None]).round_().to(torch.int8)
    return q, a / 127.0


def _weight(n, k, g):
    q, s = _int8_rows((n, k), _pad(k, 128), g)
    return q, s * k ** -0.5


def _cache(pages, case, g):
    shape = (pages, case["KV"], case["page"], case["D"])
    (k, ks), (v, vs) = (_int8_rows(shape, _pad(case["D"], 64), g) for _ in range(2))
    return (k, ks, v, vs)


def _rows(shape, dtype, g):
    """Rows of unequal size with a few channels that stand out."""
    x = torch.randn(shape, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(shape[0], *[1] * (len(shape) - 1), device="cuda", generator=g))
    x *= 1 + 9 * (torch.rand(shape[-1], device="cuda", generator=g) < 0.01)
    return x.to(dtype)


def _frequencies(rot):
    return BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, dtype, D, KV = case["kind"], TYPES[case["type"]], case["D"], case["KV"]
    s = dict(kind=kind, dtype=dtype, D=D, KV=KV)
    if kind in ("qk", "qk_train", "append", "block"):
        H = s["H"] = case["H"]
        s["eps"] = QK_EPS if case.get("norm", True) else None
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dtype)
                                        if s["eps"] else None for _ in range(2))
        s["inter"] = case.get("inter", False)
        s["freq"] = _frequencies(case.get("rot", D))
        s["sections"] = _sections(case) if case.get("axes", 1) > 1 else None
    if kind in ("qk", "qk_train", "append"):
        T = case["T"]
        # a product's rows hold queries, keys and values side by side
        s["qkv"] = _rows((T, H + 2 * KV, D), dtype, g)
        if case["axes"] > 1:
            s["pos"] = torch.randint(0, 1024, (case["axes"], T), device="cuda", generator=g)
        elif T > 64:
            s["pos"] = torch.arange(T, device="cuda") + 100 * seed % 100000
        else:
            s["pos"] = torch.randint(0, 131072, (T,), device="cuda", generator=g)
        s["q"], s["k"], s["v"] = s["qkv"].split([H, KV, KV], dim=1)
    if kind == "qk_train":
        s["q"], s["k"] = s["q"].detach().requires_grad_(True), s["k"].detach().requires_grad_(True)
        s["leaves"] = [s["q"], s["k"]]
        if s["eps"]:
            s["leaves"] += [s["q_weight"].requires_grad_(True), s["k_weight"].requires_grad_(True)]
        s["dq"] = torch.randn(T, H, D, device="cuda", generator=g).to(dtype)
        s["dk"] = torch.randn(T, KV, D, device="cuda", generator=g).to(dtype)
    if kind == "write":
        s["k"], s["v"] = (_rows((case["T"], KV, D), dtype, g) for _ in range(2))
    if kind in ("append", "write", "read"):
        T, page = case["T"], case["page"]
        n = T + 8 if T <= 64 else T // page + 1
        s["cache"] = _cache(n, case, g)
        order = torch.randperm(n, device="cuda", generator=g)
        at = torch.arange(T, device="cuda")
        # new tokens of as many sequences, or one sequence's tokens through its pages
        s["slots"] = order[:T] * page + torch.randint(0, page, (T,), device="cuda", generator=g) if T <= 64 \
            else order[at // page] * page + at % page
    if kind in ("attention", "block"):
        n, page, window = _lengths(case), case["page"], case["window"]
        need = torch.tensor([_pad(x, page) // page for x in n], device="cuda")
        total, wide = int(need.sum()), max(1, int(need.max()))
        s["cache"] = _cache(total + 1, case, g)
        # the tables' entries behind a sequence's last page are -1
        first = torch.cumsum(need, 0) - need
        col = torch.arange(wide, device="cuda")
        order = torch.randperm(total + 1, device="cuda", generator=g)
        at = (first[:, None] + col).clamp(max=total)
        s["pages"] = torch.where(col < need[:, None], order[at], -1).to(torch.int32)
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["window"], s["scale"] = window, D ** -0.5
    if kind == "attention":
        s["q"] = (2 * torch.randn(case["B"], case["H"], D, device="cuda", generator=g)).to(dtype)
    if kind == "block":
        s["x"], s["res"] = (_rows((case["B"], case["K"]), dtype, g) for _ in range(2))
        s["norm_w"] = (1 + 0.2 * torch.randn(case["K"], device="cuda", generator=g)).to(dtype)
        s["wqkv"] = _weight((H + 2 * KV) * D, case["K"], g)
        s["wout"] = _weight(case["K"], H * D, g)
        s["pos"] = s["lengths"].long() - 1
        s["slots"] = s["pages"].long().gather(1, (s["pos"] // page)[:, None])[:, 0] * page + s["pos"] % page
    return s


# ------------------------------------------------------------ plain forms
def _angles(s):
    """cos and sin [T][1][pairs] in 32 bits, of angles taken in 64."""
    pos = s["pos"]
    if s["sections"]:
        pos = pos.repeat_interleave(torch.tensor(s["sections"], device=pos.device), dim=0, output_size=s["freq"].numel()).t()
    else:
        pos = pos[:, None]
    a = pos.double() * s["freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _pairs(x, rot, inter):
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2: rot]


def _join(a, b, rest, inter):
    both = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _rotate(x, cos, sin, inter):
    rot = 2 * cos.shape[-1]
    a, b = _pairs(x, rot, inter)
    return _join(a * cos - b * sin, b * cos + a * sin, x[..., rot:], inter)


def _unit(x, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r, r


def _turned(s, x, w, cos, sin):
    """Norm and rotation of the heads x, in 32 bits."""
    y = x.float()
    if s["eps"]:
        y = _unit(y, s["eps"])[0] * w.float()
    return _rotate(y, cos, sin, s["inter"])


def _turned_back(s, x, w, dy, cos, sin):
    """Gradients of the heads x and of their weight."""
    d = _rotate(dy.float(), cos, -sin, s["inter"])
    if not s["eps"]:
        return d.to(x.dtype), None
    u, r = _unit(x.float(), s["eps"])
    g = d * w.float()
    dx = r * (g - u * (g * u).mean(-1, keepdim=True))
    return dx.to(x.dtype), (d * u).sum((0, 1)).to(w.dtype)


def _codes(y, pitch):
    """Int8 codes (as 32-bit numbers, zeros up to the pitch) and scales of the rows of y."""
    a = y.abs().amax(-1, keepdim=True)
    q = torch.round(y * torch.where(a > 0, 127.0 / a, 0.0))
    return torch.nn.functional.pad(q, (0, pitch - y.shape[-1])), (a / 127.0)[..., 0]


def _put(cache, slots, k, v):
    page = cache[0].shape[2]
    at = (slots // page, slice(None), slots % page)
    for y, codes, scales in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        q, sc = _codes(y, codes.shape[3])
        codes[at], scales[at] = q.to(torch.int8), sc


def _get(cache, slots, D, dtype):
    page = cache[0].shape[2]
    at = (slots // page, slice(None), slots % page)
    return {"k": (cache[0][at][..., :D].float() * cache[1][at][..., None]).to(dtype),
            "v": (cache[2][at][..., :D].float() * cache[3][at][..., None]).to(dtype)}


def _attend(s, q):
    """[B][H][D] in 32 bits."""
    (k, ks, v, vs), table, n, D = s["cache"], s["pages"].long().clamp(min=0), s["lengths"].long(), s["D"]
    page, KV, B = k.shape[2], k.shape[1], q.shape[0]
    t = torch.arange(table.shape[1] * page, device=q.device)
    seen = t < n[:, None]
    if s["window"]:
        seen = seen & (t >= n[:, None] - s["window"])
    # [B][pages][KV][page][D] -> [B][KV][tokens][D]
    rows = lambda c, sc: (c[table][..., :D].float() * sc[table][..., None]).transpose(1, 2).reshape(B, KV, -1, D)  # noqa: E731
    qs = q.float().reshape(B, KV, -1, D) * s["scale"]
    score = torch.matmul(qs, rows(k, ks).transpose(2, 3))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(v, vs)) / torch.where(total > 0, total, 1.0)
    return o.reshape(B, -1, D)


def _product(x, w, dtype):
    """Rows quantized, times an int8 weight."""
    q, sq = _codes(x, w[0].shape[1])
    return ((q @ w[0].float().t()) * sq[:, None] * w[1]).to(dtype)


def _plain(s):
    kind, dtype, D, KV = s["kind"], s["dtype"], s["D"], s["KV"]
    with torch.no_grad():
        if kind == "read":
            return _get(s["cache"], s["slots"], D, dtype)
        if kind == "write":
            _put(s["cache"], s["slots"], s["k"].float(), s["v"].float())
            return _get(s["cache"], s["slots"], D, dtype)
        if kind == "attention":
            return {"o": _attend(s, s["q"]).to(dtype)}
        cos, sin = _angles(s)
        if kind in ("qk", "qk_train"):
            r = {"q": _turned(s, s["q"], s["q_weight"], cos, sin).to(dtype),
                 "k": _turned(s, s["k"], s["k_weight"], cos, sin).to(dtype)}
            if kind == "qk_train":
                r["dq"], r["dq_weight"] = _turned_back(s, s["q"], s["q_weight"], s["dq"], cos, sin)
                r["dk"], r["dk_weight"] = _turned_back(s, s["k"], s["k_weight"], s["dk"], cos, sin)
            return r
        if kind == "append":
            q = _turned(s, s["q"], s["q_weight"], cos, sin).to(dtype)
            _put(s["cache"], s["slots"], _turned(s, s["k"], s["k_weight"], cos, sin), s["v"].float())
            return {"q": q, **_get(s["cache"], s["slots"], D, dtype)}
        h = (s["x"].float() + s["res"].float()).to(dtype)
        y = _unit(h.float(), EPS)[0] * s["norm_w"].float()
        qkv = _product(y, s["wqkv"], dtype).view(-1, s["H"] + 2 * KV, D)
        q, k, v = qkv.split([s["H"], KV, KV], dim=1)
        _put(s["cache"], s["slots"], _turned(s, k, s["k_weight"], cos, sin), v.float())
        o = _attend(s, _turned(s, q, s["q_weight"], cos, sin).to(dtype)).to(dtype)
        return {"y": _product(o.float().reshape(o.shape[0], -1), s["wout"], dtype), "h": h,
                **_get(s["cache"], s["slots"], D, dtype)}


# ------------------------------------------------------ this package's calls
def _own(s):
    from mxfp4_quantized_gemm_amd import attention, kv_cache, rotary
    kind, dtype, D = s["kind"], s["dtype"], s["D"]
    if kind == "attention":
        return {"o": attention.paged_attention(s["q"], s["cache"], s["pages"], s["lengths"], scale=s["scale"],
                                               window=s["window"])}
    if kind == "qk":
        q, k = rotary.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["q_weight"], s["k_weight"], s["eps"],
                                   sections=s["sections"], interleaved=s["inter"])
        return {"q": q, "k": k}
    if kind == "qk_train":
        q, k = rotary.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["q_weight"], s["k_weight"], s["eps"],
                                   sections=s["sections"], interleaved=s["inter"])
        d = torch.autograd.grad((q, k), s["leaves"], (s["dq"], s["dk"]))
        return {"q": q, "k": k, "dq": d[0], "dk": d[1], "dq_weight": d[2] if s["eps"] else None,
                "dk_weight": d[3] if s["eps"] else None}
    r = {}
    if kind == "write":
        kv_cache.int8_kv_write(s["k"], s["v"], s["cache"], s["slots"])
    if kind == "append":
        r["q"] = kv_cache.int8_kv_append(s["q"], s["k"], s["v"], s["cache"], s["slots"], s["pos"], s["freq"],
                                         s["q_weight"], s["k_weight"], s["eps"], sections=s["sections"],
                                         interleaved=s["inter"])
    if kind == "block":
        r["y"], r["h"] = attention.int8_attention(
            s["x"], s["norm_w"], EPS, *s["wqkv"], *s["wout"], s["cache"], s["slots"], s["pages"], s["lengths"],
            s["pos"], s["freq"], s["q_weight"], s["k_weight"], s["eps"], head_dim=D, scale=s["scale"],
            window=s["window"], interleaved=s["inter"], residual=s["res"])
    r["k"], r["v"] = kv_cache.int8_kv_read(s["cache"], s["slots"], D, dtype)
    return r


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind, e, D, KV = case["kind"], SIZE[case["type"]], case["D"], case["KV"]
    H = case.get("H", 0)
    if kind in ("qk", "qk_train"):
        n = case["T"] * (H + KV) * D
        # heads in and out, the positions; the gradients in and out too
        return {"bytes": (2 if kind == "qk" else 4) * n * e + 8 * case["T"] * case["axes"],
                "flops": (8 if kind == "qk" else 26) * n}
    if kind in ("append", "write", "read"):
        T, kv = case["T"], 2 * case["T"] * KV
        b = {"append": T * 2 * H * D * e + kv * (D * e + D + 4), "write": kv * (D * e + D + 4), "read": kv * (D + 4)}[kind]
        # queries in and out, keys and values in, codes and scales out, and the values they stand for
        return {"bytes": b + kv * D * e + 8 * T, "flops": T * (8 * H + 16 * KV) * D}
    n = [min(x, case["window"] or x) for x in _lengths(case)]
    tokens, B = sum(n), case["B"]
    b, f = 2 * tokens * KV * (D + 4), 4 * tokens * H * D
    if kind == "attention":
        return {"bytes": b + 2 * B * H * D * e, "flops": f}
    N, K = (H + 2 * KV) * D, case["K"]
    return {"bytes": b + K * (N + H * D) + 4 * (N + K) + 4 * B * K * e + 2 * B * KV * D * e,
            "flops": f + 2 * B * K * (N + H * D)}


# ------------------------------------------------------------- 64 bits
def _exact_turn(s, x, w):
    """The norm and the rotation, as a product of complex numbers, in 64 bits."""
    y = x.detach().double()
    if s["eps"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * w.detach().double()
    n, pos = s["freq"].numel(), s["pos"].double()
    if s["sections"]:
        axis = [a for a, m in enumerate(s["sections"]) for _ in range(m)]
        pos = pos[axis].t()
    else:
        pos = pos[:, None].expand(-1, n)
    turn = torch.polar(torch.ones_like(pos), pos * s["freq"])[:, None, :]
    first = list(range(0, 2 * n, 2)) if s["inter"] else list(range(n))
    second = list(range(1, 2 * n, 2)) if s["inter"] else list(range(n, 2 * n))
    z = torch.complex(y[..., first], y[..., second]) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rows(v):
    """Codes and scales of rows given in 64 bits: the nearest multiple of a 127th of the row's largest magnitude."""
    step = v.abs().max(dim=-1).values.unsqueeze(-1) / 127
    return torch.round(v / torch.where(step > 0, step, torch.ones_like(step))), step


def _exact_attend(s, q, new=None):
    """Sequence by sequence; new: the last token's (k, v) of each, in place of the cache's."""
    k, ks, v, vs = s["cache"]
    page, D, KV = k.shape[2], s["D"], s["KV"]
    out = []
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            out.append(torch.zeros_like(q[b]))
            continue
        t = torch.arange(max(0, n - s["window"]) if s["window"] else 0, n, device=q.device)
        at = (s["pages"][b].long()[t // page], slice(None), t % page)
        kb, vb = k[at][..., :D].double() * ks[at].double()[..., None], v[at][..., :D].double() * vs[at].double()[..., None]
        if new is not None:
            kb[-1], vb[-1] = new[0][b], new[1][b]
        qb = q[b].view(KV, -1, D)
        w = torch.softmax(torch.bmm(qb, kb.permute(1, 2, 0).contiguous()) * s["scale"], dim=-1)
        out.append(torch.bmm(w, vb.permute(1, 0, 2).contiguous()).view(-1, D))
    return torch.stack(out)


def _exact_linear(y, w):
    q, step = _exact_rows(y)
    return torch.mm(q, w[0].double()[:, : q.shape[1]].t()) * step * w[1].double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, dtype, D, KV = case["kind"], s["dtype"], case["D"], case["KV"]
    if kind == "qk_train":
        t = {n: s[n].detach().double().requires_grad_(True) for n in ("q", "k")}
        wt = {n: s[n].detach().double().requires_grad_(True) for n in ("q_weight", "k_weight")} if s["eps"] else {}
        r = {}
        for n in ("q", "k"):
            leaves = [t[n]] + ([wt[n + "_weight"]] if wt else [])
            y = t[n]
            if wt:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + s["eps"]) * wt[n + "_weight"]
            r[n] = _exact_turn(s, t[n], wt.get(n + "_weight"))
            # the rotation's transpose is the rotation by the opposite angle
            back = _exact_turn({**s, "eps": None, "freq": -s["freq"]}, s["d" + n], None)
            d = torch.autograd.grad(y, leaves, back)
            r["d" + n], r["d%s_weight" % n] = d[0], d[1] if wt else None
        return r
    with torch.no_grad():
        if kind == "qk":
            return {n: _exact_turn(s, s[n], s[n + "_weight"]) for n in ("q", "k")}
        if kind == "attention":
            return {"o": _exact_attend(s, s["q"].double())}
        if kind == "read":
            page = case["page"]
            at = (s["slots"] // page, slice(None), s["slots"] % page)
            k, ks, v, vs = s["cache"]
            return {"k": k[at].double()[..., :D] * ks[at].double().unsqueeze(-1),
                    "v": v[at].double()[..., :D] * vs[at].double().unsqueeze(-1)}
        held = lambda y: torch.mul(*_exact_rows(y))  # noqa: E731
        if kind == "write":
            return {"k": held(s["k"].double()), "v": held(s["v"].double())}
        if kind == "append":
            return {"q": _exact_turn(s, s["q"], s["q_weight"]), "k": held(_exact_turn(s, s["k"], s["k_weight"])),
                    "v": held(s["v"].double())}
        # the residual stream, the product's rows, the queries and the heads' outputs are held in the inputs' type
        h = (s["x"].double() + s["res"].double()).to(dtype).double()
        y = h / torch.sqrt(torch.mean(h * h, dim=1, keepdim=True) + EPS) * s["norm_w"].double()
        heads = _exact_linear(y, s["wqkv"]).to(dtype).double().view(case["B"], -1, D)
        q, k, v = heads[:, : case["H"]], heads[:, case["H"]: case["H"] + KV], heads[:, case["H"] + KV:]
        new = held(_exact_turn(s, k, s["k_weight"])), held(v)
        o = _exact_attend(s, _exact_turn(s, q, s["q_weight"]).to(dtype).double(), new).to(dtype).double()
        return {"y": _exact_linear(o.reshape(case["B"], -1), s["wout"]), "h": h, "k": new[0], "v": new[1]}
