"""The 8-bit attention block: every type, layout of pairs and scale against the public calls that it
stands for, in 32 bits against 64, and refused calls that leave the cache as it was."""
import pytest
import torch

from tests.attention_util import TYPES, U, angles, attend64, frequencies, make_cache, make_tables, near, rand, turned, unit

pytestmark = pytest.mark.gpu
EPS, QK_EPS, PAGE = 1e-5, 1e-6, 16


def codes64(v):
    """Codes and step of rows in 64 bits."""
    step = v.abs().amax(-1, keepdim=True) / 127
    return torch.round(v / step), step


def weights(K, H, KV, D, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    codes = lambda n, k: torch.nn.functional.pad(torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8),  # noqa: E731
                                                 (0, -k % 128))
    scales = lambda n, k: (1 + torch.rand(n, generator=g)) / (100 * k ** 0.5)  # noqa: E731
    N = (H + 2 * KV) * D
    return dict(norm=(1 + 0.1 * rand((K,), torch.float32, seed)).to(dtype), qkv=(codes(N, K), scales(N, K)),
                out=(codes(K, H * D), scales(K, H * D)),
                qw=(1 + 0.1 * rand((D,), torch.float32, seed + 1)).to(dtype), kw=(1 + 0.1 * rand((D,), torch.float32, seed + 2)).to(dtype))


def case(H, KV, D, K, lengths, dtype, seed):
    dt, pages = TYPES[dtype], sum(-(-n // PAGE) for n in lengths) + 2
    c = dict(w=weights(K, H, KV, D, seed, dt), cache=make_cache(pages, KV, PAGE, D, seed), lengths=lengths, D=D, KV=KV,
             table=make_tables(lengths, PAGE, pages, seed + 1), pos=torch.tensor(lengths) - 1, freq=frequencies(D // 2),
             x=rand((len(lengths), K), dt, seed + 3), res=rand((len(lengths), K), dt, seed + 4))
    c["slots"] = c["table"].long().gather(1, (c["pos"] // PAGE)[:, None])[:, 0] * PAGE + c["pos"] % PAGE
    return c


def gpu(v):
    return v.cuda() if isinstance(v, torch.Tensor) else type(v)(gpu(t) for t in v) if isinstance(v, (list, tuple)) else \
        {k: gpu(t) for k, t in v.items()} if isinstance(v, dict) else v


def block(c, cache, out=None, table=None, **kw):
    from mxfp4_quantized_gemm_amd.attention import int8_attention
    n = torch.tensor(c["lengths"], dtype=torch.int32).cuda()
    w = c["w"]
    return int8_attention(c["x"], w["norm"], EPS, *w["qkv"], *(w["out"] if out is None else out), cache, c["slots"],
                          c["table"] if table is None else table, n, c["pos"], c["freq"], w["qw"], w["kw"], QK_EPS,
                          head_dim=c["D"], residual=c["res"], **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale,inter,window", [(None, True, 0), (0.3, False, 20), (-0.05, True, 0)])
def test_every_type_scale_and_layout(dtype, scale, inter, window):
    """Bit for bit its parts, each of which is tested against 64 bits."""
    from mxfp4_quantized_gemm_amd.attention import paged_attention
    from mxfp4_quantized_gemm_amd.int8 import int8_gemm, int8_linear
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append
    from mxfp4_quantized_gemm_amd.norm import rms_norm_int8
    c = gpu(case(6, 2, 64, 200, [1, 40, 700], dtype, 3))
    w, one, two = c["w"], [t.clone() for t in c["cache"]], [t.clone() for t in c["cache"]]
    y, h = block(c, one, scale=scale, interleaved=inter, window=window)
    codes, s, h2 = rms_norm_int8(c["x"], w["norm"], EPS, residual=c["res"])
    heads = int8_gemm(codes, s, *w["qkv"], out_dtype=c["x"].dtype).view(3, -1, 64)
    q = int8_kv_append(*heads.split([6, 2, 2], 1), two, c["slots"], c["pos"], c["freq"], w["qw"], w["kw"], QK_EPS,
                       interleaved=inter)
    o = paged_attention(q, two, c["table"], torch.tensor(c["lengths"], dtype=torch.int32).cuda(), scale=scale, window=window)
    assert torch.equal(y, int8_linear(o.reshape(3, -1), *w["out"])) and torch.equal(h, h2) and y.dtype == TYPES[dtype]
    assert all(torch.equal(a, b) for a, b in zip(one, two)) and y.isfinite().all() and y.any()


@pytest.mark.parametrize("H,KV,D,K,scale,inter,seed", [(6, 2, 64, 256, None, False, 2), (4, 4, 80, 200, 0.2, True, 2),
                                                      (3, 1, 128, 384, -0.1, False, 1)])
def test_against_64_bits(H, KV, D, K, scale, inter, seed):
    """In 32 bits, where no rounding in between is larger than a few U. A code within its error of a half
    may be the next one; the inputs have none before the attention (asserted), and behind it those that
    are count as off by one."""
    c = case(H, KV, D, K, [1, 33, 90], "fp32", seed)
    w, B = c["w"], 3
    sc = D ** -0.5 if scale is None else scale
    h = (c["x"] + c["res"])  # one fp32 rounding, as in the call
    # r and two products: 3 U of a value; the largest's too, its division by 127 and the code's product: 8 U
    n = unit(h, EPS)[0] * w["norm"].double()
    qn, step = codes64(n)
    assert ((n / step - qn).abs() < 0.5 - 127 * 8 * U).all()
    # whole sums below 2^24 are exact; the row's scale is within 4 U, three more roundings
    mid = qn @ w["qkv"][0][:, :K].double().t() * step * w["qkv"][1].double()
    e = 8 * U  # of a value of mid
    q, k, v = mid.view(B, -1, D).split([H, KV, KV], 1)
    a = angles(c["pos"], c["freq"], None)
    # a head whose values are off by e of themselves has u within 2 e of itself
    yq, tq = turned(q, w["qw"], QK_EPS, a, inter)
    yk, tk = turned(k, w["kw"], QK_EPS, a, inter)
    tq, tk = tq * (1 + 2 * e / (8 * U)) + U * yq.abs(), tk * (1 + 2 * e / (8 * U))
    new = []
    for t, err in ((yk, tk), (v, e * v.abs())):
        codes, st = codes64(t)
        off = (err + err.amax(-1, keepdim=True)) / st + 127 * 4 * U
        assert ((t / st - codes).abs() < 0.5 - off).all()
        new += [codes, st[..., 0], err.amax(-1) / 127 + 2 * U * st[..., 0]]
    cache = [t.clone() for t in c["cache"]]
    at = (c["slots"] // PAGE, slice(None), c["slots"] % PAGE)
    wide = [cache[0].to(torch.int16), cache[1].double(), cache[2].to(torch.int16), cache[3].double()]
    for i, (codes, st) in ((0, new[:2]), (2, new[3:5])):
        wide[i][at[0], :, at[2], :D] = codes.to(torch.int16)
        wide[i + 1][at[0], :, at[2]] = st
    o, _, to = attend64(yq, wide, c["table"], c["lengths"], sc, 0, torch.float32, 2 * U)
    # the queries' error and the new token's: in every score, and in the new token's value
    for b, m in enumerate(c["lengths"]):
        t = torch.arange(m)
        pg = c["table"][b].long()[t // PAGE]
        kb = (wide[0][pg, :, t % PAGE, :D].double() * wide[1][pg, :, t % PAGE][..., None]).permute(1, 0, 2)
        vb = (wide[2][pg, :, t % PAGE, :D].double() * wide[3][pg, :, t % PAGE][..., None]).permute(1, 0, 2)
        qb, eb = yq[b].view(KV, -1, D), tq[b].view(KV, -1, D)
        p = torch.softmax(torch.matmul(qb, kb.transpose(1, 2).contiguous()) * sc, -1)
        es = torch.matmul(eb, kb.abs().transpose(1, 2).contiguous()) * abs(sc)
        ek = torch.zeros_like(kb)
        ek[:, -1] = new[0][b].abs() * new[2][b][:, None]
        es = es + torch.matmul(qb.abs() + eb, ek.transpose(1, 2).contiguous()) * abs(sc)
        ev = torch.zeros_like(vb)
        ev[:, -1] = new[3][b].abs() * new[5][b][:, None]
        more = torch.matmul(p * es, vb.abs()) + torch.matmul(p, vb.abs()) * (p * es).sum(-1, keepdim=True) + torch.matmul(p, ev)
        to[b] += 1.01 * more.reshape(-1, D)  # (second-order terms: es is below 0.01)
        assert float(es.max()) < 0.01
    o, to = o.reshape(B, -1), to.reshape(B, -1) + U * o.reshape(B, -1).abs()
    qo, st = codes64(o)
    off = (to + to.amax(-1, keepdim=True)) / st + 127 * 4 * U
    assert float(off.max()) < 0.5
    other = ((o / st - qo).abs() >= 0.5 - off).double()
    wo = w["out"][0][:, : H * D].double().t()
    y = qo @ wo * st * w["out"][1].double()
    ey = other @ wo.abs() * st * w["out"][1].double()
    ty = ey + (to.amax(-1, keepdim=True) / (127 * st) + 8 * U) * (y.abs() + ey)
    got = [t.cuda() for t in c["cache"]]
    y32, h32 = block(gpu(c), got, scale=scale, interleaved=inter)
    assert torch.equal(h32.cpu(), h)
    near(y32, y, ty, "y")
    assert float(ty.mean()) < 0.2 * float(y.abs().mean())  # the bound says something
    for i, (codes, st, err) in ((0, new[:3]), (2, new[3:])):
        rows, scales = got[i].cpu()[at[0], :, at[2]], got[i + 1].cpu()[at[0], :, at[2]]
        assert torch.equal(rows[..., :D].double(), codes) and not rows[..., D:].any()
        near(scales, st, err, "scales")


def test_a_refused_block_leaves_the_cache():
    """What is wrong with the output product's weight or the page tables is said before anything is written."""
    from mxfp4_quantized_gemm_amd import MXFP4Error
    c = gpu(case(4, 2, 64, 256, [20, 3], "bf16", 11))
    codes, scales = c["w"]["out"]
    cache = [t.clone() for t in c["cache"]]
    far = torch.zeros(1, 1, dtype=torch.int32, device="cuda").expand(2, ((1 << 31) - 16384) // PAGE + 1)
    bad = [(dict(out=(codes, scales[:-1])), ValueError), (dict(out=(codes, scales.double())), TypeError),
           (dict(out=(codes, scales.cpu())), ValueError), (dict(out=(codes.short(), scales)), TypeError),
           (dict(out=(codes.cpu(), scales)), ValueError), (dict(out=(codes[:1].expand(256, -1), scales)), ValueError),
           (dict(out=(torch.stack([codes, codes], -1)[..., 0], scales)), ValueError),
           (dict(table=far), MXFP4Error), (dict(window=-1), ValueError)]
    for i, (kw, error) in enumerate(bad):
        with pytest.raises(error):
            block(c, cache, **kw)
        assert all(torch.equal(a, b) for a, b in zip(cache, c["cache"])), i
    block(c, cache)
    assert not torch.equal(cache[0], c["cache"][0])
