"""Inputs and plain implementations in 64 bits that the tests of attention's
operators share."""
import torch

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def near(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() / tol).nan_to_num(1e9).max())}"


def frequencies(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))


def halves(pairs, interleaved):
    """Columns of the pairs' first and second values."""
    i = torch.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)


def angles(pos, freq, sections):
    """[tokens][pairs] in 64 bits; pos [tokens], or [axes][tokens] with sections."""
    if sections is not None:
        pos = pos[torch.arange(len(sections)).repeat_interleave(torch.tensor(sections))].t()
    else:
        pos = pos[:, None]
    return pos.double() * freq


def turn(z, a, interleaved):
    """z [tokens][heads][dim] turned by the angles a; and the size that its roundings go by."""
    i, j = halves(a.shape[1], interleaved)
    y, size = z.clone(), z.abs()
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    y[..., i], y[..., j] = z[..., i] * c - z[..., j] * s, z[..., j] * c + z[..., i] * s
    size[..., i] = size[..., j] = z[..., i].abs() + z[..., j].abs()
    return y, size


def unit(x, eps):
    """u = x r and r in 64 bits; eps is the fp32 number that the call takes."""
    x = x.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + torch.tensor(eps, dtype=torch.float32).double())
    return x * r, r


def turned(x, w, eps, a, interleaved):
    """Norm and rotation of heads x in 64 bits, and a bound of the fp32 result's error.

    r, x r and its product with w round once each (3 U). An angle's rest of at most
    pi / 4 has 2^-24 of itself, its sine and cosine 1.5 roundings more: 3 U of the
    other value's size at most. Two products, one of them exact in the
    multiply-add, and the sum: 2 U. Together 8 U of the pair's size."""
    z = x.double() if eps is None else unit(x, eps)[0] * (1.0 if w is None else w.double())
    y, size = turn(z, a, interleaved)
    return y, 8 * U * size


def codes_of(y):
    """Codes and scales of rows as the quantizer makes them of fp32 rows."""
    a = y.abs().amax(-1, keepdim=True)
    q = torch.round(y * torch.where(a > 0, 127.0 / a, torch.zeros_like(a)))
    return q, (a / 127.0)[..., 0]


def make_cache(pages, heads, page, dim, seed):
    """A cache of random codes, scales around 1 / 40, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    pitch = (dim + 63) // 64 * 64
    code = lambda: torch.randint(-127, 128, (pages, heads, page, pitch), generator=g, dtype=torch.int8)  # noqa: E731
    scale = lambda: torch.exp(0.5 * torch.randn(pages, heads, page, generator=g)) / 40  # noqa: E731
    return [code(), scale(), code(), scale()]


def make_tables(lengths, page, pages, seed, extra=1):
    """Page tables of sequences over a cache of `pages` pages, each page once; -1 behind a sequence's."""
    need = [(n + page - 1) // page for n in lengths]
    assert sum(need) <= pages
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lengths), max(need, default=0) + extra), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return table


def attend64(q, cache, table, lengths, scale, window, dtype, parts_err):
    """(o, lse, bound of o's error before its own rounding) in 64 bits.

    A score's error: the fp32 sum of dim products, ks * scale, its product with the sum and the
    difference to the maximum, (dim + 8) U of sum |q| |k| scale and 4 U of the score's size; with the exponential's two
    roundings that is e, relative to each probability. The sums over tokens add
    (tokens + 64) U, the split of p vs parts_err, of sum p |v|; and a p vs that is small is held to
    2^-25 of an f16 subnormal's step where 2^14 stands for at most twice the largest vs: 2^-38 of
    that for each code."""
    k, ks, v, vs = cache
    page, heads, dim = k.shape[2], k.shape[1], q.shape[2]
    out, lse, tol = [], [], []
    for b, n in enumerate(lengths):
        n = max(0, min(n, table.shape[1] * page))
        t = torch.arange(max(0, n - window) if window else 0, n)
        pg = table[b].long()[t // page]
        ok = (pg >= 0) & (pg < k.shape[0])
        t, pg = t[ok], pg[ok]
        kb = k[pg, :, t % page, :dim].double() * ks[pg, :, t % page].double()[..., None]  # [n][kv][dim]
        vb = v[pg, :, t % page, :dim].double() * vs[pg, :, t % page].double()[..., None]
        qb = q[b].double().reshape(heads, -1, dim)
        s = torch.einsum("hgd,nhd->hgn", qb, kb) * scale
        size = torch.einsum("hgd,nhd->hgn", qb.abs(), kb.abs()) * abs(scale)
        if len(t) == 0:
            out.append(torch.zeros(q.shape[1], dim, dtype=torch.float64))
            lse.append(torch.full((q.shape[1],), -float("inf"), dtype=torch.float64))
            tol.append(torch.zeros(q.shape[1], dim, dtype=torch.float64))
            continue
        p = torch.softmax(s, -1)
        e = (dim + 8) * U * size + 4 * U * (s.abs() + s.amax(-1, keepdim=True).abs()) + 2 * U
        o = torch.einsum("hgn,nhd->hgd", p, vb)
        mass = torch.einsum("hgn,nhd->hgd", p, vb.abs())
        err = torch.einsum("hgn,nhd->hgd", p * e, vb.abs()) + mass * (p * e).sum(-1, keepdim=True)
        err = err + mass * (parts_err + 2 * (len(t) + 64) * U)
        codes = v[pg, :, t % page, :dim].double().abs().sum(0)  # [kv][dim]
        top = vs[pg, :, t % page].double().abs().amax(0)
        err = err + (2.0 ** -38 * top[:, None] * codes)[:, None]
        out.append(o.reshape(-1, dim))
        lse.append(torch.logsumexp(s, -1).reshape(-1))
        tol.append(err.reshape(-1, dim))
    return torch.stack(out), torch.stack(lse), torch.stack(tol)
