"""The int8 key-value cache: codes and scales as int8_quantize makes them of the
rows, keys after norm and rotation within their roundings, slots, and the values
read back bit for bit."""
import pytest
import torch

from tests.attention_util import TYPES, U, angles, codes_of, frequencies, rand, turned

pytestmark = pytest.mark.gpu


def new_cache(pages, heads, dim, page, fill=3):
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_cache
    c = int8_kv_cache(pages, heads, dim, page)
    for t in c:
        t.fill_(fill)
    return c


def at(cache, slots):
    """(k codes, k scales, v codes, v scales) of tokens [T][heads]..., on the CPU."""
    page = cache.k.shape[2]
    s = slots.cpu()
    return [t.cpu()[s // page, :, s % page] for t in cache]


def untouched(cache, slots, fill=3):
    """Everything but the tokens at slots is as it was filled."""
    page = cache.k.shape[2]
    for t in cache:
        t = t.cpu().clone()
        t[slots // page, :, slots % page] = fill
        assert (t == fill).all()


def distinct(T, capacity, seed):
    return torch.randperm(capacity, generator=torch.Generator().manual_seed(seed))[:T]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 1, 16), (1, 8, 128, 64), (5, 2, 33, 16), (7, 3, 64, 48), (33, 2, 80, 32),
                                            (20, 4, 111, 16), (64, 2, 130, 64), (9, 1, 192, 16), (300, 3, 256, 128),
                                            (2051, 5, 96, 16), (2049, 9, 48, 16),
                                            (8203, 2, 64, 64)])
def test_write_and_read(T, heads, D, page, dtype):
    """Work-groups of one token, of two or (up to 16 heads) four from 2048 on; launches of 8192."""
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_read, int8_kv_write
    dt = TYPES[dtype]
    k, v = rand((T, heads, D), dt, T + D).cuda(), rand((T, heads, D), dt, T + D + 1, 20.0).cuda()
    pages = T // page + 3
    cache, slots = new_cache(pages, heads, D, page), distinct(T, pages * page, T)
    int8_kv_write(k, v, cache, slots.cuda())
    got = at(cache, slots)
    for x, codes, scales in ((k, got[0], got[1]), (v, got[2], got[3])):
        q, s = int8_quantize(x.reshape(-1, D))
        assert torch.equal(codes[..., :D].reshape(-1, D), q.cpu()[:, :D]) and not codes[..., D:].any()
        assert torch.equal(scales.reshape(-1), s.cpu())
    untouched(cache, slots)
    for to in TYPES.values():
        rk, rv = int8_kv_read(cache, slots.cuda(), D, to)
        assert rk.shape == (T, heads, D) and rk.dtype == to
        assert torch.equal(rk.cpu(), (got[0][..., :D].float() * got[1][..., None]).to(to))
        assert torch.equal(rv.cpu(), (got[2][..., :D].float() * got[3][..., None]).to(to))


def append(q, k, v, cache, slots, pos, freq, qw, kw, eps, **kw_):
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append
    return int8_kv_append(q.cuda(), k.cuda(), v.cuda(), cache, slots.cuda(), pos.cuda(), freq.cuda(),
                          None if qw is None else qw.cuda(), None if kw is None else kw.cuda(), eps, **kw_)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,K,D,pairs,norm,inter", [
    (1, 32, 8, 128, 64, True, False), (3, 5, 5, 64, 32, True, True), (40, 7, 1, 80, 20, True, False),
    (17, 4, 2, 96, 48, False, False), (6, 2, 1, 33, 16, True, False), (5, 6, 2, 256, 128, False, True),
    (4200, 3, 1, 64, 32, True, False)])
def test_append(T, H, K, D, pairs, norm, inter, dtype):
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    dt, page = TYPES[dtype], 16
    qkv = rand((T, H + 2 * K, D), dt, T + H + D)
    q, k, v = qkv.split([H, K, K], 1)
    qw, kw = ((1 + 0.3 * rand((D,), dt, i).float()).to(dt) if norm else None for i in (1, 2))
    eps = 1e-6 if norm else None
    pos, freq = torch.arange(T) * 3 + 11, frequencies(pairs)
    cache, slots = new_cache(T // page + 2, K, D, page), distinct(T, (T // page + 2) * page, D)
    g = qkv.cuda()
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append
    gq, gk, gv = g.split([H, K, K], 1)
    gw = [None if w is None else w.cuda() for w in (qw, kw)]
    got_q = int8_kv_append(gq, gk, gv, cache, slots.cuda(), pos.cuda(), freq.cuda(), *gw, eps, interleaved=inter)
    want_q, _ = qk_norm_rope(gq, gk, pos.cuda(), freq.cuda(), *gw, eps, interleaved=inter)
    assert torch.equal(got_q, want_q)
    kc, ks, vc, vs = at(cache, slots)
    qv, sv = int8_quantize(gv.reshape(-1, D))
    assert torch.equal(vc[..., :D].reshape(-1, D), qv.cpu()[:, :D]) and torch.equal(vs.reshape(-1), sv.cpu())
    # keys: the fp32 values are within tol of y, so a row's largest is too; the code's
    # product rounds twice, the scale's division once
    y, tol = turned(k, kw, eps, angles(pos, freq, None), inter)
    a = y.abs().amax(-1)
    ea = tol.amax(-1)
    assert ((ks.double() * 127 - a).abs() <= ea + 2 * U * a).all()
    far = (kc[..., :D].double() - y * (127 / a)[..., None]).abs()
    assert (far <= 0.5 + 127 / a[..., None] * (tol + ea[..., None]) + 127 * 4 * U).all()
    assert not kc[..., D:].any()
    untouched(cache, slots)


def test_without_norm_and_rotation_append_is_write():
    q, k, v = (rand((9, h, 64), torch.bfloat16, h) for h in (4, 2, 2))
    slots = distinct(9, 48, 1)
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_write
    a, b = new_cache(3, 2, 64, 16), new_cache(3, 2, 64, 16)
    got = append(q, k, v, a, slots, torch.arange(9), torch.zeros(0, dtype=torch.float64), None, None, None)
    int8_kv_write(k.cuda(), v.cuda(), b, slots.cuda())
    assert torch.equal(got.cpu(), q)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_slots_outside_the_cache():
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_read, int8_kv_write
    k, v = (rand((6, 2, 64), torch.bfloat16, i).cuda() for i in (1, 2))
    slots = torch.tensor([-1, 5, 48, 1 << 40, -(1 << 40), 47])
    cache = new_cache(3, 2, 64, 16)
    int8_kv_write(k, v, cache, slots.cuda())
    untouched(cache, torch.tensor([5, 47]))
    rk, rv = int8_kv_read(cache, slots.cuda(), 64)
    for i in (0, 2, 3, 4):
        assert not rk[i].any() and not rv[i].any()
    for i in (1, 5):
        step = k[i].float().abs().amax(-1, keepdim=True) / 127
        assert ((rk[i].float() - k[i].float()).abs() <= 0.51 * step + rk[i].float().abs() * 2.0 ** -8).all()


@pytest.mark.parametrize("T", [2, 3, 5, 300, 2047, 5001, 8193, 17001])
def test_the_last_of_equal_slots_stays(T):
    """Codes and scales of one token, whatever the launches."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_write
    k, v = (rand((T, 3, 64), torch.float32, T + i, 5.0).cuda() for i in (1, 2))
    slots = torch.randint(0, max(1, min(32, T // 2)), (T,), generator=torch.Generator().manual_seed(T))
    cache, once = new_cache(2, 3, 64, 16), new_cache(2, 3, 64, 16)
    int8_kv_write(k, v, cache, slots.cuda())
    last = {int(s): i for i, s in enumerate(slots)}
    keep = torch.tensor(sorted(last.values()))
    int8_kv_write(k[keep.cuda()], v[keep.cuda()], once, slots[keep].cuda())
    assert all(torch.equal(a, b) for a, b in zip(cache, once))


@pytest.mark.parametrize("D", [2, 40, 80, 200])
def test_narrow_heads_after_others_memory(D):
    """What is left in the LDS by a call whose weights are all NaN changes no code or scale."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append
    T, slots, pos = 600, torch.arange(600).cuda(), torch.arange(600).cuda()

    def one(D, w):
        x = rand((T, 8, D), torch.float32, D).cuda()
        cache = new_cache(10, 8, D, 64)
        w = torch.full((D,), w).cuda()
        return int8_kv_append(x, x, x, cache, slots, pos, frequencies(D // 4).cuda(), w, w, 1e-6), *cache
    want = one(D, 1.0)
    for _ in range(4):
        assert one(256, float("nan"))[0].isnan().all()
        got = one(D, 1.0)
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and got[2].isfinite().all() and got[2].any()


def test_autograd_sees_the_write():
    """A gradient whose saved scales a write has replaced is refused, as after torch's own changes."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append, int8_kv_write
    x, slots = rand((2, 3, 64), torch.float32, 1).cuda(), torch.tensor([3, 40]).cuda()
    for write in (lambda c: int8_kv_write(x, x, c, slots),
                  lambda c: int8_kv_append(x, x, x, c, slots, slots, frequencies(32).cuda())):
        cache = new_cache(4, 3, 64, 16)
        w = torch.ones_like(cache.k_scales).requires_grad_(True)
        y = (w * cache.k_scales).sum()
        write(cache)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        with torch.inference_mode():
            write(new_cache(4, 3, 64, 16))


def test_rows_of_zeros_and_not_finite():
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_write
    k = rand((4, 1, 64), torch.float32, 1)
    k[0] = 0
    k[1, 0, 3], k[2, 0, 4] = float("nan"), -float("inf")
    k[3] *= 1e-44
    cache = new_cache(1, 1, 64, 16)
    int8_kv_write(k.cuda(), k.cuda(), cache, torch.arange(4).cuda())
    kc, ks, _, _ = at(cache, torch.arange(4))
    assert not kc[:3].any() and ks[0] == 0 and ks[1:3].isnan().all()
    q, s = codes_of(k[3].double())
    assert int(kc[3].abs().max()) == 127 and abs(float(ks[3]) - float(s)) <= 1.5e-45


def test_empty_and_leading_dimensions():
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_read, int8_kv_write
    cache = new_cache(2, 2, 64, 16)
    none = torch.empty(0, 2, 64, device="cuda")
    int8_kv_write(none, none, cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert int8_kv_read(cache, torch.empty(0, dtype=torch.int64, device="cuda"), 64)[0].shape == (0, 2, 64)
    untouched(cache, torch.empty(0, dtype=torch.int64))
    k = rand((2, 3, 2, 64), torch.bfloat16, 1).cuda()
    slots = torch.arange(6).cuda()
    int8_kv_write(k, k, cache, slots.view(2, 3))
    a = int8_kv_read(cache, slots.view(2, 3), 64)[0]
    assert a.shape == (2, 3, 2, 64) and torch.equal(a.view(6, 2, 64), int8_kv_read(cache, slots, 64)[0])


def test_offsets_past_32_bits():
    """Pages on both sides of byte 2^32 of the codes."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_read, int8_kv_write
    pages = (1 << 32) // (8 * 64 * 128) + 2
    cache = new_cache(pages, 8, 128, 64, fill=0)
    slots = torch.tensor([0, pages * 64 - 1, (pages - 1) * 64, (pages - 2) * 64 - 1, 77]).cuda()
    k, v = (rand((5, 8, 128), torch.bfloat16, i).cuda() for i in (1, 2))
    int8_kv_write(k, v, cache, slots)
    small = new_cache(1, 8, 128, 64)
    int8_kv_write(k, v, small, torch.arange(5).cuda())
    for a, b in zip(int8_kv_read(cache, slots, 128), int8_kv_read(small, torch.arange(5).cuda(), 128)):
        assert torch.equal(a, b)
    assert int((cache.k_scales != 0).sum()) == 40


def test_c_entry_points():
    import mxfp4_quantized_gemm_amd as mx
    q, k, v = (rand((9, h, 80), torch.float16, h).cuda() for h in (4, 2, 2))
    w = (1 + 0.1 * rand((80,), torch.float32, 5)).cuda()
    pos, freq, slots = torch.arange(9).cuda(), frequencies(40).cuda(), distinct(9, 48, 2).cuda()
    a, b = new_cache(3, 2, 80, 16), new_cache(3, 2, 80, 16)
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append, int8_kv_read
    want = int8_kv_append(q, k, v, a, slots, pos, freq, w, None, 1e-6)
    out, rk, rv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mx.mxfp4_int8_kv_write(q, k, v, pos, freq, w, None, 1e-6, b, slots, out, stream=s)
    mx.mxfp4_int8_kv_read(b, slots, rk, rv, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip((rk, rv), int8_kv_read(a, slots, 80, torch.float16)))
