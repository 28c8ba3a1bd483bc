"""Refusals of attention's entry points (no GPU: every check returns before any
HIP call) and of their bindings."""
import ctypes

import pytest
import torch

import mxfp4_quantized_gemm_amd as mx

P = 0x10000  # aligned, never read
ODD, TWO, EIGHT = P + 1, P + 2, P + 8
OK, ENULL, ESHAPE, EMODE, EWS, EALIGN = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def heads(n=4, p=P, ts=512, hs=64):
    return mx.Heads(p, n, ts, hs)


def rotation(**kw):
    a = dict(positions=P, frequencies=P, pairs=32, axes=1, interleaved=0, axis_pairs=(32, 0, 0, 0))
    a.update(kw)
    a["axis_pairs"] = (ctypes.c_int64 * 4)(*a["axis_pairs"])
    return mx.Rotation(*a.values())


def cache(**kw):
    a = dict(k=P, ks=P, v=P, vs=P, pages=8, heads=2, page=16, pitch=64)
    assert not set(kw) - set(a)
    a.update(kw)
    return mx.Int8KV(*a.values())


def args(defaults, kw):
    assert not set(kw) - set(defaults)
    return {**defaults, **kw}.values()


def turn(lib, **kw):
    return lib.mxfp4_qk_norm_rope(*args(dict(q=heads(), k=heads(2), tokens=0 + 3, dim=64, dt=1, rot=rotation(), qw=P, kw=P,
                                             wt=1, eps=1e-6, qo=P, ko=P, rstd=P), kw), None)


def turn_bwd(lib, **kw):
    a = dict(dq=heads(), dk=heads(2), q=heads(), k=heads(2), tokens=3, dim=64, dt=1, rot=rotation(), qw=P, kw=P, wt=1,
             rstd=P, qo=P, ko=P, dqw=P, dkw=P, ws=P, wsb=lib.mxfp4_qk_norm_rope_bwd_workspace_bytes(3, 4, 2, 64))
    return lib.mxfp4_qk_norm_rope_bwd(*args(a, kw), None)


def write(lib, **kw):
    a = dict(q=heads(), k=heads(2), v=heads(2), tokens=3, dim=64, dt=1, rot=rotation(), qw=P, kw=P, wt=1, eps=1e-6,
             cache=cache(), slots=P, qo=P)
    return lib.mxfp4_int8_kv_write(*args(a, kw), None)


def attend(lib, **kw):
    a = dict(q=heads(), batch=3, dim=64, dt=1, cache=cache(), pages=P, ld=40, table=40, lengths=P, scale=1.0, window=0,
             out=P, lse=P, ws=P, wsb=lib.mxfp4_paged_attention_workspace_bytes(3, 4, 2, 64, 40, 16))
    return lib.mxfp4_paged_attention(*args(a, kw), None)


def check_shared(call, lib):
    assert call(lib, dt=3) == EMODE and call(lib, dt=-1) == EMODE
    assert call(lib, wt=2) == EMODE and call(lib, dt=0, wt=1) == EMODE
    if call is turn_bwd:
        assert call(lib, rstd=None) == EMODE                   # weights without a norm
        assert call(lib, rstd=None, qw=None, dqw=None, dkw=None) == EMODE
    else:
        assert call(lib, eps=float("nan")) == EMODE
        assert call(lib, eps=-1.0) == EMODE
        assert call(lib, eps=-1.0, qw=None) == EMODE
    for dim in (0, -1, 257, 63):
        # 63: the rotation is wider than the head
        assert call(lib, dim=dim) == ESHAPE, dim
    for tokens in (-1, 1 << 31):
        assert call(lib, tokens=tokens) == ESHAPE
    for bad in (heads(-1), heads(1025), heads(ts=-1), heads(hs=-1), heads(ts=1 << 50), heads(hs=1 << 50)):
        assert call(lib, q=bad) == ESHAPE
        assert call(lib, k=bad) == ESHAPE
    for r in (rotation(pairs=33), rotation(pairs=-1), rotation(axes=0), rotation(axes=5),
              rotation(axes=2, axis_pairs=(16, 15, 0, 0)), rotation(axes=2, axis_pairs=(33, -1, 0, 0))):
        assert call(lib, rot=r) == ESHAPE
    assert call(lib, rot=rotation(positions=None)) == ENULL
    assert call(lib, rot=rotation(frequencies=None)) == ENULL
    assert call(lib, rot=rotation(positions=P + 4)) == EALIGN
    assert call(lib, q=heads(p=None)) == ENULL
    assert call(lib, k=heads(2, p=None)) == ENULL
    assert call(lib, qo=None) == ENULL
    for k in ("qw", "kw", "qo"):
        assert call(lib, **{k: ODD}) == EALIGN, k
    assert call(lib, q=heads(p=ODD)) == EALIGN
    assert call(lib, k=heads(2, p=ODD)) == EALIGN
    assert call(lib, wt=0, qw=TWO) == EALIGN


def test_norm_rope_refusals(lib):
    check_shared(turn, lib)
    assert turn(lib, rstd=TWO) == EALIGN
    assert turn(lib, q=None) == ENULL and turn(lib, k=None) == ENULL and turn(lib, ko=None) == ENULL
    assert turn(lib, tokens=0, q=heads(p=None), k=heads(p=None), qo=None, ko=None, rot=rotation(positions=None)) == OK
    assert turn(lib, q=heads(0, None), k=heads(0, None), qo=None, ko=None) == OK


def test_norm_rope_bwd_refusals(lib):
    check_shared(turn_bwd, lib)
    need = lib.mxfp4_qk_norm_rope_bwd_workspace_bytes(3, 4, 2, 64)
    assert need >= 2 * 64 * 4
    for sizes in ((-1, 4, 2, 64), (3, 4, 2, 0), (3, 4, 2, 257), (1 << 31, 4, 2, 64)):
        assert lib.mxfp4_qk_norm_rope_bwd_workspace_bytes(*sizes) == 0
    assert turn_bwd(lib, wsb=need - 1) == EWS
    assert turn_bwd(lib, ws=None) == ENULL
    assert turn_bwd(lib, dq=heads(3)) == ESHAPE and turn_bwd(lib, dk=heads(3)) == ESHAPE
    assert turn_bwd(lib, dq=heads(p=None)) == ENULL and turn_bwd(lib, dk=heads(2, p=None)) == ENULL
    assert turn_bwd(lib, ko=None) == ENULL
    assert turn_bwd(lib, dqw=ODD) == EALIGN and turn_bwd(lib, ws=TWO) == EALIGN and turn_bwd(lib, rstd=TWO) == EALIGN
    assert turn_bwd(lib, rstd=None, qw=None, kw=None) == EMODE       # a weight's gradient without a norm
    assert turn_bwd(lib, tokens=0, dqw=None, dkw=None, ws=None, wsb=0) == OK
    for k in ("dq", "dk", "q", "k"):
        assert turn_bwd(lib, **{k: None}) == ENULL


def check_cache(call, lib):
    for bad in (dict(pages=0), dict(heads=0), dict(page=0), dict(page=8), dict(page=24), dict(pitch=128), dict(pitch=48),
                dict(pages=1 << 27), dict(heads=1025)):
        assert call(lib, cache=cache(**bad)) == ESHAPE, bad
    for k in ("k", "ks", "v", "vs"):
        assert call(lib, cache=cache(**{k: None})) == ENULL
        assert call(lib, cache=cache(**{k: EIGHT})) == EALIGN
    assert call(lib, cache=None) == ENULL


def test_kv_write_refusals(lib):
    check_shared(write, lib)
    check_cache(write, lib)
    assert write(lib, k=heads(3)) == ESHAPE and write(lib, v=heads(1)) == ESHAPE  # the cache has two
    assert write(lib, v=heads(2, p=None)) == ENULL and write(lib, slots=None) == ENULL
    assert write(lib, slots=P + 4) == EALIGN and write(lib, v=heads(2, p=ODD)) == EALIGN
    assert write(lib, k=None) == ENULL and write(lib, v=None) == ENULL
    assert write(lib, tokens=0, q=None, slots=None, qo=None) == OK


def test_kv_read_refusals(lib):
    def read(lib, **kw):
        return lib.mxfp4_int8_kv_read(*args(dict(cache=cache(), slots=P, tokens=3, dim=64, dt=1, k=P, v=P), kw), None)
    check_cache(read, lib)
    assert read(lib, dt=3) == EMODE
    for kw in (dict(dim=0), dict(dim=65), dict(dim=257), dict(tokens=-1), dict(tokens=1 << 31)):
        assert read(lib, **kw) == ESHAPE
    for k in ("slots", "k", "v"):
        assert read(lib, **{k: None}) == ENULL
        assert read(lib, **{k: ODD}) == EALIGN
    assert read(lib, tokens=0, slots=None, k=None, v=None) == OK


def test_paged_attention_refusals(lib):
    check_cache(attend, lib)
    assert attend(lib, dt=3) == EMODE
    for kw in (dict(dim=0), dict(dim=65), dict(batch=-1), dict(batch=1 << 31), dict(q=heads(3)), dict(q=heads(0)),
               dict(q=heads(1026)), dict(ld=39), dict(ld=1 << 50), dict(table=-1), dict(window=-1),
               dict(table=1 << 27, ld=1 << 27), dict(q=heads(ts=-1)),
               dict(table=(1 << 27) - 1023, ld=1 << 27)):
        assert attend(lib, **kw) == ESHAPE, kw
    for k in ("q", "lengths", "out", "pages", "ws"):
        assert attend(lib, **{k: None}) == ENULL, k
    assert attend(lib, q=heads(p=None)) == ENULL
    need = lib.mxfp4_paged_attention_workspace_bytes(3, 4, 2, 64, 40, 16)
    assert need > 0 and attend(lib, wsb=need - 1) == EWS
    for k in ("out", "pages", "lengths", "lse", "ws"):
        assert attend(lib, **{k: ODD}) == EALIGN, k
    assert attend(lib, batch=0, q=heads(p=None), lengths=None, out=None, pages=None, ws=None, wsb=0) == OK
    for sizes in ((-1, 4, 2, 64, 20, 16), (3, 4, 3, 64, 20, 16), (3, 0, 2, 64, 20, 16), (3, 4, 2, 0, 20, 16),
                  (3, 4, 2, 64, -1, 16), (3, 4, 2, 64, 20, 24)):
        assert lib.mxfp4_paged_attention_workspace_bytes(*sizes) == 0
    assert lib.mxfp4_paged_attention_workspace_bytes(3, 4, 2, 64, 8, 16) == 0  # one unit: nothing to join


def test_bindings_take_no_cpu_tensors():
    from mxfp4_quantized_gemm_amd import attention, kv_cache, rotary
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos, freq, slots = torch.arange(3), torch.ones(32, dtype=torch.float64), torch.arange(3)
    cache = kv_cache.int8_kv_cache(2, 2, 64, 16, device="cpu")
    n, pages = torch.ones(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: rotary.qk_norm_rope(q, k, pos, freq), lambda: kv_cache.int8_kv_write(k, k, cache, slots),
                 lambda: kv_cache.int8_kv_append(q, k, k, cache, slots, pos, freq),
                 lambda: kv_cache.int8_kv_read(cache, slots, 64),
                 lambda: attention.paged_attention(q, cache, pages, n),
                 lambda: attention.int8_attention(torch.zeros(3, 128), None, 1e-5, torch.zeros(512, 128, dtype=torch.int8),
                                                  torch.ones(512), torch.zeros(128, 256, dtype=torch.int8), torch.ones(128),
                                                  cache, slots, pages, n, pos, freq, head_dim=64)):
        with pytest.raises(ValueError, match="GPU memory"):
            call()


def test_cache_sizes():
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_cache
    c = int8_kv_cache(3, 2, 80, 48, device="cpu")
    assert [tuple(t.shape) for t in c] == [(3, 2, 48, 128), (3, 2, 48)] * 2
    assert not any(t.any() for t in c)
    for kw in (dict(page_size=8), dict(page_size=24), dict(head_dim=0), dict(head_dim=257)):
        with pytest.raises(ValueError):
            int8_kv_cache(**{**dict(pages=3, kv_heads=2, head_dim=64, device="cpu"), **kw})


def test_calls_without_a_gradient_are_refused():
    """Whatever the device: a gradient or a tangent would be dropped."""
    from mxfp4_quantized_gemm_amd import attention, kv_cache, rotary
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos, freq, slots = torch.arange(3), torch.ones(32, dtype=torch.float64), torch.arange(3)
    cache = kv_cache.int8_kv_cache(2, 2, 64, 16, device="cpu")
    n, pages = torch.ones(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    r = lambda t: t.clone().requires_grad_(True)  # noqa: E731
    graded = cache._replace(v_scales=r(cache.v_scales))
    for call in (lambda: rotary.qk_norm_rope(q, k, pos, r(freq)),
                 lambda: kv_cache.int8_kv_write(r(k), k, cache, slots), lambda: kv_cache.int8_kv_write(k, r(k), cache, slots),
                 lambda: kv_cache.int8_kv_append(r(q), k, k, cache, slots, pos, freq),
                 lambda: kv_cache.int8_kv_read(graded, slots, 64), lambda: attention.paged_attention(r(q), cache, pages, n),
                 lambda: attention.paged_attention(q, graded, pages, n)):
        with pytest.raises(RuntimeError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU memory"):
            call()
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        d = fwd.make_dual(q, q)
        for call in (lambda: rotary.qk_norm_rope(d, k, pos, freq), lambda: attention.paged_attention(d, cache, pages, n)):
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
                call()
    with pytest.raises(RuntimeError, match="jit.trace"):
        torch.jit.trace(lambda t: rotary.qk_norm_rope(t, k, pos, freq), (q,))
