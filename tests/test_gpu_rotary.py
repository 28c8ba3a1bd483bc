"""Norm and rotation of queries and keys, and their gradient, against plain
implementations in 64 bits. Tolerances count roundings (attention_util.turned)."""
import pytest
import torch

from tests.attention_util import TYPES, U, angles, frequencies, half_step, near, rand, turn, turned, unit

pytestmark = pytest.mark.gpu
EPS = 1e-6


def case(T, H, K, D, pairs, dtype, seed, norm=True, sections=None, interleaved=False, wide=False, far=False):
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    most = 1 << 40 if far else 5000
    pos = torch.randint(-3, most, (T,) if sections is None else (len(sections), T), generator=g)
    c = dict(q=rand((T, H, D), dt, seed), k=rand((T, K, D), dt, seed + 1, 3.0), pos=pos, freq=frequencies(pairs),
             qw=None, kw=None, eps=EPS if norm else None, sections=sections, inter=interleaved)
    if norm:
        c["qw"], c["kw"] = (1 + 0.3 * rand((D,), torch.float32 if wide else dt, seed + i).float() for i in (2, 3))
        c["qw"], c["kw"] = (w.to(torch.float32 if wide else dt) for w in (c["qw"], c["kw"]))
    c["dq"], c["dk"] = rand((T, H, D), dt, seed + 4), rand((T, K, D), dt, seed + 5)
    return c


def call(c, q, k, qw, kw):
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    return qk_norm_rope(q, k, c["pos"].cuda(), c["freq"].cuda(), qw, kw, c["eps"], sections=c["sections"],
                        interleaved=c["inter"])


def gpu(t):
    return None if t is None else t.cuda()


def check(c):
    dt = c["q"].dtype
    a = angles(c["pos"], c["freq"], c["sections"])
    leaves = [gpu(c[n]) for n in ("q", "k", "qw", "kw")]
    for t in leaves:
        if t is not None:
            t.requires_grad_(True)
    out = call(c, *leaves)
    given = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad(out, given, (c["dq"].cuda(), c["dk"].cuda())))
    dx = [next(grads) if t is not None else None for t in leaves]
    for i, n in enumerate(("q", "k")):
        x, w, dy = c[n], c[n + "w"], c["d" + n]
        y, tol = turned(x, w, c["eps"], a, c["inter"])
        assert out[i].dtype == dt and out[i].is_contiguous()
        near(out[i], y, tol + half_step(y, dt), n)
        d, size = turn(dy.double(), -a, c["inter"])
        e = 5 * U * size  # the turn without the norm's three roundings
        if c["eps"] is None:
            near(dx[i], d, e + half_step(d, dt), "d" + n)
            continue
        u, r = unit(x, c["eps"])
        w64 = 1.0 if w is None else w.double().abs() * 0 + w.double()
        g, eg = d * w64, e * abs(w64)
        gu = (g * u).mean(-1, keepdim=True)
        ref = r * (g - u * gu)
        # u has 2 roundings, g one more; the row's sum at most 8 values a thread and 5
        # steps; then the difference and the product with r
        t = r * (eg + 4 * U * g.abs() + 8 * U * (u * gu).abs()
                 + u.abs() * (eg * u.abs() + 24 * U * (g * u).abs()).mean(-1, keepdim=True)) + 2 * U * ref.abs()
        near(dx[i], ref, t + half_step(ref, dt), "d" + n)
        if w is not None:
            rows = x.shape[0] * x.shape[1]
            s = (d * u).sum((0, 1))
            st = U * (rows + 24) * (d * u).abs().sum((0, 1)) + (e * u.abs()).sum((0, 1))
            near(dx[2 + i], s, st + half_step(s, w.dtype), "dw of " + n)


# every width of thread group, odd and ragged widths and rotated parts, the smallest
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,pairs,inter", [
    (1, 0, False), (2, 1, False), (2, 1, True), (7, 3, False), (8, 4, True), (16, 5, False), (33, 16, True),
    (64, 32, False), (64, 32, True), (72, 20, False), (80, 30, True), (80, 40, False), (96, 48, False),
    (111, 55, False), (128, 64, False), (128, 64, True), (128, 24, False), (128, 0, False), (130, 65, False),
    (192, 96, False), (255, 127, False), (256, 128, False), (256, 64, True)])
def test_widths(D, pairs, inter, dtype):
    check(case(5, 3, 2, D, pairs, dtype, 100 * D + pairs, interleaved=inter))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [2, 40, 80, 200])
def test_narrow_heads_after_others_memory(D, dtype):
    """What is left in the LDS by a call whose weights are all NaN counts in no column past a head's width."""
    bad = case(4096, 8, 8, 256, 128, dtype, 1)
    bad["qw"].fill_(float("nan"))
    bad["kw"].fill_(float("nan"))
    args = [gpu(bad[n]) for n in ("q", "k", "qw", "kw")]
    c = case(700, 5, 3, D, D // 4, dtype, D)
    assert call(bad, *args)[0].isnan().all()
    check(c)
    leaves = [t.requires_grad_(True) for t in args]
    torch.autograd.grad(call(bad, *leaves), leaves, (gpu(bad["dq"]), gpu(bad["dk"])))
    check(c)


@pytest.mark.parametrize("T,H,K", [(1, 1, 1), (1, 32, 8), (4, 1, 0), (3, 0, 2), (17, 9, 3), (130, 5, 5), (2049, 2, 1),
                                   (5000, 3, 1), (8195, 1, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_tokens_and_heads(T, H, K, norm):
    """Work-groups of one token, of two from 2048 tokens on and of four from 8192."""
    check(case(T, H, K, 64, 32, "bf16", T + H, norm=norm))


@pytest.mark.parametrize("sections", [(32,), (16, 16), (8, 12, 12), (0, 20, 12), (32, 0, 0, 0), (5, 9, 11, 7)])
@pytest.mark.parametrize("inter", [False, True])
def test_axes(sections, inter):
    check(case(21, 4, 2, 64, 32, "fp32", len(sections), sections=sections, interleaved=inter))


def test_weights_in_32_bits_beside_16():
    check(case(9, 4, 2, 128, 64, "bf16", 5, wide=True))
    check(case(9, 4, 2, 80, 40, "fp16", 6, wide=True))


@pytest.mark.parametrize("which", ["q", "k"])
def test_one_weight(which):
    c = case(9, 4, 2, 64, 32, "fp32", 7)
    c["kw" if which == "q" else "qw"] = None
    check(c)


def test_far_positions():
    """Positions up to 2^40: fp64 holds the angle to 2^-12 of a turn at worst there, and the
    reference takes the same product, so what is tested is the reduction of whole turns."""
    c = case(50, 2, 1, 64, 32, "fp32", 8, far=True)
    c["freq"] = c["freq"] * 2.0 ** -12
    c["pos"] %= 1 << 34
    a = angles(c["pos"], c["freq"], None)
    q, k = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    for got, n in ((q, "q"), (k, "k")):
        y, tol = turned(c[n], c[n + "w"], EPS, a, False)
        # the call multiplies by 2 / pi after the product with the frequency: one more
        # rounding of an angle of up to 2^22
        size = turn(c[n].double() * 0 + 1, a, False)[1] * unit(c[n], EPS)[0].abs().amax() * 3
        near(got, y, tol + half_step(y, torch.float32) + 2.0 ** -30 * size, n)


def test_strides():
    """Views into a product's rows, transposed heads, broadcast ones, a stride in the last dimension."""
    c = case(6, 4, 2, 64, 32, "bf16", 9)
    want = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    qkv = torch.cat([c["q"], c["k"], c["k"]], 1).cuda()
    views = qkv.split([4, 2, 2], dim=1)[:2]
    t = [gpu(c[n]).transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k")]
    last = [torch.stack([gpu(c[n])] * 2, -1)[..., 0] for n in ("q", "k")]
    for q, k in (views, t, last):
        got = call(c, q, k, gpu(c["qw"]), gpu(c["kw"]))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one head shown four times: a stride of zero, and the sum of their gradients
    x = gpu(c["q"])[:, :1].clone().requires_grad_(True)
    k = gpu(c["k"])
    y, _ = call(c, x.expand(6, 4, 64), k, gpu(c["qw"]), gpu(c["kw"]))
    d, = torch.autograd.grad(y, x, gpu(c["dq"]))
    x4 = x.detach().expand(6, 4, 64).contiguous().requires_grad_(True)
    y4, _ = call(c, x4, k, gpu(c["qw"]), gpu(c["kw"]))
    d4, = torch.autograd.grad(y4, x4, gpu(c["dq"]))
    assert torch.equal(y, y4) and torch.equal(d, d4.sum(1, keepdim=True))


def test_unaligned_rows():
    c = case(6, 3, 2, 40, 20, "bf16", 10)
    want = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    flat = torch.empty(6 * 5 * 43 + 1, dtype=torch.bfloat16, device="cuda")
    rows = flat[1:].view(6, 5, 43)
    rows[:, :3, 1:41], rows[:, 3:, 1:41] = gpu(c["q"]), gpu(c["k"])
    got = call(c, rows[:, :3, 1:41], rows[:, 3:, 1:41], gpu(c["qw"]), gpu(c["kw"]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_leading_dimensions():
    c = case(6, 4, 2, 64, 32, "bf16", 11, sections=(12, 20))
    want = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    d = dict(c, pos=c["pos"].view(2, 2, 3))
    got = call(d, gpu(c["q"]).view(2, 3, 4, 64), gpu(c["k"]).view(2, 3, 2, 64), gpu(c["qw"]), gpu(c["kw"]))
    assert got[0].shape == (2, 3, 4, 64) and torch.equal(got[0].view(6, 4, 64), want[0])
    assert torch.equal(got[1].view(6, 2, 64), want[1])
    one = dict(c, pos=c["pos"][:, 0])  # a token without leading dimensions
    got = call(one, gpu(c["q"])[0], gpu(c["k"])[0], gpu(c["qw"]), gpu(c["kw"]))
    assert got[0].shape == (4, 64) and torch.equal(got[0], want[0][0])


def test_empty():
    c = case(0, 4, 2, 64, 32, "bf16", 12)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    q, k = call(c, *leaves)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    d = torch.autograd.grad((q, k), leaves, (gpu(c["dq"]), gpu(c["dk"])))
    assert d[0].shape == q.shape and not d[2].any() and not d[3].any()


@pytest.mark.parametrize("unused", ["q", "k"])
def test_an_output_no_loss_reads(unused):
    c = case(7, 4, 2, 64, 32, "fp32", 13)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    both = torch.autograd.grad(call(c, *leaves), leaves, (gpu(c["dq"]), gpu(c["dk"])))
    i = 1 if unused == "q" else 0  # the one that is read
    got = torch.autograd.grad(call(c, *leaves)[i], leaves, gpu(c["dk" if i else "dq"]), allow_unused=True)
    assert torch.equal(got[i], both[i]) and torch.equal(got[2 + i], both[2 + i])
    assert got[1 - i] is None and not got[3 - i].any()


def test_gradients_by_differences():
    """Central differences of the call itself, of a loss with fixed weights."""
    c = case(3, 2, 1, 8, 3, "fp32", 14)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    loss = lambda *t: sum((o.double() * gpu(c[d]).double()).sum() for o, d in zip(call(c, *t), ("dq", "dk")))  # noqa: E731
    grads = torch.autograd.grad(loss(*leaves), leaves)
    h = 2.0 ** -7
    for i, t in enumerate(leaves):
        flat = t.detach().reshape(-1)
        for j in range(0, flat.numel(), 5):
            v = []
            for s in (1, -1):
                moved = flat.clone()
                moved[j] += s * h
                args = [x.detach() for x in leaves]
                args[i] = moved.view_as(t)
                v.append(float(loss(*args)))
            # third derivatives of order 30 / |x|^3 at most here times h^2 / 6, and the outputs' roundings:
            # 72 of them of 2^-24 of values up to 8, over h
            far = abs((v[0] - v[1]) / (2 * h) - float(grads[i].reshape(-1)[j]))
            assert far <= 0.02 + 0.02 * abs(float(grads[i].reshape(-1)[j])), (i, j, far)


def test_rows_of_zeros_and_not_finite():
    """A row's values stay its own: a zero row gives zeros (eps > 0), an infinity or NaN leaves the others."""
    c = case(4, 4, 2, 64, 24, "bf16", 15)
    want = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    q = c["q"].clone()
    q[0, 1], q[1, 2, 5], q[2, 3, 60] = 0, float("nan"), float("inf")
    got, _ = call(c, q.cuda(), gpu(c["k"]), gpu(c["qw"]), gpu(c["kw"]))
    assert not got[0, 1].any() and got[1, 2].isnan().all()
    same = torch.ones(4, 4, dtype=torch.bool)
    same[0, 1] = same[1, 2] = same[2, 3] = False
    assert torch.equal(got[same], want[0][same])
    # without a norm an infinity behind the rotated part changes nothing else
    d = dict(c, eps=None)
    y, _ = call(d, q.cuda(), gpu(c["k"]), None, None)
    z, _ = call(d, gpu(c["q"]), gpu(c["k"]), None, None)
    assert y[2, 3, 60] == float("inf")
    y[2, 3, 60] = z[2, 3, 60]
    assert torch.equal(y[2, 3], z[2, 3])


def test_the_largest_values():
    """Squares past fp32's range are summed in fp64."""
    c = case(2, 2, 1, 64, 0, "fp32", 16)
    c["q"] = c["q"] * 2.0 ** 100
    y, tol = turned(c["q"], c["qw"], EPS, angles(c["pos"], c["freq"], None), False)
    q, _ = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    near(q, y, tol + half_step(y, torch.float32), "q")


def test_in_place_changes_are_seen():
    c = case(3, 2, 1, 64, 32, "bf16", 17)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    x = leaves[0] * 1
    q, _ = call(c, x, *leaves[1:])
    x.mul_(2)
    with pytest.raises(RuntimeError, match="inplace"):
        q.sum().backward()


def test_second_derivative_is_refused():
    c = case(3, 2, 1, 64, 32, "fp32", 18)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    q, _ = call(c, *leaves)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(q.sum(), leaves[0], create_graph=True)


def test_offsets_past_32_bits():
    """A token's heads on both sides of element 2^31 of a wide row pitch."""
    c = case(2, 2, 1, 64, 32, "bf16", 19)
    flat = torch.empty((1 << 31) + 1024, dtype=torch.bfloat16, device="cuda")
    rows = flat.as_strided((2, 3, 64), ((1 << 31) - 100, 64, 1))
    rows[:, :2], rows[:, 2:] = gpu(c["q"]), gpu(c["k"])
    got = call(c, rows[:, :2], rows[:, 2:], gpu(c["qw"]), gpu(c["kw"]))
    want = call(c, *(gpu(c[n]) for n in ("q", "k", "qw", "kw")))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_c_entry_points():
    """The C-named calls give what the binding gives, on a stream of their own."""
    import mxfp4_quantized_gemm_amd as mx
    c = case(20, 4, 2, 96, 40, "bf16", 20, sections=(16, 24))
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    out = call(c, *leaves)
    want = torch.autograd.grad(out, leaves, (gpu(c["dq"]), gpu(c["dk"])))
    q, k, qw, kw = (t.detach() for t in leaves)
    pos, freq, dq, dk = gpu(c["pos"]), gpu(c["freq"]), gpu(c["dq"]), gpu(c["dk"])
    qo, ko, dqo, dko, dqw, dkw = (torch.full_like(t, 7) for t in (q, k, q, k, qw, kw))
    ws = torch.empty(mx.mxfp4_qk_norm_rope_bwd_workspace_bytes(20, 4, 2, 96), dtype=torch.uint8, device="cuda")
    rstd = torch.empty(20, 6, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mx.mxfp4_qk_norm_rope(q, k, pos, freq, qw, kw, EPS, qo, ko, rstd, axis_pairs=(16, 24), stream=s)
    mx.mxfp4_qk_norm_rope_bwd(dq, dk, q, k, pos, freq, qw, kw, rstd, dqo, dko, dqw, dkw, ws, axis_pairs=(16, 24), stream=s)
    s.synchronize()
    for got, ref in zip((qo, ko, dqo, dko, dqw, dkw), (*out, *want)):
        assert torch.equal(got, ref)


def test_captured_forward_and_backward():
    c = case(40, 4, 2, 64, 32, "bf16", 21)
    leaves = [gpu(c[n]).requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    pos, freq, dq, dk = gpu(c["pos"]), gpu(c["freq"]), gpu(c["dq"]), gpu(c["dk"])
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope

    def step():
        out = qk_norm_rope(leaves[0], leaves[1], pos, freq, leaves[2], leaves[3], EPS)
        return (*out, *torch.autograd.grad(out, leaves, (dq, dk)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        with torch.no_grad():
            leaves[0].copy_(rand(leaves[0].shape, torch.bfloat16, 50 + i))
            pos.add_(17)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
