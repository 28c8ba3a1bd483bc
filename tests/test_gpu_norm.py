"""RMS norm with the residual's addition and its gradient against plain
implementations in 64 bits. Tolerances count roundings: half a step of the
output's type (torch.finfo(t).eps / 2, and half its smallest subnormal), and
one 2^-24 for each fp32 rounding on the way."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
# one value, one wave, odd widths, every width of work-group, vector and
# single-value rows
WIDTHS = [1, 2, 7, 8, 63, 64, 200, 512, 520, 1000, 1024, 1111, 1536, 4096, 4097, 8192, 8200, 16384,
          16385, 32768]


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def forward64(x, res, w, eps=EPS):
    """(h as held, r, y) in 64 bits; eps is the fp32 number that the call takes."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    h64 = h.double()
    r = 1 / torch.sqrt(h64.square().mean(1, keepdim=True) + torch.tensor(eps, dtype=torch.float32).double())
    return h, r, h64 * r * (1.0 if w is None else w.double())


def near(got, ref, tol, what):
    got = got.detach().cpu().double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() / tol).max())}"


def check_forward(x, res, w, y, h, eps=EPS):
    h_ref, r, ref = forward64(x, res, w, eps)
    if res is not None:
        assert torch.equal(h.detach().cpu(), h_ref)
    # r, h r and the product with w round to fp32 once each; then y's type
    near(y, ref, 4 * U * ref.abs() + half_step(ref, x.dtype), "y")


def check_gradient(x, res, w, dy, dh, dx, dw):
    h, r, _ = forward64(x, res, w)
    u = h.double() * r
    g = dy.double() * (1.0 if w is None else w.double())
    gu = (g * u).mean(1, keepdim=True)
    ref = r * (g - u * gu) + (0 if dh is None else dh.double())
    # u: 2 roundings, g: 1; the row's sum: at most 32 values a thread, 6
    # steps in a wave, 16 waves and the division, so 64 U of the mean of |g u|
    # covers it; then the difference, the product with r and the addition
    tol = U * (r * (4 * g.abs() + 8 * (u * gu).abs() + 64 * u.abs() * (g * u).abs().mean(1, keepdim=True))
               + 2 * ref.abs() + (0 if dh is None else 2 * dh.double().abs()))
    near(dx, ref, tol + half_step(ref, x.dtype), "dx")
    if dw is not None:
        t = dy.double() * u
        rows = x.shape[0]
        near(dw, t.sum(0), U * (rows + 24) * t.abs().sum(0) + half_step(t.sum(0), dw.dtype), "dw")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_and_gradient(cols, dtype):
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    dt, rows = TYPES[dtype], 5
    x, res, dy, dh = (rand((rows, cols), dt, 10 * cols + i) for i in range(4))
    w = rand((cols,), dt, 10 * cols + 5) + 1
    leaves = [t.cuda().requires_grad_(True) for t in (x, res, w)]
    y, h = rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    check_forward(x, res, w, y, h)
    dx, dres, dw = torch.autograd.grad((y, h), leaves, (dy.cuda(), dh.cuda()))
    assert torch.equal(dx, dres) and dw.dtype == dt
    check_gradient(x, res, w, dy, dh, dx, dw)
    # without autograd, the same bits
    with torch.no_grad():
        y2, h2 = rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cols", [64, 77, 4096, 4100])
def test_weight_in_32_bits(cols, dtype):
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    dt = TYPES[dtype]
    x, dy = rand((33, cols), dt, 1), rand((33, cols), dt, 2)
    w = rand((cols,), torch.float32, 3) + 1
    xg, wg = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    y = rms_norm(xg, wg, EPS)
    check_forward(x, None, w, y, None)
    dx, dw = torch.autograd.grad(y, (xg, wg), dy.cuda())
    assert dw.dtype == torch.float32
    check_gradient(x, None, w, dy, None, dx, dw)


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 4, 5, 1023, 1025, 4097])
@pytest.mark.parametrize("cols", [48, 96, 1000])
def test_row_counts(rows, cols):
    """Rows below, at and above the gradient's work-groups; none at all."""
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x, dy = rand((rows, cols), torch.bfloat16, rows), rand((rows, cols), torch.bfloat16, rows + 1)
    w = rand((cols,), torch.bfloat16, 3)
    xg, wg = x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    y = rms_norm(xg, wg, EPS)
    dx, dw = torch.autograd.grad(y, (xg, wg), dy.cuda())
    assert y.shape == dx.shape == (rows, cols)
    if rows == 0:
        assert torch.equal(dw, torch.zeros_like(dw))
        return
    check_forward(x, None, w, y, None)
    check_gradient(x, None, w, dy, None, dx, dw)


def test_gradient_against_differences():
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    rows, cols, step = 3, 21, 1e-4
    x, res, dy, dh = (rand((rows, cols), torch.float32, i) for i in range(4))
    w = rand((cols,), torch.float32, 5) + 1

    def loss(x, res, w):  # 64 bits throughout, unrounded h
        h = x + res
        r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        return float((h * r * w * dy.double()).sum() + (h * dh.double()).sum())
    leaves = [t.cuda().requires_grad_(True) for t in (x, res, w)]
    y, h = rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    grads = torch.autograd.grad((y, h), leaves, (dy.cuda(), dh.cuda()))
    base = [t.double() for t in (x, res, w)]
    for k in range(3):
        flat = base[k].reshape(-1)
        for i in range(flat.numel()):
            v = float(flat[i])
            flat[i] = v + step
            up = loss(*base)
            flat[i] = v - step
            down = loss(*base)
            flat[i] = v
            d = (up - down) / (2 * step)
            # h is rounded to fp32 before the norm (2^-24 of h, which moves
            # the gradient as little); differences are good to step^2
            assert abs(float(grads[k].reshape(-1)[i]) - d) <= 1e-5 * max(1.0, abs(d)), (k, i)


def test_strides_and_leading_dimensions():
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    big = rand((6, 3, 400), torch.bfloat16, 1)
    w = rand((128,), torch.bfloat16, 2)
    for off in (0, 8, 3):  # 16-byte aligned rows, and not
        x = big[..., off:off + 128]
        y = rms_norm(big.cuda()[..., off:off + 128], w.cuda(), EPS)
        assert y.shape == (6, 3, 128)
        check_forward(x.reshape(18, 128), None, w, y.reshape(18, 128), None)
    # a view with another column stride, an expanded residual, an expanded gradient
    x, r = rand((40, 64), torch.float32, 3), rand((1, 40), torch.float32, 4)
    w = rand((40,), torch.float32, 5)
    xg = x.cuda().requires_grad_(True)
    rg, wg = r.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    y, h = rms_norm(xg.t(), wg, EPS, residual=rg.expand(64, 40))
    check_forward(x.t().contiguous(), r.expand(64, 40), w, y, h)
    (y.sum() + h.sum()).backward()
    one = torch.ones(64, 40)
    dx = xg.grad.t()
    check_gradient(x.t().contiguous(), r.expand(64, 40), w, one, one, dx, wg.grad)
    near(rg.grad, dx.cpu().double().sum(0, keepdim=True), 64 * U * dx.cpu().double().abs().sum(0, keepdim=True), "dres")


@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_outputs_that_no_loss_reads(use):
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x, res, dy, dh = (rand((9, 160), torch.float32, i) for i in range(4))
    w = rand((160,), torch.float32, 5)
    leaves = [t.cuda().requires_grad_(True) for t in (x, res, w)]
    y, h = rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    loss = 0
    if use != "h":
        loss = loss + (y * dy.cuda()).sum()
    if use != "y":
        loss = loss + (h * dh.cuda()).sum()
    loss.backward()
    zero = torch.zeros_like(dy)
    check_gradient(x, res, w, zero if use == "h" else dy, None if use == "y" else dh, leaves[0].grad,
                   leaves[2].grad)


def test_gradients_that_are_not_wanted():
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x, dy, w = rand((9, 160), torch.bfloat16, 0), rand((9, 160), torch.bfloat16, 1), rand((160,), torch.bfloat16, 2)
    xg, wg = x.cuda().requires_grad_(True), w.cuda()
    rms_norm(xg, wg, EPS).backward(dy.cuda())
    check_gradient(x, None, w, dy, None, xg.grad, None)
    wg = w.cuda().requires_grad_(True)
    rms_norm(x.cuda(), wg, EPS).backward(dy.cuda())
    check_gradient(x, None, w, dy, None, xg.grad, wg.grad)
    y = rms_norm(x.cuda(), None, EPS)
    check_forward(x, None, None, y, None)


def test_rows_of_zeros_infinities_and_nan():
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x = rand((6, 256), torch.bfloat16, 0)
    x[1] = 0
    x[2, 17] = float("inf")
    x[3, 250] = float("nan")
    x[4] = torch.finfo(torch.bfloat16).max     # squares leave fp32's range
    w = rand((256,), torch.bfloat16, 1)
    y = rms_norm(x.cuda(), w.cuda(), EPS).cpu()
    good = [0, 1, 4, 5]
    check_forward(x[good], None, w, y[good], None)
    assert torch.equal(y[1], torch.zeros(256, dtype=torch.bfloat16).copysign(y[1]))
    assert torch.isnan(y[2, 17]) and (y[2, :17] == 0).all()  # r = 0: inf * 0, finite * 0
    assert torch.isnan(y[3]).all()


def test_in_place_residual_stream():
    """h may be the residual's own memory."""
    import mxfp4_quantized_gemm_amd as mx
    x, res, w = rand((70, 1536), torch.bfloat16, 0), rand((70, 1536), torch.bfloat16, 1), rand((1536,), torch.bfloat16, 2)
    h, y = res.cuda(), torch.empty(70, 1536, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_rmsnorm(x.cuda(), h, w.cuda(), EPS, h, y, None)
    check_forward(x, res, w, y, h)


def test_pitched_outputs_leave_their_surroundings():
    import mxfp4_quantized_gemm_amd as mx
    x, w = rand((9, 100), torch.float16, 0), rand((100,), torch.float16, 2)
    y = torch.full((9, 120), 7.0, dtype=torch.float16, device="cuda")
    mx.mxfp4_rmsnorm(x.cuda(), None, w.cuda(), EPS, None, y[:, 8:108], None)
    check_forward(x, None, w, y[:, 8:108], None)
    assert (y[:, :8] == 7).all() and (y[:, 108:] == 7).all()


def test_another_stream_and_repeated_calls():
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x, w = rand((300, 4096), torch.bfloat16, 0).cuda(), rand((4096,), torch.bfloat16, 1).cuda()
    want = rms_norm(x, w, EPS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [rms_norm(x, w, EPS) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got)


def test_norm_in_front_of_an_mxfp4_linear():
    """The training path: norm (with the residual stream) into MXFP4Linear and
    back; the layer's own gradients are the ones that its tests pin."""
    from mxfp4_quantized_gemm_amd.linear import MXFP4Linear
    from mxfp4_quantized_gemm_amd.norm import RMSNorm
    norm, layer = RMSNorm(256, device="cuda"), MXFP4Linear(256, 128, device="cuda")
    x, res = (rand((64, 256), torch.bfloat16, i).cuda().requires_grad_(True) for i in range(2))
    y, h = norm(x, res)
    out = layer(y)
    dy, = torch.autograd.grad(out, y, torch.ones_like(out), retain_graph=True)
    (out.sum() + h.float().sum()).backward()
    check_gradient(x.detach().cpu(), res.detach().cpu(), norm.weight.detach().cpu(), dy.cpu(),
                   torch.ones(64, 256), x.grad, norm.weight.grad)
    assert torch.equal(x.grad, res.grad)
