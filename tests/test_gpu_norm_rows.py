"""The norm's gradient where a work-group takes several rows (the sums over its
rows, the slots it uses again, the wide form that keeps them in LDS), with row
pitches of its own, past 32 bits; and row operators on more rows than one grid
dimension holds. Against the formula in 64 bits."""
import pytest
import torch

import mxfp4_quantized_gemm_amd as mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def rand(shape, dtype, seed, add=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) + add).to(dtype)


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def near(got, ref, tol, what):
    far = (got.double() - ref).abs() / tol
    assert bool((far <= 1).all()), f"{what}: worst {float(far.nan_to_num(1e9).max())} of the tolerance"


def work_groups(rows, cols):
    """Partial sums of the weight's gradient: the workspace holds one row of fp32 each."""
    return mx.mxfp4_rmsnorm_bwd_workspace_bytes(rows, cols) // (4 * cols)


def check(x, w, dy, dh, dx, dw, eps=EPS):
    """dx and dw of y = norm(x) w (and of h = x, with gradient dh)."""
    rows, cols = x.shape
    h = x.double()
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + torch.tensor(eps, dtype=torch.float32).double())
    u, d = h * r, dy.double()
    g = d * (1.0 if w is None else w.double())
    gu = (g * u).mean(1, keepdim=True)
    ref = r * (g - u * gu) + (0 if dh is None else dh.double())
    # r, u, g round once each, u gu twice more, then the difference, the product with
    # r and the addition; the row's sum: at most 32 terms a thread, 6 steps in a wave,
    # 16 waves and the division
    tol = U * (r * (4 * g.abs() + 8 * (u * gu).abs() + 64 * u.abs() * (g * u).abs().mean(1, keepdim=True))
               + 2 * ref.abs() + (0 if dh is None else 2 * dh.double().abs()))
    near(dx, ref, tol + half_step(ref, x.dtype), "dx")
    if dw is None:
        return
    t = d * u
    # a term: r and u round (2) and the product with dy is fused. The sum in fp32: at most
    # rows / work-groups (rounded up, and as many again where a work-group takes several
    # at a time) steps in a work-group, 16 where its parts meet, parts / 32 a half-wave, 32 across them
    parts = work_groups(rows, cols)
    depth = -(-rows // parts) + 16 + -(-parts // 32) + 32
    ref = t.sum(0)
    near(dw, ref, U * (depth + 2) * t.abs().sum(0) + half_step(ref, dw.dtype), "dw")


def gradient(rows, cols, dtype, wtype, seed, added=True):
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x = rand((rows, cols), dtype, seed).requires_grad_(True)
    w = rand((cols,), wtype, seed + 1, 1.0).requires_grad_(True)
    dy = rand((rows, cols), dtype, seed + 2)
    if not added:
        y = rms_norm(x, w, EPS)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        dh = None
    else:
        # a residual of zeros: h is x, and h's own gradient joins
        dh = rand((rows, cols), dtype, seed + 3)
        y, h = rms_norm(x, w, EPS, residual=torch.zeros_like(x))
        dx, dw = torch.autograd.grad((y, h), (x, w), (dy, dh))
    assert dw.dtype == wtype
    check(x.detach(), w.detach(), dy, dh, dx, dw)


# several rows a work-group at every number of waves a row, in whole and ragged
# rounds; the wide form (above 8192 columns and odd, or above 16384)
SEVERAL = [(40000, 40), (40000, 100), (20000, 200), (5000, 300), (9001, 500), (5000, 1000), (1100, 1111), (1541, 1111),
           (1100, 1500), (1537, 4096), (1100, 4095), (2049, 2048), (600, 4100), (600, 8192), (700, 8200), (513, 8191),
           (600, 8201), (600, 16383), (600, 16384), (513, 16385), (600, 20000), (600, 32767), (700, 32768)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SEVERAL, ids=lambda s: "x".join(map(str, s)))
def test_several_rows_a_work_group(size, dtype):
    rows, cols = size
    assert rows > work_groups(rows, cols), "one row a work-group only"
    gradient(rows, cols, TYPES[dtype], TYPES[dtype], rows + cols, added=cols % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [(3, 5000), (600, 8200), (300, 8201), (600, 16383), (513, 16385), (600, 20000), (300, 32767),
                                  (600, 32768)], ids=lambda s: "x".join(map(str, s)))
def test_weight_in_32_bits_beside_wide_rows(size, dtype):
    gradient(*size, TYPES[dtype], torch.float32, sum(size), added=size[1] % 2 == 1)


def apart(t, before, after):
    """t as the middle columns of a wider matrix of NaN."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[:, before:before + t.shape[1]]
    v.copy_(t)
    return wide, v


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(700, 1111), (600, 4096), (40, 100), (600, 8201), (600, 20000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_rows_inside_wider_matrices(size, dtype):
    """dy, dh, h and dx with pitches and offsets of their own, through the C-named call."""
    (rows, cols), dt = size, TYPES[dtype]
    x, dy, dh = (rand((rows, cols), dt, i) for i in range(3))
    w = rand((cols,), dt, 3, 1.0)
    _, xv = apart(x, 3, 5)
    _, dyv = apart(dy, 1, 0)
    _, dhv = apart(dh, 8, 9)
    wide, dx = apart(torch.zeros_like(x), 5, 2)
    y, rstd, dw = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(w)
    ws = torch.empty(mx.mxfp4_rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    mx.mxfp4_rmsnorm(xv, None, w, EPS, None, y, rstd)
    mx.mxfp4_rmsnorm_bwd(dyv, dhv, xv, w, rstd, dx, dw, ws)
    check(x, w, dy, dh, dx, dw)
    assert wide[:, :5].isnan().all() and wide[:, -2:].isnan().all()


@pytest.mark.parametrize("cols", [32768, 32767])
def test_gradient_past_32_bits(cols):
    """Over 4 GiB of bf16 in each of dy, h and dx; the rows repeat, so the
    weight's gradient is a multiple of one period's."""
    rows, period = 70000, 7
    base, dyb = rand((period, cols), torch.bfloat16, 1), rand((period, cols), torch.bfloat16, 2)
    w = rand((cols,), torch.bfloat16, 3, 1.0)
    x, dy = base.repeat(rows // period, 1), dyb.repeat(rows // period, 1)
    assert x.shape[0] == rows and x.numel() * 2 > 1 << 32
    rstd = torch.empty(rows, device="cuda")
    dw, dx = torch.empty_like(w), torch.empty_like(x)
    ws = torch.empty(mx.mxfp4_rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    mx.mxfp4_rmsnorm(x, None, w, EPS, None, dx, rstd)  # (y goes where dx comes later)
    mx.mxfp4_rmsnorm_bwd(dy, None, x, w, rstd, dx, dw, ws)
    check(base, w, dyb, None, dx[:period], None)
    assert bool((dx.view(-1, period, cols) == dx[:period]).all())
    r = 1 / torch.sqrt(base.double().square().mean(1, keepdim=True) + torch.tensor(EPS, dtype=torch.float32).double())
    t = dyb.double() * base.double() * r
    parts = work_groups(rows, cols)
    depth = -(-rows // parts) + 16 + -(-parts // 32) + 32
    ref = t.sum(0) * (rows // period)
    near(dw, ref, U * (depth + 2) * t.abs().sum(0) * (rows // period) + half_step(ref, torch.bfloat16), "dw")
    del x, dy, dx
    torch.cuda.empty_cache()


# more work-groups than one grid dimension of 2^20 holds: a row each above 1024
# columns, sixteen up to 128
@pytest.mark.parametrize("rows,cols", [((1 << 20) + 1030, 1100), ((1 << 24) + 40, 24)], ids=["a row each", "sixteen rows each"])
def test_more_rows_than_a_grid_dimension(rows, cols):
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    from mxfp4_quantized_gemm_amd.norm import rms_norm, rms_norm_int8
    period = 10
    base = rand((period, cols), torch.bfloat16, 5)
    base[3] = 0
    x = base.repeat(-(-rows // period), 1)[:rows]
    edge = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, rows - 2, rows - 1]

    def same(out, small):
        """Every row is its row of the small call's, whose values other tests hold to the formula."""
        n = rows // period * period
        return bool((out[:n].reshape(-1, *small.shape) == small).all()) and bool((out[n:] == small[:rows - n]).all())
    with torch.no_grad():
        y, small = rms_norm(x, None, EPS), rms_norm(base, None, EPS)
    h = base.double()
    ref = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    near(small, ref, 4 * U * ref.abs() + half_step(ref, torch.bfloat16), "y")
    assert same(y, small) and all(torch.equal(y[i], small[i % period]) for i in edge)
    del y
    for call in (int8_quantize, lambda t: rms_norm_int8(t, None, EPS), lambda t: int8_quantize(t, gate=t)):
        (q, s), (q0, s0) = call(x), call(base)
        assert same(q, q0) and same(s, s0)
        del q, s
    torch.cuda.empty_cache()
