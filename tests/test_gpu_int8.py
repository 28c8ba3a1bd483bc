"""Int8 operands (codes and a scale a row) and their product against plain
implementations in 64 bits. The codes' rule is fp32 arithmetic in a stated
order, so codes and scales are compared bit for bit; the product's sum is
exact, so its tolerance counts the fp32 roundings after it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
F = np.float32


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def pitch(cols):
    return (cols + 127) // 128 * 128


def codes_of(v):
    """The rule: v fp32 [rows][cols] -> codes int8, scales fp32."""
    v = np.ascontiguousarray(v, dtype=F)
    with np.errstate(all="ignore"):
        a = np.max(np.abs(v), axis=1)
        bad = ~np.isfinite(v).all(axis=1)
        up = np.where(a < F(2.0 ** -64), F(2.0 ** 64), F(1))
        inv = np.where(bad | (a == 0), F(0), F(127) / (a * up))
        q = np.rint(v * up[:, None] * inv[:, None])
        return np.where(bad[:, None], 0, q).astype(np.int8), np.where(bad, F("nan"), a / F(127))


def check_codes(codes, scales, v):
    q, s = codes_of(v)
    cols = q.shape[1]
    got = codes.cpu().numpy()
    assert got.shape[1] == pitch(cols) and not got[:, cols:].any()
    assert np.array_equal(got[:, :cols], q)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)


WIDTHS = [1, 3, 8, 127, 128, 129, 512, 777, 1024, 2048, 4096, 5000, 8192, 14336, 16385, 32768]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", WIDTHS)
def test_quantize(cols, dtype):
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    x = rand((6, cols), TYPES[dtype], cols)
    x[2] = 0
    x[3] *= 1e-3
    codes, scales = int8_quantize(x.cuda())
    check_codes(codes, scales, x.float().numpy())
    # the definition: within half a step of the value, the largest at +-127
    s = scales.cpu().double()[:, None]
    far = (codes.cpu()[:, :cols].double() * s - x.double()).abs()
    assert (far <= s * (0.5 + 127 * 4 * U)).all()
    assert (codes.cpu().abs().amax(1)[[0, 1, 3, 4, 5]] == 127).all()


def test_quantize_extremes():
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    x = rand((9, 300), torch.float32, 0)
    x[1, 299] = float("inf")
    x[2, 0] = float("-inf")
    x[3, 150] = float("nan")
    x[4] *= 2.0 ** -140          # subnormal
    x[5] *= 2.0 ** -110
    x[6] = torch.finfo(torch.float32).max
    x[7] = -0.0
    x[8] = torch.linspace(-127, 127, 300)
    codes, scales = int8_quantize(x.cuda())
    check_codes(codes, scales, x.numpy())
    assert torch.isnan(scales[1:4]).all() and not codes[1:4].any()
    assert (codes[6, :300] == 127).all() and scales[7] == 0 and not codes[7].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", [8, 77, 512, 1000, 4096, 5001, 8192, 16384])
@pytest.mark.parametrize("added", [False, True])
def test_norm_codes(cols, dtype, added):
    from mxfp4_quantized_gemm_amd.norm import rms_norm_int8
    dt = TYPES[dtype]
    x, res, w = rand((7, cols), dt, cols), rand((7, cols), dt, cols + 1), rand((cols,), dt, cols + 2) + 1
    x[3] = 0
    res[3] = 0
    out = rms_norm_int8(x.cuda(), w.cuda(), EPS, res.cuda() if added else None)
    h = (x.float() + res.float()).to(dt) if added else x
    if added:
        assert torch.equal(out[2].cpu(), h)
    h64 = h.double()
    r = (1 / torch.sqrt(h64.square().sum(1, keepdim=True) / cols + float(F(EPS)))).float()
    check_codes(out[0], out[1], (h.float() * r * w.float()).numpy())


def test_norm_codes_of_bad_rows_and_wide_weights():
    from mxfp4_quantized_gemm_amd.norm import rms_norm_int8
    x, w = rand((5, 640), torch.bfloat16, 0), rand((640,), torch.float32, 1)
    x[1, 3], x[2, 639] = float("inf"), float("nan")
    codes, scales = rms_norm_int8(x.cuda(), w.cuda(), EPS)
    good = [0, 3, 4]
    r = (1 / torch.sqrt(x.double().square().sum(1, keepdim=True) / 640 + float(F(EPS)))).float()
    check_codes(codes[good], scales[good], (x.float() * r * w)[good].numpy())
    assert torch.isnan(scales[[1, 2]]).all() and not codes[[1, 2]].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", [5, 128, 1000, 4096, 14336, 28672])
def test_gated_codes(cols, dtype):
    """silu is not fp32 arithmetic in a fixed order: codes are held to half a
    step and the stated error of silu; the gate and up halves of one matrix
    have its pitch."""
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    gu = rand((5, 2 * cols), TYPES[dtype], cols, 2.0)
    gu[2, :cols] = -60.0
    gu[3] = 0
    dev = gu.cuda()
    codes, scales = int8_quantize(dev[:, cols:], gate=dev[:, :cols])
    g, u = gu[:, :cols].double(), gu[:, cols:].double()
    v = g / (1 + torch.exp(-g)) * u
    err = v.abs() * (2.0 ** -19 + g.abs() * 2.0 ** -23 + 4 * U)
    s = scales.cpu().double()[:, None]
    a = v.abs().amax(1, keepdim=True)
    assert ((s - a / 127).abs() <= err.amax(1, keepdim=True) / 127 + 2 * U * a / 127).all()
    got = codes.cpu()[:, :cols].double() * s
    assert ((got - v).abs() <= s * (0.5 + 127 * 4 * U) + err).all()
    assert not codes[:, cols:].any()


def test_gate_of_infinity_and_nan():
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    x, g = torch.ones(4, 64), torch.ones(4, 64)
    g[0, 5], g[1, 5], x[2, 7] = float("inf"), float("nan"), float("nan")
    codes, scales = int8_quantize(x.cuda(), gate=g.cuda())
    assert torch.isnan(scales[:3]).all() and not codes[:3].any()
    assert (codes[3, :64] == 127).all()


# ------------------------------------------------------------- product
def operands(M, N, K, seed, full=False):
    rng = np.random.default_rng(seed)
    a = rng.integers(-128, 128, (M, K)).astype(np.int8)
    b = rng.integers(-128, 128, (N, K)).astype(np.int8)
    if full:
        a[:], b[:] = -128, -128
    sa = np.exp(rng.normal(size=M)).astype(F) / 127
    sb = np.exp(rng.normal(size=N)).astype(F) / 127
    return a, b, sa, sb, rng.normal(size=N).astype(F) * 100


def check_product(c, a, b, sa, sb, bias, dtype):
    # fp64 sums of integers below 2^31 are exact
    s = a.astype(np.float64) @ b.astype(np.float64).T
    p = s * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
    ref = p if bias is None else p + bias.astype(np.float64)
    fi = torch.finfo(dtype)
    tol = 4 * U * np.abs(p) + (0 if bias is None else 2 * U * np.abs(ref)) + np.abs(ref) * fi.eps / 2 \
        + fi.smallest_normal * fi.eps / 2
    got = c.detach().cpu().double().numpy()
    assert got.shape == ref.shape
    # half a step past the type's largest value is infinity
    past = np.abs(ref) / (fi.max * (1 + fi.eps / 4))
    with np.errstate(invalid="ignore"):
        good = (np.abs(got - ref) <= tol) & (past <= 1 + 6 * U)
    good |= (got == np.copysign(np.inf, ref)) & (past >= 1 - 6 * U)
    bad = ~good
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist())


def product(M, N, K, dtype, seed, bias=False, full=False):
    from mxfp4_quantized_gemm_amd.int8 import int8_gemm
    a, b, sa, sb, bi = operands(M, N, K, seed, full)
    d = [torch.from_numpy(t).cuda() for t in (a, sa, b, sb)]
    c = int8_gemm(*d, bias=torch.from_numpy(bi).cuda() if bias else None, out_dtype=dtype)
    check_product(c, a, b, sa, sb, bi if bias else None, dtype)


SIZES = [(1, 1, 1), (1, 16, 128), (1, 17, 128), (1, 4096, 1024), (2, 100, 256), (3, 33, 77), (7, 1024, 4096),
         (8, 640, 384), (15, 256, 640), (16, 256, 14336), (16, 1000, 128), (17, 64, 128), (31, 129, 256), (32, 512, 2048),
         (33, 65, 16), (48, 4096, 4096), (63, 63, 63), (64, 64, 64), (64, 128, 128), (64, 1024, 8192), (65, 200, 512),
         (100, 96, 896), (127, 255, 384), (128, 128, 128), (128, 4096, 4096), (129, 300, 1000), (200, 513, 1152), (256, 256, 256),
         (255, 257, 384), (257, 512, 2816), (300, 260, 128), (512, 768, 640), (700, 1100, 1408),
         (1024, 1024, 1024), (1000, 2050, 1152), (2048, 512, 896)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_product(size, dtype):
    product(*size, TYPES[dtype], seed=sum(size), bias=dtype != "bf16")


@pytest.mark.parametrize("M", [1, 5, 16, 40, 64, 100, 128, 320])
def test_product_largest_sums(M):
    """-128 * -128 in every place of the longest sum: just below 2^31."""
    product(M, 96, 131071, torch.float32, seed=M, full=True)
    product(M, 96, 131071 // 128 * 128, torch.float32, seed=M, full=True)


@pytest.mark.parametrize("size", [(1, 200, 256), (16, 96, 128), (50, 200, 384), (300, 500, 256), (1100, 520, 256)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("lda,ldb,off", [(0, 0, 0), (16, 32, 0), (48, 16, 16), (1, 0, 0), (0, 7, 3)])
def test_product_pitches_and_alignment(size, lda, ldb, off):
    """Operands inside wider matrices (whose other bytes are not zero) and a
    pitched output whose surroundings stay as they were."""
    import mxfp4_quantized_gemm_amd as mx
    M, N, K = size
    a, b, sa, sb, _ = operands(M, N, K, 5)

    def inside(t, more):
        wide = torch.full((t.shape[0] * (t.shape[1] + more) + off + 64,), 99, dtype=torch.int8, device="cuda")
        v = wide[off:off + t.shape[0] * (t.shape[1] + more)].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(torch.from_numpy(t))
        return v
    c = torch.full((M + 2, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    need = mx.mxfp4_int8_gemm_workspace_bytes(M, N, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    out = c[1:M + 1, 3:N + 3]
    mx.mxfp4_int8_gemm(inside(a, lda), torch.from_numpy(sa).cuda(), inside(b, ldb), torch.from_numpy(sb).cuda(),
                       None, out, ws)
    check_product(out, a, b, sa, sb, None, torch.bfloat16)
    assert (c[0] == 7).all() and (c[-1] == 7).all() and (c[:, :3] == 7).all() and (c[:, N + 3:] == 7).all()


@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_scales_of_zero_infinity_and_nan(M):
    from mxfp4_quantized_gemm_amd.int8 import int8_gemm
    a, b, sa, sb, _ = operands(M, 70, 256, 9)
    sa[0], sb[3], sb[5] = np.nan, np.nan, 0
    c = int8_gemm(*[torch.from_numpy(t).cuda() for t in (a, sa, b, sb)], out_dtype=torch.float32).cpu()
    assert torch.isnan(c[0]).all() and torch.isnan(c[:, 3]).all()
    assert (c[1:, 5] == 0).all() and torch.isfinite(c[1:, 6:]).all()


def test_empty_products():
    from mxfp4_quantized_gemm_amd.int8 import int8_gemm, int8_linear
    q, s = torch.zeros(4, 128, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    assert int8_gemm(q[:0], s[:0], q, s).shape == (0, 4)
    assert int8_gemm(q, s, q[:0], s[:0]).shape == (4, 0)
    assert int8_linear(torch.zeros(0, 100, dtype=torch.bfloat16, device="cuda"), q, s).shape == (0, 4)


# ------------------------------------------------- layers and blocks
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", [(1, 96, 256), (5, 70, 333), (64, 512, 1000), (400, 384, 640)])
def test_linear(rows, n, k, dtype):
    from mxfp4_quantized_gemm_amd.int8 import Int8Linear
    x, w, bias = rand((rows, k), TYPES[dtype], 1), rand((n, k), TYPES[dtype], 2), rand((n,), torch.float32, 3)
    layer = Int8Linear.from_weight(w.cuda(), bias.cuda())
    y = layer(x.cuda())
    assert y.dtype == TYPES[dtype]
    qx, sx = codes_of(x.float().numpy())
    qw, sw = codes_of(w.float().numpy())
    check_product(y, qx, qw, sx, sw, bias.numpy(), TYPES[dtype])
    # leading dimensions, and a weight without the padding columns
    if rows == 64:
        assert torch.equal(layer(x.cuda().view(8, 8, k)), y.view(8, 8, n))
        from mxfp4_quantized_gemm_amd.int8 import int8_linear
        assert torch.equal(int8_linear(x.cuda(), torch.from_numpy(qw).cuda(), layer.scales, layer.bias), y)


def test_state_dict_round_trip():
    from mxfp4_quantized_gemm_amd.int8 import Int8Linear
    layer = Int8Linear.from_weight(rand((48, 200), torch.bfloat16, 0).cuda())
    other = Int8Linear(200, 48, device="cuda")
    other.load_state_dict(layer.state_dict())
    x = rand((3, 200), torch.bfloat16, 1).cuda()
    assert torch.equal(layer(x), other(x))


def test_mlp_block():
    """The block is its parts' composition, bit for bit."""
    from mxfp4_quantized_gemm_amd import int8, norm
    T, K, Fh = 37, 320, 500
    x, res = rand((T, K), torch.bfloat16, 0).cuda(), rand((T, K), torch.bfloat16, 1).cuda()
    w = rand((K,), torch.bfloat16, 2).cuda()
    gu, gs = int8.int8_quantize(rand((2 * Fh, K), torch.bfloat16, 3).cuda())
    dn, ds = int8.int8_quantize(rand((K, Fh), torch.bfloat16, 4).cuda())
    y, h = int8.int8_mlp(x, w, EPS, gu, gs, dn, ds, residual=res)
    codes, scales, h2 = norm.rms_norm_int8(x, w, EPS, residual=res)
    mid = int8.int8_gemm(codes, scales, gu, gs)
    codes, scales = int8.int8_quantize(mid[:, Fh:], gate=mid[:, :Fh])
    assert torch.equal(h, h2) and torch.equal(y, int8.int8_gemm(codes, scales, dn, ds))
    y3, h3 = int8.int8_mlp(x.view(1, T, K), w, EPS, gu, gs, dn, ds)
    assert y3.shape == (1, T, K) and h3.shape == (1, T, K)


@pytest.mark.parametrize("T,K,N", [(2, 1024, 768), (48, 1024, 768), (512, 1024, 768), (65, 4096, 4100), (2100, 512, 2100)])
def test_graph_replays(T, K, N):
    """Decode's sequence in a HIP graph: every replay equals the eager result,
    with the inputs overwritten and other work in between."""
    from mxfp4_quantized_gemm_amd import int8, norm
    x, res = rand((T, K), torch.bfloat16, 0).cuda(), rand((T, K), torch.bfloat16, 1).cuda()
    w = rand((K,), torch.bfloat16, 2).cuda()
    b, sb = int8.int8_quantize(rand((N, K), torch.bfloat16, 3).cuda())

    def step():
        q, s, h = norm.rms_norm_int8(x, w, EPS, residual=res)
        return int8.int8_gemm(q, s, b, sb), h
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(rand((T, K), torch.bfloat16, 10 + i))
        want = step()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), i
        torch.randn(1000, device="cuda").sum()


# --------------------------------------- offsets past 32 bits, C-named calls
def sampled(c, a, b, sa, sb, rows, cols):
    """Rows and columns of C against fp64 sums of the same codes."""
    s = a[rows].double() @ b[cols].double().t()
    p = s * sa[rows].double()[:, None] * sb[cols].double()
    tol = p.abs() * (4 * U + torch.finfo(c.dtype).eps / 2) + 1e-30
    got = c[rows][:, cols].double()
    assert ((got - p).abs() <= tol).all()


@pytest.mark.parametrize("M,N,K", [(70000, 96, 65536), (3, 70000, 65536), (48, 70000, 65536), (40000, 60000, 128),
                                   (70000, 200, 65504)],
                         ids=["A over 4 GiB", "B over 4 GiB, few", "B over 4 GiB", "C over 4 GiB", "A over 4 GiB, general"])
def test_product_past_32_bits(M, N, K):
    from mxfp4_quantized_gemm_amd.int8 import int8_gemm
    g = torch.Generator(device="cuda").manual_seed(M + N)
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    b = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(M, device="cuda", generator=g) + 0.1, torch.rand(N, device="cuda", generator=g) + 0.1
    c = int8_gemm(a, sa, b, sb)
    pick = lambda n: torch.tensor(sorted({0, 1, n // 3, n // 2, n - 2, n - 1} & set(range(n))), device="cuda")
    sampled(c, a, b, sa, sb, pick(M), pick(N))
    del a, b, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cols", [32768, 32767])
def test_rows_past_32_bits(cols):
    """70000 rows: over 4 GiB of bf16, both sides of every 32-bit border."""
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    from mxfp4_quantized_gemm_amd.norm import rms_norm_int8
    rows = 70000
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:] = torch.arange(-2, cols - 2, device="cuda") % 97 - 48.0
    x *= (torch.arange(rows, device="cuda") % 31 + 1.0)[:, None]
    at = [0, 1, 32767, 32768, 65535, 65536, 65538, rows - 1]
    codes, scales = int8_quantize(x)
    check_codes(codes[at], scales[at], x[at].float().cpu().numpy())
    codes, scales = rms_norm_int8(x, None, EPS)
    h = x[at].cpu()
    r = (1 / torch.sqrt(h.double().square().sum(1, keepdim=True) / cols + float(F(EPS)))).float()
    check_codes(codes[at], scales[at], (h.float() * r).numpy())
    del x, codes
    torch.cuda.empty_cache()


def test_c_named_calls_on_a_stream():
    """The ctypes binding, with the caller's buffers and stream, gives the
    bits of the functions that allocate."""
    import mxfp4_quantized_gemm_amd as mx
    from mxfp4_quantized_gemm_amd import int8, norm
    T, K, N = 70, 333, 96
    x, res, dy, dh = (rand((T, K), torch.bfloat16, i).cuda() for i in range(4))
    w = rand((K,), torch.bfloat16, 5).cuda()
    wq, ws = int8.int8_quantize(rand((N, K), torch.bfloat16, 6).cuda())
    q, s, h = norm.rms_norm_int8(x, w, EPS, residual=res)
    c = int8.int8_gemm(q, s, wq, ws)
    g, gs = int8.int8_quantize(x, gate=res)
    leaves = [t.clone().requires_grad_(True) for t in (x, res, w)]
    y, _ = out = norm.rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    dx, _, dw = torch.autograd.grad(out, leaves, (dy, dh))
    torch.cuda.synchronize()

    st = torch.cuda.Stream()
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")
    h2, y2, dx2, dw2, rstd = new(T, K), new(T, K), new(T, K), new(K), new(T, dtype=torch.float32)
    q2, s2 = new(T, 384, dtype=torch.int8), new(T, dtype=torch.float32)
    g2, gs2 = new(T, 384, dtype=torch.int8), new(T, dtype=torch.float32)
    c2 = new(T, N)
    need = mx.mxfp4_int8_gemm_workspace_bytes(T, N, 384)
    gemm_ws = new(need, dtype=torch.uint8) if need else None
    bwd_ws = new(mx.mxfp4_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8)
    torch.cuda.synchronize()
    mx.mxfp4_rmsnorm_int8(x, res, w, EPS, h2, q2, s2, stream=st)
    mx.mxfp4_int8_gemm(q2, s2, wq, ws, None, c2, gemm_ws, stream=st)
    mx.mxfp4_int8_quantize(x, res, g2, gs2, stream=st)
    mx.mxfp4_rmsnorm(x, res, w, EPS, None, y2, rstd, stream=st)
    mx.mxfp4_rmsnorm_bwd(dy, dh, h2, w, rstd, dx2, dw2, bwd_ws, stream=st.cuda_stream)
    st.synchronize()
    for a, b in ((h, h2), (q, q2), (s, s2), (c, c2), (g, g2), (gs, gs2), (y, y2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        mx.mxfp4_rmsnorm(x, res, w, EPS, None, y2[:3], rstd)
    with pytest.raises(TypeError):
        mx.mxfp4_rmsnorm(x, res.float(), w, EPS, None, y2, rstd)
    with pytest.raises(ValueError):
        mx.mxfp4_int8_gemm(q2.t(), s2, wq, ws, None, c2, None)


@pytest.mark.parametrize("M,N,K", [(64, 100, 4096), (200, 130, 2048), (33, 4099, 1024), (300, 1000, 8192)])
def test_product_without_its_workspace_is_refused(M, N, K):
    import mxfp4_quantized_gemm_amd as mx
    need = mx.mxfp4_int8_gemm_workspace_bytes(M, N, K)
    a, b = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(N, K, dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    c = torch.empty(M, N, device="cuda")
    if need:
        with pytest.raises(mx.MXFP4Error) as e:
            mx.mxfp4_int8_gemm(a, sa, b, sb, None, c, None)
        assert e.value.status == 1
        with pytest.raises(mx.MXFP4Error) as e:
            mx.mxfp4_int8_gemm(a, sa, b, sb, None, c, torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 4
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    mx.mxfp4_int8_gemm(a, sa, b, sb, None, c, ws)
    assert not c.any()


# Sizes past those above, so that every tile, split and streaming form is
# reached: several rounds of tiles, one and an odd number of k-tiles, ragged
# edges in both directions.
LARGER = [(1, 5003, 384), (5, 5000, 2048), (9, 12010, 384), (16, 6144, 1408), (20, 5001, 640), (40, 5003, 256),
          (64, 8200, 128), (64, 28672, 256), (129, 14336, 384), (200, 4100, 8192), (60, 8200, 8192), (65, 8000, 8192), (65, 14000, 14336), (130, 14000, 14336), (400, 2050, 8192),
          (512, 4100, 2048), (520, 8190, 640), (640, 14337, 256), (1300, 2100, 512), (2301, 3503, 640), (3000, 3000, 384),
          (5001, 5100, 128), (4097, 4097, 256)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", LARGER, ids=lambda s: "x".join(map(str, s)))
def test_larger_product(size, dtype):
    product(*size, TYPES[dtype], seed=sum(size), bias=dtype == "bf16")


# streamed weights of 64 MB and more, whole and split, splits of other sizes,
# the largest tiles in one and two rounds
STREAMED = [(40, 28700, 2432, "fp16"), (3, 20000, 6912, "fp32"), (16, 28672, 4096, "bf16"), (1, 13121, 10240, "fp16"),
            (1, 7828, 17280, "bf16"), (1, 4133, 17408, "fp32"), (2, 2371, 28800, "fp16"), (2, 8485, 7296, "bf16"),
            (29, 1, 3840, "fp32"), (118, 2195, 8576, "fp16"), (65, 8700, 7296, "bf16"), (1300, 18200, 384, "bf16"),
            (642, 18153, 128, "fp16"), (642, 18153, 256, "fp32")]


@pytest.mark.parametrize("size", STREAMED, ids=lambda s: "x".join(map(str, s)))
def test_streamed_product(size):
    M, N, K, dtype = size
    product(M, N, K, TYPES[dtype], seed=M + N + K, bias=dtype == "bf16")
