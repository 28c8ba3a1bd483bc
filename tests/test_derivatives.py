"""Calls whose derivative the library does not have refuse the inputs that
would need it (no GPU: the refusals come before any other check)."""
import pytest
import torch

from mxfp4_quantized_gemm_amd import int8, norm


def operands():
    """x [4][64], codes and scales of 8 rows, a bias, all in host memory."""
    return (torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.int8), torch.ones(8),
            torch.zeros(8))


def leaf(t):
    return t.clone().requires_grad_(True)


def products(mark):
    """Every call with a product, with one of its scales or its bias marked by ``mark``."""
    x, q, s, b = operands()
    down, ds = torch.zeros(64, 128, dtype=torch.int8), torch.ones(64)
    w = torch.ones(64, dtype=torch.bfloat16)
    return {
        "gemm a_scales": lambda: int8.int8_gemm(q, mark(s), q, s),
        "gemm b_scales": lambda: int8.int8_gemm(q, s, q, mark(s)),
        "gemm bias": lambda: int8.int8_gemm(q, s, q, s, bias=mark(b)),
        "linear w_scales": lambda: int8.int8_linear(x, q, mark(s)),
        "linear bias": lambda: int8.int8_linear(x, q, s, bias=mark(b)),
        "mlp gate_up_scales": lambda: int8.int8_mlp(x, w, 1e-5, q, mark(s), down, ds),
        "mlp down_scales": lambda: int8.int8_mlp(x, w, 1e-5, q, s, down, mark(ds)),
    }


@pytest.mark.parametrize("call", list(products(leaf)))
def test_products_refuse_to_be_recorded(call):
    with pytest.raises(RuntimeError, match="no gradient"):
        products(leaf)[call]()
    with torch.no_grad(), pytest.raises(ValueError, match="GPU memory"):
        products(leaf)[call]()


# ------------------------------------------------------------ forward mode
def dual(t):
    import torch.autograd.forward_ad as fwd
    return fwd.make_dual(t.clone(), torch.ones_like(t))


def rows(mark):
    """The norm and the quantizers, with one of their inputs marked by ``mark``."""
    x, w = torch.zeros(4, 64), torch.ones(64)
    return {
        "norm x": lambda: norm.rms_norm(mark(x), w),
        "norm weight": lambda: norm.rms_norm(x, mark(w)),
        "norm residual": lambda: norm.rms_norm(x, w, residual=mark(x)),
        "norm x, recorded too": lambda: norm.rms_norm(mark(x), w.clone().requires_grad_(True)),
        "norm codes x": lambda: norm.rms_norm_int8(mark(x), w),
        "norm codes weight": lambda: norm.rms_norm_int8(x, mark(w)),
        "norm codes residual": lambda: norm.rms_norm_int8(x, w, residual=mark(x)),
        "codes x": lambda: int8.int8_quantize(mark(x)),
        "codes gate": lambda: int8.int8_quantize(x, gate=mark(x)),
    }


@pytest.mark.parametrize("call", [*rows(leaf), *products(leaf)])
def test_tangents_are_refused(call):
    """A forward-mode tangent would be dropped: a derivative of zero."""
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="forward-mode"):
                {**rows(dual), **products(dual)}[call]()


# ------------------------------------------------------------ tracing
@pytest.mark.filterwarnings("ignore::DeprecationWarning")
@pytest.mark.parametrize("call", [*rows(leaf), *products(leaf)])
def test_tracing_is_refused(call):
    """A trace would hold the outputs' allocation alone, and its replays return
    memory that nothing wrote."""
    def traced(t):
        with torch.no_grad():
            return {**rows(lambda a: a), **products(lambda a: a)}[call]()
    with pytest.raises(RuntimeError, match="trace"):
        torch.jit.trace(traced, (torch.zeros(1),), check_trace=False)
