"""Int8Linear as part of a model: its codes, scales and bias keep their types
and values when the model is cast. (No GPU: nothing is multiplied.)"""
import pytest
import torch

from mxfp4_quantized_gemm_amd import int8


def layer():
    m = int8.Int8Linear(200, 6, bias=True)
    g = torch.Generator().manual_seed(0)
    m.weight.copy_(torch.randint(-127, 128, m.weight.shape, generator=g))
    m.scales.copy_(torch.rand(6, generator=g) * 1e-3)
    m.bias.copy_(torch.randn(6, generator=g))
    return m


CASTS = {"bfloat16": lambda m: m.bfloat16(), "half": lambda m: m.half(), "double": lambda m: m.double(),
         "to bfloat16": lambda m: m.to(torch.bfloat16), "to device and type": lambda m: m.to("cpu", torch.float16),
         "type": lambda m: m.type(torch.bfloat16), "back and forth": lambda m: m.half().float()}


@pytest.mark.parametrize("cast", list(CASTS))
def test_casts_of_a_model_leave_the_layer_as_it_is(cast):
    m = layer()
    want = {k: v.clone() for k, v in m.state_dict().items()}
    model = torch.nn.Sequential(torch.nn.Linear(4, 200), m)
    CASTS[cast](model)
    assert set(m.state_dict()) == set(want)
    for k, v in m.state_dict().items():
        assert v.dtype == want[k].dtype and torch.equal(v, want[k]), k
    if cast != "back and forth":  # the rest of the model is cast
        assert model[0].weight.dtype != torch.float32


def test_moves_of_a_model_move_the_layer():
    m = layer().to("meta", torch.bfloat16)
    assert all(b.device.type == "meta" for b in m.buffers())
    assert [b.dtype for b in m.buffers()] == [torch.int8, torch.float32, torch.float32]
    assert int8.Int8Linear(200, 6).half().bias is None


def test_from_weight_copies_the_bias(monkeypatch):
    """Steps of an optimizer on the source's bias must not reach the layer, whose codes they do not reach."""
    monkeypatch.setattr(int8, "int8_quantize", lambda w: (torch.zeros(len(w), 256, dtype=torch.int8), torch.ones(len(w))))
    source = torch.nn.Linear(200, 6)
    want = source.bias.detach().clone()
    for bias in (source.bias, source.bias.to(torch.bfloat16), torch.stack((want, want), 1)[:, 0]):
        m = int8.Int8Linear.from_weight(source.weight, bias)
        with torch.no_grad():
            held = bias.detach().float().clone()
            bias += 1
        assert m.bias.dtype == torch.float32 and m.bias.is_contiguous() and not m.bias.requires_grad
        assert torch.equal(m.bias, held)
        with torch.no_grad():
            bias -= 1
    with pytest.raises(ValueError, match="bias"):
        int8.Int8Linear.from_weight(source.weight, torch.zeros(1))
    # a bias of another shape, as the product takes it
    assert torch.equal(int8.Int8Linear.from_weight(source.weight, want[None]).bias, want)
