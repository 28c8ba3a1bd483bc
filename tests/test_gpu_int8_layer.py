"""Int8Linear in GPU memory after its model was cast, and with a bias that its
source goes on training."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cast", ["bfloat16", "half"])
def test_forward_after_a_cast(cast):
    from mxfp4_quantized_gemm_amd.int8 import Int8Linear
    source = torch.nn.Linear(200, 48, device="cuda")
    layer = Int8Linear.from_weight(source.weight, source.bias)
    x = torch.randn(5, 200, device="cuda")
    want = layer(x)
    model = torch.nn.Sequential(layer)
    getattr(model, cast)()
    with torch.no_grad():
        source.bias += 1
    assert torch.equal(model(x), want)
    y = model(x.to(getattr(torch, cast)))
    assert y.dtype == getattr(torch, cast) and torch.isfinite(y).all()
    back = Int8Linear(200, 48, bias=True).cuda()
    back.load_state_dict(layer.state_dict())
    assert torch.equal(back(x), want)
