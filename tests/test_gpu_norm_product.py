"""The serving layer of norm and 8-bit product: what it refuses."""
import pytest
import torch

from sparse_embeddings_feature_gb300.layers import NormProduct

pytestmark = pytest.mark.gpu


def test_a_forward_needs_weights():
    layer = NormProduct(4, 64, 32)
    x = torch.randn((4, 64), device="cuda").to(torch.bfloat16)
    with pytest.raises(RuntimeError):
        layer.forward(x, None, None)
    with pytest.raises(ValueError):
        layer.set_weights(torch.zeros((32, 65), device="cuda"))
    with pytest.raises(RuntimeError):
        layer.forward(x, None, None)
    layer.set_weights(torch.randn((32, 64), device="cuda"))
    s, y = layer.forward(x, None, None)
    assert torch.equal(s, x) and bool(torch.isfinite(y.float()).all()) and layer.check_status() == 0
    with pytest.raises(ValueError):   # weights that are refused leave none
        layer.set_weights(torch.zeros((32, 64), device="cuda", dtype=torch.float16))
    with pytest.raises(RuntimeError):
        layer.forward(x, None, None)
