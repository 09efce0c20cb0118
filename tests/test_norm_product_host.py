"""The serving layer of norm and 8-bit product has nothing to multiply by before its weights are set (CPU only)."""
import pytest
import torch

from sparse_embeddings_feature_gb300.layers import NormProduct


def test_a_forward_needs_weights():
    layer = NormProduct(4, 64, 32, device="cpu")
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="set_weights"):
        layer.forward(x, None, None)
    with pytest.raises(ValueError):
        layer.set_weights(torch.zeros((32, 65)))
    with pytest.raises(RuntimeError, match="set_weights"):
        layer.forward(x, None, None)
