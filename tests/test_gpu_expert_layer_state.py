"""What ExpertLayer keeps between its calls, and what it refuses."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr
from sparse_embeddings_feature_gb300.experts import ExpertLayer

pytestmark = pytest.mark.gpu

T, K, N, E, TOP = 300, 479, 96, 8, 2


def _case(seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, s, dy = (torch.randn(shape, generator=g, device="cuda").to(dtype) for shape in ((T, K), (T, E), (T, N)))
    return x, s, torch.randn((E, N, K), generator=g, device="cuda") / K ** 0.5, dy


def _layer(w, **kw):
    layer = ExpertLayer(T, K, N, E, TOP, **kw)
    layer.set_weights(w)
    return layer


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_may_change_after_forward(dtype, renorm):
    x, s, w, dy = _case()
    s = s.to(dtype)
    layer = _layer(w, train=True, renormalize=renorm)
    layer.forward(x, s)
    ref = [t.clone() for t in layer.backward(dy)]
    layer.forward(x, s)
    s.copy_(torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda"))
    for a, b in zip(ref, layer.backward(dy)):
        assert torch.equal(a, b)


def test_strided_scores_of_either_type_in_turn():
    x, s, w, dy = _case()
    layer, fresh = _layer(w, train=True), _layer(w, train=True)
    wide = torch.zeros((T, E + 5), device="cuda")
    for scores in (s, s.bfloat16(), wide[:, :E].copy_(s), s):
        layer.forward(x, scores)
        fresh.forward(x, scores.contiguous())
        a, b = layer.backward(dy)[1], fresh.backward(dy)[1]
        assert a.dtype == scores.dtype and torch.equal(a, b)


def test_new_weights_end_the_forward():
    x, s, w, dy = _case()
    layer = _layer(w, train=True)
    layer.forward(x, s)
    layer.set_weights(w * 2)
    with pytest.raises(RuntimeError):
        layer.backward(dy)
    layer.forward(x, s)
    layer.backward(dy)


def test_a_refused_forward_leaves_none():
    x, s, w, dy = _case()
    layer = _layer(w, train=True)
    layer.forward(x, s)
    with pytest.raises(ValueError):
        layer.forward(x.double(), s.flip(1))
    with pytest.raises(RuntimeError):
        layer.backward(dy)


@pytest.mark.parametrize("train", [False, True])
def test_forward_takes_its_own_sizes_only(train):
    x, s, w, _ = _case()
    layer = _layer(w, train=train)
    more = torch.zeros((T + 1, K), device="cuda")
    for bad in (x[:, :400], x[:, :K - 1], x[:-1], more, x[0], None):
        with pytest.raises(ValueError):
            layer.forward(bad, s)
    for bad in (s[:-1], s[:, :-1], torch.zeros((T, E + 1), device="cuda")):
        with pytest.raises(ValueError):
            layer.forward(x, bad)
    layer.forward(x, s)
    assert all(v == 0 for v in layer.check_status().values())


def test_clip_needs_gradients():
    with pytest.raises(RuntimeError):
        _layer(_case()[2]).clip(1.0)


def test_clip_with_a_list_built_once(monkeypatch):
    x, s, w, dy = _case()
    layer, other = _layer(w, train=True), torch.randn(1000, device="cuda")
    layer.forward(x, s)
    layer.backward(dy)
    dw = layer.dw.clone()
    ref = float((dw.double().square().sum() + other.double().square().sum()).sqrt())
    kept = layer.grads([other])
    monkeypatch.setattr(ctr, "grad_list", None)     # nothing is put together in the call
    assert abs(layer.clip(2 * ref, kept).item() - ref) <= 1e-5 * ref
    assert torch.equal(layer.dw, dw)
    assert abs(layer.clip(0.5 * ref, kept).item() - ref) <= 1e-5 * ref
    assert torch.allclose(layer.dw, dw * 0.5, rtol=1e-5, atol=0)
