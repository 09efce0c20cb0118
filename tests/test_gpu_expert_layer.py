"""The expert layer as a user runs it: every stage against 64 bits on the stage's own inputs, serving against
training, a captured graph, and a few steps of training behind the CTR path."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr
from sparse_embeddings_feature_gb300.experts import ExpertLayer, train_demo

import _experts_ref as R

pytestmark = pytest.mark.gpu


def _np(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _case(T, K, N, E, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), generator=g, device="cuda").to(dtype)
    s = torch.randn((T, E), generator=g, device="cuda")
    s[torch.rand((T, E), generator=g, device="cuda") < 0.2] = -float("inf")
    s[::7] = -float("inf")
    w = (torch.randn((E, N, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    dy = torch.randn((T, N), generator=g, device="cuda").to(dtype)
    return x, s, w, dy


def _blocks(w):
    q, s = R.quantize(w, 128, 128)
    return q * R.spread(s, 128, 128, *w.shape)


def _rows(x):
    q, s = R.quantize(x, 1, 128)
    return q * R.spread(s, 1, 128, *x.shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,N,E,k,renorm", [(1, 479, 64, 4, 2, True), (300, 479, 130, 8, 2, False),
                                               (2000, 256, 256, 16, 3, True)])
def test_forward_and_backward_stage_by_stage(T, K, N, E, k, renorm, dtype):
    name = "f32" if dtype == torch.float32 else "bf16"
    x, s, w, dy = _case(T, K, N, E, dtype, seed=T)
    layer = ExpertLayer(T, K, N, E, k, dtype=dtype, renormalize=renorm, train=True)
    layer.set_weights(w)
    y = layer.forward(x, s)
    expert, weight, slot, token, offsets, _ = R.route(_np(s), k, renorm)
    np.testing.assert_array_equal(_np(layer.slot), slot)
    np.testing.assert_array_equal(_np(layer.offsets), offsets)
    wt = _np(layer.weight)
    wv = [_blocks(_np(w[e])) for e in range(E)]
    used = offsets[-1]
    xr = _rows(_np(x)[token[:used]]) if used else np.zeros((0, K))
    ys = _np(layer.ys)
    assert np.all(ys[used:] == 0)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        ref, mag = xr[r] @ wv[e].T, np.abs(xr[r]) @ np.abs(wv[e]).T
        assert R.within(ys[r], ref, 1.01 * R.product_bound(mag, ctr.fp8_blocks(K)), name)
    live = (slot >= 0)[:, :, None]
    terms = np.where(live, ys[slot], 0.0) * wt[:, :, None]
    assert R.within(_np(y), terms.sum(1), 1.01 * k * R.U * np.abs(terms).sum(1), name)

    dx, dscores, dw = layer.backward(dy)
    assert all(v == 0 for v in layer.check_status().values())
    dyv, dys = _np(dy), _np(layer.dys)
    dq = _rows(dys[:used]) if used else np.zeros((0, N))
    dxs = _np(layer.dxs)
    dwv = _np(dw)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        ref, mag = dq[r] @ wv[e], np.abs(dq[r]) @ np.abs(wv[e])
        assert R.within(dxs[r], ref, 1.01 * R.product_bound(mag, ctr.fp8_blocks(N)), name)
        n = offsets[e + 1] - offsets[e]
        if n == 0:
            assert np.all(dwv[e] == 0)
            continue
        q, sc = R.quantize(dys[r], 128, 1)
        d_val, x_val = q * R.spread(sc, 128, 1, n, N), _blocks(_np(x)[token[r]])
        ref, mag = d_val.T @ x_val, np.abs(d_val).T @ np.abs(x_val)
        assert R.within(dwv[e], ref, 1.01 * R.product_bound(mag, -(-n // 128)), "f32")
    terms = np.where(live, dxs[slot], 0.0)
    assert R.within(_np(dx), terms.sum(1), 1.01 * k * R.U * np.abs(terms).sum(1), name)
    dots = np.where(live, ys[slot], 0.0) * dyv[:, None]
    assert np.all(np.abs(_np(layer.dweight) - dots.sum(2)) <= 1.01 * N * R.U * np.abs(dots).sum(2))
    ref, mag = R.route_grad(_np(layer.dweight), _np(s), k, renorm)
    assert R.within(_np(dscores), ref, (2 * E + 24) * R.U * mag + 1e-38, "f32")


def test_serving_gives_the_training_forward_and_replays_as_a_graph():
    x, s, w, _ = _case(64, 479, 200, 8, torch.float32)
    train = ExpertLayer(64, 479, 200, 8, 2, train=True)
    serve = ExpertLayer(64, 479, 200, 8, 2)
    train.set_weights(w)
    serve.set_weights(w)
    ref = train.forward(x, s).clone()
    assert torch.equal(serve.forward(x, s), ref)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        serve.forward(x, s)
    x2, s2 = _case(64, 479, 200, 8, torch.float32, seed=9)[:2]
    x.copy_(x2)
    s.copy_(s2)
    g.replay()
    assert torch.equal(serve.y, train.forward(x2, s2))
    rows = torch.empty((128, 479), device="cuda")
    serve.sorted_rows(x, rows)
    tok = serve.token.long()
    assert torch.equal(rows, torch.where((tok >= 0)[:, None], x[tok.clamp(min=0)], 0.0))


def test_clip_covers_the_layer_and_others():
    x, s, w, dy = _case(200, 96, 64, 4, torch.float32)
    layer = ExpertLayer(200, 96, 64, 4, 2, train=True)
    layer.set_weights(w)
    layer.forward(x, s)
    _, _, dw = layer.backward(dy)
    other = torch.randn(1000, device="cuda")
    total = float(dw.double().square().sum() + other.double().square().sum()) ** 0.5
    norm = layer.clip(0.5, [other])
    assert abs(norm.item() - total) <= 1e-5 * total
    after = float(dw.double().square().sum() + other.double().square().sum()) ** 0.5
    assert abs(after - 0.5) <= 1e-5


def test_training_behind_the_ctr_path_learns():
    losses = train_demo(steps=40, batch=1024)
    assert losses[0] > 0.5 and np.isfinite(losses).all()
    assert np.mean(losses[-5:]) < 0.6 * losses[0]


def test_refusals():
    with pytest.raises(ValueError):
        ExpertLayer(8, 16, 16, 4, 5)
    with pytest.raises(ValueError):
        ExpertLayer(8, 16, 16, 4, 2, dtype=torch.float16)
    with pytest.raises(ValueError):
        ExpertLayer(0, 16, 16, 4, 2)
    layer = ExpertLayer(8, 16, 16, 4, 2)
    with pytest.raises(ValueError):
        layer.set_weights(torch.zeros((4, 16, 8), device="cuda"))
    with pytest.raises(RuntimeError):
        layer.backward(torch.zeros((8, 16), device="cuda"))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros((7, 16), device="cuda"), torch.zeros((8, 3), device="cuda"))
