"""The layers around the experts as they are used together: against autograd in 64 bits, captured, and in training."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr
from sparse_embeddings_feature_gb300.experts import ExpertLayer
from sparse_embeddings_feature_gb300.layers import NormProduct, ResidualBlock, train_demo

import _experts_ref as R
import _layers_ref as L

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _g(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _params(width, hidden, dtype, g):
    def d(*shape, scale=1.0, dt=dtype):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)
    return {"w1": d(hidden, width, scale=width ** -0.5), "b1": d(hidden, scale=0.3), "w2": d(width, hidden, scale=hidden ** -0.5),
            "b2": d(width, scale=0.3), "gamma": 1 + d(width, scale=0.2, dt=torch.float32)}


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width,hidden,act", [(1, 24, 40, "silu"), (7, 128, 96, "gelu"), (300, 479, 256, "gelu"),
                                                  (1000, 264, 1032, "sigmoid")])
def test_block_against_autograd(rows, width, hidden, act, dtype):
    g = _g(rows)
    p = _params(width, hidden, DT[dtype], g)
    x = torch.randn((rows, width), generator=g, device="cuda").to(DT[dtype])
    dy = torch.randn((rows, width), generator=g, device="cuda").to(DT[dtype])
    block = ResidualBlock(rows, width, hidden, dtype=DT[dtype], act=act, train=True)
    y = block.forward(x, p).clone()
    dx, grads = block.backward(dy)
    q = {n: t.double().requires_grad_() for n, t in p.items()}
    xd = x.double().requires_grad_()
    v = xd / torch.sqrt((xd * xd).mean(1, keepdim=True) + float(np.float32(1e-6))) * q["gamma"]
    ref = L.act64(act, v @ q["w1"].t() + q["b1"])[0] @ q["w2"].t() + q["b2"] + xd
    ref.backward(dy.double())
    # 2-norms.  fp32: four sums of at most 16 u behind one another, and the rest: 100 u.  bf16: a rounding is off by at
    # most 2^-8 of the value; the result went through v, h and itself, a gradient also through pre, dz, dh or dv
    most = {"f32": 100 * L.U, "bf16": 6 * 2.0 ** -8}[dtype]
    assert _rel(y, ref.detach()) <= most
    assert _rel(dx, xd.grad) <= most
    for n in p:
        assert _rel(grads[n], q[n].grad) <= most, n
    assert not any(block.check_status().values())


def test_block_that_has_no_forward_refuses():
    block = ResidualBlock(8, 16, 16, train=True)
    with pytest.raises(RuntimeError):
        block.backward(torch.zeros((8, 16), device="cuda"))
    p = _params(16, 16, torch.float32, _g(1))
    block.forward(torch.zeros((8, 16), device="cuda"), p)
    with pytest.raises(ValueError):
        block.forward(torch.zeros((8, 17), device="cuda"), p)
    with pytest.raises(RuntimeError):   # a forward that was refused leaves none
        block.backward(torch.zeros((8, 16), device="cuda"))
    for bad in (dict(act="tanh"), dict(dtype=torch.float16), dict(width=0)):
        with pytest.raises(ValueError):
            ResidualBlock(**{**dict(rows=8, width=16, hidden=16), **bad})


def test_block_captured_beside_an_eager_one():
    p = _params(256, 512, torch.bfloat16, _g(2))
    x, dy = (torch.randn((500, 256), generator=_g(i), device="cuda").to(torch.bfloat16) for i in (3, 4))
    eager, block = (ResidualBlock(500, 256, 512, dtype=torch.bfloat16, train=True) for _ in range(2))
    y = eager.forward(x, p)
    dx, grads = eager.backward(dy)
    block.forward(x, p)
    block.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, p)
        block.backward(dy)
    for t in (block.y, block.dx, *block.grads.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(block.y, y) and torch.equal(block.dx, dx)
    assert all(torch.equal(block.grads[n], grads[n]) for n in grads)


@pytest.mark.parametrize("rows,width,out", [(1, 128, 64), (9, 200, 130), (300, 479, 256), (700, 1024, 512)])
def test_norm_codes_are_the_products_operand(rows, width, out):
    g = _g(rows)
    dt = torch.bfloat16
    x, r = (torch.randn((rows, width), generator=g, device="cuda").to(dt) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn((width,), generator=g, device="cuda")
    w = (torch.randn((out, width), generator=g, device="cuda") * width ** -0.5).to(dt)
    layer = NormProduct(rows, width, out)
    layer.set_weights(w)
    s, y = layer.forward(x, r, gamma)
    assert layer.check_status() == 0
    sd = (x.float() + r.float()).to(dt).double()
    assert torch.equal(s.double(), sd)
    # what codes and scales stand for, multiplied in 64 bits
    kb = ctr.fp8_blocks(width)
    a = torch.from_numpy(R.e4m3_values(layer.q.cpu().numpy())).cuda() * layer.scale.t().double().repeat_interleave(128, 1)
    b = torch.from_numpy(R.e4m3_values(layer.wq[0].cpu().numpy())).cuda() * \
        layer.ws[0].double().repeat_interleave(128, 0)[:out].repeat_interleave(128, 1)
    assert L.fits(y, a @ b.t(), R.product_bound(a.abs() @ b.abs().t(), kb), "bf16")
    # and what they stand for is the norm: each of its codes, within half a step of 2^-3 to 2^-4 of the value or of 2^-10
    # of the block's largest
    v = sd / torch.sqrt((sd * sd).mean(1, keepdim=True) + float(np.float32(1e-6))) * gamma.double()
    top = layer.scale.t().double().repeat_interleave(128, 1)[:, :width] * 448
    assert bool(((a[:, :width] - v).abs() <= 2.0 ** -4 * v.abs() + top * 2.0 ** -18 + 1e-12).all())


@pytest.mark.parametrize("score,groups,group_k,with_bias", [("sigmoid", 4, 2, True), ("softmax", 1, None, True),
                                                           ("sigmoid", 1, None, False)])
def test_expert_layer_with_balance(score, groups, group_k, with_bias):
    T, width, out, E, k = 257, 96, 64, 16, 3
    g = _g(5)
    x = torch.randn((T, width), generator=g, device="cuda")
    scores = torch.randn((T, E), generator=g, device="cuda")
    w = torch.randn((E, out, width), generator=g, device="cuda") * width ** -0.5
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda") if with_bias else None
    dy = torch.randn((T, out), generator=g, device="cuda")
    layer = ExpertLayer(T, width, out, E, k, train=True, score=score, groups=groups, group_k=group_k, factor=1.5)
    layer.set_weights(w)
    y = layer.forward(x, scores, bias).clone()
    gk = groups if group_k is None else group_k
    ref = L.balanced(scores.double().cpu().numpy(), k, score, None if bias is None else bias.cpu().numpy(), groups, gk, True, 1.5)
    np.testing.assert_array_equal(layer.expert.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(layer.loads().cpu().numpy(), np.bincount(ref[0].ravel(), minlength=E))
    # the same rows through the plain layer's calls
    again = torch.empty_like(y)
    ctr.ctr_expert_combine(layer.ys, layer.slot, torch.from_numpy(ref[1].astype(np.float32)).cuda(), again, layer.ws_rows)
    assert _rel(y, again.double()) <= 200 * L.U
    dx, dscores, dw = layer.backward(dy)
    dref, mag = L.balanced_grad(layer.dweight.double().cpu().numpy(), scores.double().cpu().numpy(), score, True, 1.5, ref[0], ref[5])
    assert R.within(dscores.double().cpu().numpy(), dref, (2 * E + 40) * L.U * mag + 1e-37, "f32")
    assert not any(layer.check_status().values())
    plain = ExpertLayer(T, width, out, E, k, train=True)
    assert not plain.balanced
    for bad in (dict(score="tanh"), dict(groups=3), dict(groups=4, group_k=5), dict(groups=16, group_k=2)):
        with pytest.raises(ValueError):
            ExpertLayer(T, width, out, E, k, **bad)


def test_training_runs():
    losses, skew = train_demo(steps=4, batch=256)
    assert len(losses) == len(skew) == 4 and all(np.isfinite(losses)) and all(s >= 1 for s in skew)
