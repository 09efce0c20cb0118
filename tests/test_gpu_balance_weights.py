"""Balanced routing's weights where a token's choices lie far apart: in proportion to their sigmoids, down to fp32's smallest
numbers."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R
import _layers_ref as L
from test_gpu_balance import _bias, _on, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [60.0, 3.0, 0.0, -3.0, -8.0, -14.0, -19.9, -20.1, -40.0, -300.0])
def test_weights_far_below_the_largest(top, dtype):
    # the largest choice at `top`, the others from 0 to 86 below: the smallest weights are e^-86 and still fp32 numbers, whatever
    # the sigmoids themselves are
    rng = np.random.default_rng(int(10 * abs(top)))
    T, E, k = 200, 24, 8
    s = top - 85.0 * rng.random((T, E))
    s[np.arange(T), rng.integers(0, E, size=T)] = top
    s = torch.from_numpy(s).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype]).double().numpy()
    for bias, groups, group_k in ((None, 1, 1), (_bias(E, 3, 3.0), 1, 1), (None, 4, 4), (_bias(E, 4), 4, 3)):
        for renorm in (True, False):
            expert, p = check(s, k, "sigmoid", bias, groups, group_k, renorm, dtype, factor=1.5)
            dw = rng.normal(size=(T, k)).astype(np.float32)
            d = torch.empty((T, E), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
            ctr.ctr_expert_route_balanced_bwd(torch.from_numpy(dw).cuda(), _on(s, dtype), ctr.SCORE_SIGMOID, renorm, 1.5,
                                              torch.from_numpy(expert).cuda(), d, ctr.workspace(256))
            ref, mag = L.balanced_grad(dw.astype(np.float64), s, "sigmoid", renorm, 1.5, expert, p)
            assert R.within(d.double().cpu().numpy(), ref, (2 * E + 113) * L.U * mag + 1e-37, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [1, 4])
def test_the_gradient_of_a_single_choice_is_zero(k, score, dtype):
    # renormalised, its weight is 1 whatever its score: no rounding may be left over
    rng = np.random.default_rng(k)
    T, E = 300, 40
    s = 4 * rng.normal(size=(T, E)) - 2
    if k > 1:
        live = rng.integers(0, E, size=T)
        s[np.arange(E)[None] != live[:, None]] = -np.inf
    s = torch.from_numpy(s).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype]).double().numpy()
    expert, _ = check(s, k, score, _bias(E, 2), 1, 1, True, dtype, factor=2.5)
    dw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()
    d = torch.full((T, E), 7.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    ctr.ctr_expert_route_balanced_bwd(dw, _on(s, dtype), ctr.SCORES[score], True, 2.5, torch.from_numpy(expert).cuda(), d,
                                      ctr.workspace(256))
    assert bool((d == 0).all())
