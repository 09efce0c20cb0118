"""Gradients that are exactly zero (an expert without rows has them) cost no more than others, and numbers whose
squares are too small for fp32 still count."""
import math

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu


def _us(grads):
    ws, norm = ctr.workspace(ctr.ctr_clip_grads_workspace_size()), torch.empty(1, device="cuda")
    lst = ctr.grad_list(grads)
    best = math.inf
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ctr.ctr_clip_grads(lst, 1.0, norm, ws)
        b.record()
        b.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best, norm.item()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_are_as_fast(dtype, shift):
    # the same bytes, 256 MB; the kernels' time does not depend on the values, so 1.5 leaves room for noise alone
    n = (256 << 20) // (4 if dtype == torch.float32 else 2)
    t = torch.randn(n + 1, device="cuda").to(dtype)[shift:n]
    dense, _ = _us([t])
    t.zero_()
    zeros, norm = _us([t])
    assert norm == 0.0
    assert zeros <= 1.5 * dense, (zeros, dense)
    t.fill_(-0.0)
    minus, norm = _us([t])
    assert norm == 0.0 and minus <= 1.5 * dense, (minus, dense)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [1e-45, 1e-39, 1e-30, 1e-23, -1e-30])
def test_one_small_number_among_zeros_counts(value, dtype, shift):
    for n in (1, 9, 8192, 20001):
        for at in {0, n // 2, n - 1}:
            t = torch.zeros(n + 1, dtype=dtype, device="cuda")[shift:n + shift]
            t[at] = value
            want = abs(float(t[at].double()))
            assert _norm([t]) == want              # one number's root of its square, rounded to fp32: the number


def _norm(grads):
    ws, norm = ctr.workspace(ctr.ctr_clip_grads_workspace_size()), torch.empty(1, device="cuda")
    ctr.ctr_clip_grads(ctr.grad_list(grads), 1.0, norm, ws)
    return float(norm.double().item())
