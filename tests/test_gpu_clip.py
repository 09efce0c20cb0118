"""The global gradient norm and clipping against 64 bits (tolerances derived in _experts_ref)."""
import math

import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R

pytestmark = pytest.mark.gpu

NORM_TOL = 130 * R.U * 1.01


def _ws():
    return ctr.workspace(ctr.ctr_clip_grads_workspace_size())


def _make(sizes, scale=1.0, seed=0, shift=0):
    """Tensors of alternating types, each starting `shift` elements into its buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + shift, generator=g, device="cuda") * scale
        out.append(t.to(torch.bfloat16 if i % 2 else torch.float32)[shift:])
    return out


def _norm(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def _check(grads, max_norm, outs_in_place=False):
    before = [t.clone() for t in grads]
    outs = grads if outs_in_place else [torch.full_like(t, 5.0) for t in grads]
    ws, norm = _ws(), torch.full((1,), -1.0, device="cuda")
    ctr.ctr_clip_grads(ctr.grad_list(grads, outs), max_norm, norm, ws)
    assert ctr.ctr_check_status(ws) == 0
    ref = _norm(before)
    got = norm.item()
    assert abs(got - ref) <= NORM_TOL * ref
    c = max_norm / ref if got > max_norm else 1.0
    for t, o in zip(before, outs):
        want = t.double() * c
        # the factor carries the norm's error and a division, then one product
        tol = (NORM_TOL + 4 * R.U) * want.abs() + 1e-44
        if c == 1.0:
            assert torch.equal(o, t)
        else:
            assert bool((o.double() >= (want - tol).to(t.dtype)).all() and (o.double() <= (want + tol).to(t.dtype)).all())
    return got


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("sizes", [[1], [0], [5, 0, 1], [8192], [8191, 8193, 16384], [100, 479 * 512, 512, 1, 26],
                                   [3] * 300, [70_000] * 600])
def test_norm_and_clip(sizes, shift):
    for in_place in (False, True):
        grads = _make(sizes, seed=len(sizes), shift=shift)
        ref = _norm(grads)
        _check(grads, 0.25 * ref if ref else 1.0, in_place)
        _check(_make(sizes, seed=len(sizes), shift=shift), 2.0 * ref + 1.0, in_place)


def test_no_tensors_and_norm_alone():
    ws, norm = _ws(), torch.full((1,), -1.0, device="cuda")
    ctr.ctr_clip_grads(ctr.grad_list([], []), 1.0, norm, ws)
    assert norm.item() == 0.0
    grads = _make([1000, 37])
    keep = [t.clone() for t in grads]
    ctr.ctr_clip_grads(ctr.grad_list(grads), 0.5, norm, ws)
    assert abs(norm.item() - _norm(grads)) <= NORM_TOL * _norm(grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))


@pytest.mark.parametrize("size", [3e-38, 1e-30, 1e-22, 1e-18, 1e18, 1e25, 1e34])
def test_norm_where_squares_leave_fp32(size):
    grads = [t.float() * size for t in _make([9000, 513], seed=3)] + _make([77], seed=4)[:1]
    grads[2] *= 0.0
    ws, norm = _ws(), torch.empty(1, device="cuda")
    ctr.ctr_clip_grads(ctr.grad_list(grads), 1.0, norm, ws)
    ref = _norm(grads)
    assert abs(norm.item() - ref) <= NORM_TOL * ref
    # and beside ordinary values
    grads[2] += 1.0
    ctr.ctr_clip_grads(ctr.grad_list(grads), 1.0, norm, ws)
    ref = _norm(grads)
    assert abs(norm.item() - ref) <= NORM_TOL * ref


@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_no_number_leaves_the_gradients(odd):
    for pos in (0, 8191, 19999):
        grads = _make([20000, 11])
        grads[0][pos] = odd
        outs = [torch.full_like(t, 5.0) for t in grads]
        ws, norm = _ws(), torch.empty(1, device="cuda")
        ctr.ctr_clip_grads(ctr.grad_list(grads, outs), 0.1, norm, ws)
        assert math.isnan(norm.item()) if math.isnan(odd) else norm.item() == math.inf
        assert all(torch.equal(a.nan_to_num(1.5), b.nan_to_num(1.5)) for a, b in zip(grads, outs))


def test_zero_bound_and_zero_gradients():
    grads = _make([300, 20])
    outs = [torch.full_like(t, 5.0) for t in grads]
    ws, norm = _ws(), torch.empty(1, device="cuda")
    ctr.ctr_clip_grads(ctr.grad_list(grads, outs), 0.0, norm, ws)
    assert all(bool((t == 0).all()) for t in outs)
    zeros = [torch.zeros(50, device="cuda")]
    ctr.ctr_clip_grads(ctr.grad_list(zeros, zeros), 0.0, norm, ws)
    assert norm.item() == 0.0 and bool((zeros[0] == 0).all())


def test_same_norm_every_time_and_on_another_stream():
    grads = _make([3_000_000, 500_001, 77], seed=9)
    ws, norm = _ws(), torch.empty(1, device="cuda")
    seen = set()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            ctr.ctr_clip_grads(ctr.grad_list(grads), 1.0, norm, ws)
            torch.cuda.synchronize()
        seen.add(norm.item())
    assert len(seen) == 1


def test_refusals():
    ws, norm = _ws(), torch.empty(1, device="cuda")
    g = torch.ones(8, device="cuda")
    for bad in (lambda: ctr.grad_list([g.cpu()]), lambda: ctr.grad_list([g.half()]),
                lambda: ctr.grad_list([torch.ones((4, 4), device="cuda").t()[1:]]),
                lambda: ctr.grad_list([g], [g, g]), lambda: ctr.grad_list([g], [g.bfloat16()]),
                lambda: ctr.ctr_clip_grads(ctr.grad_list([g]), 1.0, norm.double(), ws)):
        with pytest.raises(ValueError):
            bad()
    for max_norm in (-1.0, float("nan")):
        with pytest.raises(ctr.CtrError) as e:
            ctr.ctr_clip_grads(ctr.grad_list([g]), max_norm, norm, ws)
        assert e.value.status == ctr.ERR_INVALID_ARG
    with pytest.raises(ctr.CtrError) as e:
        ctr.ctr_clip_grads(ctr.grad_list([g]), 1.0, norm, ws[:256])
    assert e.value.status == ctr.ERR_WORKSPACE
