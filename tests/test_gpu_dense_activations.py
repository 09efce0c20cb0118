"""Activations and their derivatives, accurate relative to their own size.

u = 2^-24.  fp32: e^-|z| is within 5 u (the exponential 2^-22, its correction one rounding), 1 + it within 4 u, its
reciprocal 2 u more; sigmoid (a product, one rounding) within 12 u, sigmoid' = e r^2 within 18 u; silu one rounding
more, silu' the same of its two terms' magnitudes.  gelu: the tail of the normal distribution is bell P, P within 8 u (a
polynomial of degree 8 within 1 u, its evaluation 5 u, its argument's reciprocal 2 u) and bell within 6 u: 16 u with the
products; gelu' the same of its two terms' magnitudes.

bf16 layers: what rounding to bf16 covers, 2^-9 of the derivative, is far above the exponential's (|z| + 8) 2^-24; gelu's erf is
within 1.5e-7 of itself, so its derivative below 1e-4 by that much.  An exponential below 2^-126 is zero: 1e-37 (1 + |z|)."""
import math

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _layers_ref as L

pytestmark = pytest.mark.gpu

U = L.U
ABS = 1e-37
ACTS = ["sigmoid", "silu", "gelu"]


def _points(n, seed=0):
    """z from -100 to 100, and dense around zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.cat([torch.linspace(-100, 100, n // 2, device="cuda"), torch.randn(n - n // 2, generator=g, device="cuda") * 3])
    z[:8] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 17.0, -17.0, 88.5, -88.5], device="cuda")
    return z


def _terms(act, z):
    """(value, the magnitude that its error goes by, derivative, its magnitude) in 64 bits, without cancellation in the tails."""
    e = torch.exp(-z.abs())
    big, small = 1 / (1 + e), e / (1 + e)
    s, t = torch.where(z >= 0, big, small), torch.where(z >= 0, small, big)   # t = 1 - s
    if act == "sigmoid":
        return s, s, big * small, big * small
    if act == "silu":
        return z * s, z.abs() * s, s * (1 + z * t), s * (1 + z.abs() * t)
    below = 0.5 * torch.special.erfcx(z.abs() / math.sqrt(2)) * torch.exp(-z * z / 2)
    phi = torch.where(z < 0, below, 1 - below)
    bell = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z * phi, z.abs() * phi, phi + bell, phi + bell.abs()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 7, 40])
def test_fp32_activations(rows, act):
    # z = x * 1 with one column of x and w; 1 and 7 rows take the kernel for few rows, 40 the tensor cores
    n = 4096
    x = torch.ones((rows, 1), device="cuda")
    z = _points(n)
    y, pre = torch.empty((rows, n), device="cuda"), torch.empty((rows, n), device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, 1, torch.float32))
    ctr.ctr_dense(x, z[:, None].contiguous(), None, ctr.ACTIVATIONS[act], None, y, pre, ws)
    value, mag, _, _ = _terms(act, pre.double())
    assert bool(((y.double() - value).abs() <= 16 * U * mag + ABS * (1 + pre.double().abs())).all())
    assert ctr.ctr_check_status(ws) == 0


@pytest.mark.parametrize("act", ACTS)
def test_fp32_derivatives(act):
    # one row: the bias's gradient is dz itself
    n = 8192
    z, dy = _points(n)[None], torch.ones((1, n), device="cuda")
    x, w = torch.ones((1, 1), device="cuda"), torch.ones((n, 1), device="cuda")
    db = torch.empty((n,), device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(1, n, 1, torch.float32, True))
    ctr.ctr_dense_bwd(dy, x, w, z, ctr.ACTIVATIONS[act], None, None, db, ws)
    zz = z[0].double()
    _, _, d, mag = _terms(act, zz)
    assert bool(((db.double() - d).abs() <= 20 * U * mag + ABS * (1 + zz.abs())).all())


@pytest.mark.parametrize("act", ACTS)
def test_bf16_derivatives(act):
    n = 8192
    z = _points(n)[None].to(torch.bfloat16)
    dy, x, w = (torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in ((1, n), (1, 1), (n, 1)))
    db = torch.empty((n,), device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(1, n, 1, torch.bfloat16, True))
    ctr.ctr_dense_bwd(dy, x, w, z, ctr.ACTIVATIONS[act], None, None, db, ws)
    zz = z[0].double()
    _, _, d, mag = _terms(act, zz)
    tol = 2.0 ** -9 * (mag + (1e-4 if act == "gelu" else 0)) + ABS * (1 + zz.abs())
    assert bool(((db.double() - d).abs() <= tol).all())


def test_what_is_no_number_stays_so():
    inf, nan = math.inf, math.nan
    z = torch.tensor([nan, inf, -inf], device="cuda")
    for act, want in (("sigmoid", [nan, 1.0, 0.0]), ("silu", [nan, inf, nan]), ("gelu", [nan, inf, nan]), ("relu", [nan, inf, 0.0])):
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.empty((1, 3), device="cuda", dtype=dtype)
            ctr.ctr_dense(torch.ones((1, 1), device="cuda", dtype=dtype), torch.ones((3, 1), device="cuda", dtype=dtype),
                          z.to(dtype), ctr.ACTIVATIONS[act], None, y, None, ctr.workspace(4096))
            assert torch.equal(y[0].float().nan_to_num(nan=77.0), torch.tensor(want, device="cuda").nan_to_num(nan=77.0)), act
