"""bf16 layers whose sums are longer than a tensor core's accumulator is accurate for: terms of one sign, against 64 bits."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _layers_ref as L

pytestmark = pytest.mark.gpu

U = L.U


# a sum is read back every 512 terms, 2 * 512 u of its magnitude at most, and added up in registers, k / 512 u
def _long_tol(k, mag):
    return (2 * 512 + k / 512 + 2) * U * mag


@pytest.mark.parametrize("rows,n,k", [(20, 24, 1 << 20), (300, 260, 70000), (20, 24, 65600)])
def test_long_sums_of_positive_terms(rows, n, k):
    # all of one sign: additions that drop bits would show
    g = torch.Generator(device="cuda").manual_seed(k)
    x = (torch.rand((rows, k), generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    w = (torch.rand((n, k), generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    bias = torch.randn((n,), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((rows, n), generator=g, device="cuda").to(torch.bfloat16)
    y, pre = (torch.empty((rows, n), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, k, torch.bfloat16, True))
    z = x.double() @ w.double().t()
    tol = _long_tol(k, z)
    ctr.ctr_dense(x, w, None, ctr.ACT_NONE, None, y, None, ws)
    assert L.fits(y, z, tol, "bf16")
    ctr.ctr_dense(x, w, bias, ctr.ACT_SILU, r, y, pre, ws)
    zb = z + bias.double()
    assert L.fits(pre, zb, tol + U * zb.abs(), "bf16")
    assert L.fits(y, zb * torch.sigmoid(zb) + r.double(), tol * 1.1 + 40 * U * zb.abs(), "bf16")
    # the input gradient's sum runs over the layer's columns: dy [rows, k] and W [k, n]
    dx = torch.empty((rows, n), device="cuda", dtype=torch.bfloat16)
    wt = w.t().contiguous()
    xin = torch.zeros((rows, n), device="cuda", dtype=torch.bfloat16)
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, k, n, torch.bfloat16, True))
    ctr.ctr_dense_bwd(x, xin, wt, None, ctr.ACT_NONE, dx, None, None, ws)
    assert L.fits(dx, z, tol, "bf16")
    assert ctr.ctr_check_status(ws) == 0


def test_long_sums_of_rows_off_16_bytes():
    rows, n, k = 130, 33, 66001
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = ((torch.rand((m, k), generator=g, device="cuda") + 0.5).to(torch.bfloat16) for m in (rows, n))
    y = torch.empty((rows, n), device="cuda", dtype=torch.bfloat16)
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, k, torch.bfloat16))
    ctr.ctr_dense(x, w, None, ctr.ACT_RELU, None, y, None, ws)
    z = x.double() @ w.double().t()
    assert L.fits(y, z, _long_tol(k, z), "bf16")
