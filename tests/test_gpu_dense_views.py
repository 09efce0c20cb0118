"""Dense layers of matrices that are views: rows that end inside 16 bytes with anything behind them, rows megabytes apart,
a workspace of a larger batch."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _layers_ref as L

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _view(g, rows, cols, ld, dtype=BF16, behind=float("nan"), scale=1.0):
    buf = torch.full((rows, ld), behind, dtype=dtype, device="cuda")
    view = buf[:, :cols]
    view.copy_(torch.randn((rows, cols), generator=g, device="cuda") * scale)
    return buf, view


def _check(x, w, bias, dy, y, pre, dx, dw, db, ws, dtype, act="silu"):
    """Both calls on what is given, against 64 bits."""
    ctr.ctr_dense(x, w, bias, ctr.ACTIVATIONS[act], None, y, pre, ws)
    ctr.ctr_dense_bwd(dy, x, w, pre, ctr.ACTIVATIONS[act], dx, dw, db, ws)
    name = "bf16" if dtype == BF16 else "f32"
    rows, n, k = x.shape[0], w.shape[0], x.shape[1]
    x64, w64, dy64 = x.double(), w.double(), dy.double()
    z, mag = x64 @ w64.t() + bias.double(), x64.abs() @ w64.abs().t() + bias.double().abs()
    tol = L.sum_bound(name, k, mag) + 1e-40
    ref = L.act64(act, z)[0]
    assert L.fits(pre, z, tol, name)
    assert L.fits(y, ref, L.act_tol(z, ref, tol), name)
    dz, off, raw, err = L.dz64(name, act, dy64, pre.double())
    assert L.fits(dx, dz @ w64, L.sum_bound(name, n, dz.abs() @ w64.abs()) + off @ w64.abs() + 1e-40, name)
    mag = dz.abs().t() @ x64.abs()
    assert L.fits(dw, dz.t() @ x64, L.sum_bound(name, rows, mag, True) + off.t() @ x64.abs() + 1e-40, "f32")
    assert bool(((db.double() - raw.sum(0)).abs() <= (max(rows, 32) / 4 + 100) * L.U * raw.abs().sum(0) + err.sum(0)).all())
    assert ctr.ctr_check_status(ws) == 0


# widths that end 1 to 15 elements before a multiple of 16; both operands of every product are read as they lie
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,n,k", [(1, 135, 479), (2, 479, 129), (9, 65, 73), (70, 135, 479), (300, 479, 135),
                                      (2000, 263, 257), (5000, 129, 1025), (20000, 250, 331), (1, 1, 77), (40, 1, 77)])
def test_nothing_behind_a_row_enters(rows, n, k, act):
    g = torch.Generator(device="cuda").manual_seed(rows + n)

    def up(c):
        return -(-c // 8) * 8
    xb, x = _view(g, rows, k, up(k))
    wb, w = _view(g, n, k, up(k), scale=k ** -0.5)
    dyb, dy = _view(g, rows, n, up(n))
    bias = torch.randn(n, generator=g, device="cuda").to(BF16)
    yb, y = _view(g, rows, n, up(n), behind=3.0)
    pb, pre = _view(g, rows, n, up(n), behind=float("nan"))
    dxb, dx = _view(g, rows, k, up(k), behind=3.0)
    dw, db = torch.empty((n, k), device="cuda"), torch.empty(n, device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, k, BF16, True, packed=False))
    _check(x, w, bias, dy, y, pre, dx, dw, db, ws, BF16, act)
    assert bool((yb[:, n:] == 3.0).all()) and bool((dxb[:, k:] == 3.0).all()) and bool(pb[:, n:].isnan().all())
    # the residual's rows too
    rb, r = _view(g, rows, n, up(n))
    ctr.ctr_dense(x, w, bias, ctr.ACTIVATIONS[act], r, y, None, ws)
    assert bool(torch.isfinite(y).all()) and bool((yb[:, n:] == 3.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_apart(dtype):
    # offsets past 2^31 elements in every matrix; what lies between the rows is one allocation that nobody reads
    rows, n, k = 130, 40, 72
    far = (1 << 31) // 100 // 8 * 8
    big = torch.empty((rows - 1) * far + 8 * 128, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    at = iter(range(0, 8 * 128, 128))

    def view(r, cols, scale=1.0):
        v = torch.as_strided(big, (r, cols), (far, 1), next(at))
        v.copy_(torch.randn((r, cols), generator=g, device="cuda") * scale)
        return v
    x, w, dy, y, pre, dx = (view(rows, k), view(n, k, k ** -0.5), view(rows, n), view(rows, n), view(rows, n), view(rows, k))
    assert (rows - 1) * x.stride(0) > 1 << 31
    bias = torch.randn(n, generator=g, device="cuda").to(dtype)
    dw, db = torch.empty((n, k), device="cuda"), torch.empty(n, device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, k, dtype, True))
    _check(x, w, bias, dy, y, pre, dx, dw, db, ws, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,k", [(1, 24), (128, 128), (264, 512), (1024, 520)])
def test_a_workspace_has_room_for_fewer_rows(n, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(n)
    most = 30000
    size = ctr.ctr_dense_workspace_size(most, n, k, dtype, True)
    x = torch.randn((most, k), generator=g, device="cuda").to(dtype)
    w = (torch.randn((n, k), generator=g, device="cuda") * k ** -0.5).to(dtype)
    dy, pre = (torch.randn((most, n), generator=g, device="cuda").to(dtype) for _ in range(2))
    dx, dw, db = torch.empty_like(x), torch.empty((n, k), device="cuda"), torch.empty(n, device="cuda")
    full = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    full[:256].zero_()
    last = 0
    for rows in (0, 1, 8, 9, 511, 513, 1100, 4095, 4097, 10001, 29184, 29185, 29999, most):
        need = ctr.ctr_dense_workspace_size(rows, n, k, dtype, True)
        assert need >= last
        last = need
        ctr.ctr_dense_bwd(dy[:rows], x[:rows], w, pre[:rows], ctr.ACT_SILU, dx[:rows], dw, db, full[:size])
        dz, off, _, _ = L.dz64("bf16" if dtype == BF16 else "f32", "silu", dy[:rows].double(), pre[:rows].double())
        x64 = x[:rows].double()
        tol = L.sum_bound("bf16" if dtype == BF16 else "f32", max(rows, 1), dz.abs().t() @ x64.abs(), True) + off.t() @ x64.abs()
        assert L.fits(dw, dz.t() @ x64, tol + 1e-40, "f32")
    assert ctr.ctr_check_status(full[:size]) == 0 and bool((full[size:] == 0xA5).all())
