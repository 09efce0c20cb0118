"""The norm on the residual stream, its codes and its gradient, against 64-bit plain forms.

Widths cross the kernels' own boundaries (8 lanes, a warp, 2 to 16 warps a row; rows on and off 16 bytes), rows
include none and one; the tolerances are derived in _layers_ref."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R
import _layers_ref as L

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = float(np.float32(1e-6))


def _rows(a, dtype, pad):
    """a [rows, d] on the GPU, its rows pad elements further apart than d; (whole buffer, view)."""
    rows, d = a.shape
    buf = torch.full((max(rows, 1), d + pad), 7.0, dtype=dtype, device="cuda")
    buf[:rows, :d].copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return buf, buf[:rows, :d]


def _wide(t):
    return t.double().cpu().numpy()


def _draw(rows, d, dtype, seed):
    rng = np.random.default_rng(seed)
    a = rng.normal(size=(rows, d)) * np.exp(0.5 * rng.normal(size=(1, d)))
    return _wide(torch.from_numpy(a).to(DT[dtype]))


SIZES = [(0, 16, 0), (1, 1, 0), (1, 1024, 0), (3, 7, 1), (5, 64, 0), (33, 65, 0), (17, 128, 8), (200, 16, 0), (9, 129, 3),
         (40, 256, 0), (13, 257, 0), (64, 479, 0), (64, 480, 16), (31, 512, 4), (12, 513, 0), (10, 1000, 0), (7, 1025, 0),
         (6, 2048, 0), (5, 2050, 2), (3, 4099, 0), (3, 8192, 8), (2, 9001, 0), (2, 16384, 0), (5000, 128, 0),
         (3000, 1024, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,pad", SIZES)
def test_forward(rows, d, pad, dtype):
    x, r = _draw(rows, d, dtype, rows + d), _draw(rows, d, dtype, rows + d + 1)
    rng = np.random.default_rng(d)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    xb, xv = _rows(x, DT[dtype], pad)
    rb, rv = _rows(r, DT[dtype], 2 * pad)
    ws = ctr.workspace(256)
    for residual, g in ((None, gamma), (rv, gamma), (rv, None)):
        sb, sv = _rows(np.full((rows, d), 3.0), DT[dtype], pad)
        yb, yv = _rows(np.full((rows, d), 3.0), DT[dtype], pad)
        q = torch.full((rows, ctr.fp8_padded(d)), 0x55, dtype=torch.uint8, device="cuda")
        scale = torch.full((ctr.fp8_blocks(d), rows), -1.0, device="cuda")
        gt = None if g is None else torch.from_numpy(g).cuda()
        ctr.ctr_rms_norm(xv, residual, gt, EPS, sv, yv, q, scale, ws)
        s = x if residual is None else _wide((torch.from_numpy(x).float() + torch.from_numpy(r).float()).to(DT[dtype]))
        np.testing.assert_array_equal(_wide(sv), s)
        v = L.norm(s, np.ones(d) if g is None else g.astype(np.float64), EPS)[0]
        assert R.within(_wide(yv), v, L.norm_tol(v), dtype)
        assert L.codes_fit(q.cpu().numpy(), _wide(scale), v)
        for b in (sb, yb):
            assert bool((b[:, d:] == 7.0).all()), "a write left its row"
    assert ctr.ctr_check_status(ws) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,pad", SIZES)
def test_gradient_is_the_formulas(rows, d, pad, dtype):
    s, dy, ds = (_draw(rows, d, dtype, rows + d + i) for i in range(3))
    gamma = (1 + 0.2 * np.random.default_rng(d).normal(size=d)).astype(np.float32)
    gt = torch.from_numpy(gamma).cuda()
    sv, dyv, dsv = (_rows(a, DT[dtype], pad)[1] for a in (s, dy, ds))
    need = ctr.ctr_rms_norm_workspace_size(rows, d)
    full = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    full[:256].zero_()
    for stream, g in ((dsv, gt), (None, gt), (dsv, None)):
        db, dv = _rows(np.full((rows, d), 3.0), DT[dtype], pad)
        dg = torch.full((d,), -5.0, device="cuda")
        ctr.ctr_rms_norm_bwd(dyv, stream, sv, g, EPS, dv, dg, full[:need])
        ref, tol, dref, mag = L.norm_grad(dy, ds if stream is not None else 0 * ds, s,
                                          gamma.astype(np.float64) if g is not None else np.ones(d), EPS)
        assert R.within(_wide(dv), ref, tol, dtype)
        assert np.all(np.abs(_wide(dg) - dref) <= L.norm_sums(rows, d) * L.U * mag + 1e-44)
        assert bool((db[:, d:] == 7.0).all()) and bool((full[need:] == 0xA5).all()), "a write left its place"
        again, dg2 = torch.empty_like(dv), torch.empty_like(dg)
        ctr.ctr_rms_norm_bwd(dyv, stream, sv, g, EPS, again, dg2, full[:need])
        assert torch.equal(again, dv) and torch.equal(dg, dg2)


def test_gradient_is_the_differences():
    # central differences in 64 bits of L = sum dy v; fp32's share as in the formulas' bound, third-order term
    # h^2 L''' / 6 < 1e-7 for |L'''| < 1e3, cancellation 1e-16 * 50 / 1e-5
    rows, d, h = 3, 37, 1e-5
    s, dy = _draw(rows, d, "f32", 1), _draw(rows, d, "f32", 2)
    gamma = 1 + 0.2 * np.random.default_rng(3).normal(size=d).astype(np.float32).astype(np.float64)
    gamma = gamma.astype(np.float32).astype(np.float64)
    dx, dg = torch.empty((rows, d), device="cuda"), torch.empty(d, device="cuda")
    t = [torch.from_numpy(a.astype(np.float32)).cuda() for a in (dy, s, gamma)]
    ctr.ctr_rms_norm_bwd(t[0], None, t[1], t[2], EPS, dx, dg, ctr.workspace(ctr.ctr_rms_norm_workspace_size(rows, d)))
    tol = L.norm_grad(dy, 0 * dy, s, gamma, EPS)[1]
    for j in range(d):
        e = np.zeros((1, d))
        e[0, j] = h
        diff = ((L.norm(s + e, gamma, EPS)[0] - L.norm(s - e, gamma, EPS)[0]) * dy).sum(axis=1) / (2 * h)
        assert np.all(np.abs(_wide(dx)[:, j] - diff) <= 1e-7 + tol[:, j])
        diff = ((L.norm(s, gamma + e, EPS)[0] - L.norm(s, gamma - e, EPS)[0]) * dy).sum() / (2 * h)
        assert abs(_wide(dg)[j] - diff) <= 1e-7 + L.norm_sums(rows, d) * L.U * np.abs(dy * s).sum()


@pytest.mark.parametrize("d", [48, 130, 1024, 3000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_the_ends_of_the_range(d, dtype):
    # zeros, squares above and below fp32's range, the type's largest number; a NaN and an infinity stay in their rows
    top = float(torch.finfo(DT[dtype]).max)
    s = _draw(9, d, dtype, 5)
    s[0] = 0
    s[1] *= 2.0 ** 100
    s[2] *= 2.0 ** -100
    s[3] = top
    s[4, ::2] = 0
    s[6, d // 2], s[8, d - 1] = np.nan, -np.inf
    fine = [0, 1, 2, 3, 4, 5, 7]
    for eps in (EPS, 2.0 ** -120):
        x = torch.from_numpy(s).to(DT[dtype]).cuda()
        y = torch.empty_like(x)
        q, scale = torch.empty((9, ctr.fp8_padded(d)), dtype=torch.uint8, device="cuda"), torch.empty(
            (ctr.fp8_blocks(d), 9), device="cuda")
        ctr.ctr_rms_norm(x, None, None, eps, None, y, q, scale, ctr.workspace(256))
        v = L.norm(s[fine], np.ones(d), eps)[0]
        assert R.within(_wide(y)[fine], v, L.norm_tol(v), dtype)
        assert L.codes_fit(q.cpu().numpy()[fine], _wide(scale)[:, fine], v)
        assert np.isnan(_wide(y)[6]).all() and np.isnan(_wide(y)[8, d - 1])


def test_in_place_and_captured():
    rows, d = 300, 479
    x, r = _draw(rows, d, "f32", 1), _draw(rows, d, "f32", 2)
    xs, rs = (torch.from_numpy(a).float().cuda() for a in (x, r))
    s, y = torch.empty_like(xs), torch.empty_like(xs)
    ws = ctr.workspace(256)
    ctr.ctr_rms_norm(xs, rs, None, EPS, s, y, None, None, ws)
    a, b = xs.clone(), rs.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ctr.ctr_rms_norm(a, b, None, EPS, b, a, None, None, ws)   # s over the residual, y over x
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, s) and torch.equal(a, y)
    dy, ds = torch.from_numpy(_draw(rows, d, "f32", 3)).float().cuda(), torch.from_numpy(_draw(rows, d, "f32", 4)).float().cuda()
    ref = torch.empty_like(dy)
    big = ctr.workspace(ctr.ctr_rms_norm_workspace_size(rows, d))
    ctr.ctr_rms_norm_bwd(dy, ds, s, None, EPS, ref, None, big)
    for k in range(3):
        t = [dy.clone(), ds.clone(), s.clone()]
        ctr.ctr_rms_norm_bwd(t[0], t[1], t[2], None, EPS, t[k], None, big)
        assert torch.equal(t[k], ref)


def test_rows_past_two_billion_elements():
    # 70000 rows, 32768 apart: the last rows start past 2^31 elements
    rows, d, ld = 70000, 64, 32768
    buf = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    x = buf[:, 8:8 + d]
    g = torch.Generator(device="cuda").manual_seed(3)
    x.copy_(torch.randn((rows, d), generator=g, device="cuda"))
    y = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    ctr.ctr_rms_norm(x, None, None, EPS, None, y, None, None, ctr.workspace(256))
    pick = torch.tensor([0, 1, 65535, 65536, 65537, rows - 1], device="cuda")
    v = L.norm(_wide(x[pick]), np.ones(d), EPS)[0]
    assert R.within(_wide(y[pick]), v, L.norm_tol(v), "bf16")
