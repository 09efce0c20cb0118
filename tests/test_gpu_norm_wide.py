"""Norms of wide rows at the type's largest numbers."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R
import _layers_ref as L
from test_gpu_norm import DT, EPS, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [4096, 4120, 8192, 9001, 12289, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_the_largest_numbers(d, dtype):
    # a row of the type's largest number, one of random parts of it, one of a root mean square just past where squares leave
    # fp32's range, and ordinary ones beside them.  rstd may be below 2^-126: half of its last place, 2^-150, is up to 2^-150 /
    # rstd of the result more, and so are products that small
    rng = np.random.default_rng(d)
    top = float(torch.finfo(DT[dtype]).max)
    s = rng.normal(size=(6, d))
    s[0] = top
    s[1] = top * (2 * rng.random(d) - 1)
    s[2] *= 4e18
    s[3] = -top
    s[3, ::2] = 0
    s = _wide(torch.from_numpy(s).to(DT[dtype]))
    x = torch.from_numpy(s).to(DT[dtype]).cuda()
    y = torch.empty_like(x)
    q, scale = torch.empty((6, ctr.fp8_padded(d)), dtype=torch.uint8, device="cuda"), torch.empty((ctr.fp8_blocks(d), 6), device="cuda")
    ctr.ctr_rms_norm(x, None, None, EPS, None, y, q, scale, ctr.workspace(256))
    v, rstd = L.norm(s, np.ones(d), EPS)
    tol = L.norm_tol(v) + np.abs(v) * 2.0 ** -150 / rstd
    assert R.within(_wide(y), v, tol, dtype)
    # gradients: dgamma = sum over rows of dy u
    dy = _wide(torch.from_numpy(rng.normal(size=(6, d))).to(DT[dtype]))
    dg, dx = torch.empty(d, device="cuda"), torch.empty_like(x)
    ctr.ctr_rms_norm_bwd(torch.from_numpy(dy).to(DT[dtype]).cuda(), None, x, None, EPS, dx, dg,
                         ctr.workspace(ctr.ctr_rms_norm_workspace_size(6, d)))
    mag = np.abs(dy * v)
    off = (L.norm_sums(6, d) * L.U * mag + mag * 2.0 ** -150 / rstd).sum(axis=0)
    assert np.all(np.abs(_wide(dg) - (dy * v).sum(axis=0)) <= off + 1e-44)
    assert bool(torch.isfinite(dx).all())
