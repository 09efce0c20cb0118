"""Norms of wide rows at the type's largest numbers, and of several widths from two threads at once."""
import threading

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


def test_gradients_of_two_widths_from_two_threads():
    # both widths want more shared memory than a kernel has without asking, one more than the other
    widths, rows = (16384, 12800), 64
    wrong, start = [], threading.Barrier(2)

    def work(d):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                g = torch.Generator(device="cuda").manual_seed(d)
                s, dy = (torch.randn((rows, d), generator=g, device="cuda") for _ in range(2))
                dx, dg = torch.empty_like(s), torch.empty(d, device="cuda")
                ws = ctr.workspace(ctr.ctr_rms_norm_workspace_size(rows, d))
                stream.synchronize()
                start.wait(timeout=60)
                for _ in range(400):
                    ctr.ctr_rms_norm_bwd(dy, None, s, None, EPS, dx, dg, ws)
                stream.synchronize()
                ref = (dy.double() * s.double() / torch.sqrt(s.double().square().mean(1, keepdim=True) + EPS)).sum(0)
                if not bool(((dg.double() - ref).abs() <= 1e-3).all()):
                    wrong.append((d, "dgamma"))
        except Exception as e:   # noqa: BLE001
            wrong.append((d, repr(e)))
    threads = [threading.Thread(target=work, args=(d,)) for d in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
