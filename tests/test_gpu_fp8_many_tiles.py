"""Products with many tiles to a CTA and an fp32 result whose last columns fill an odd number of 32-column
pieces: a piece on its way out must not be overwritten by the next tile's.

The operands are codes and scales drawn directly, and the 64-bit result is of the values that they stand for
(tolerances derived in _experts_ref)."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R

pytestmark = pytest.mark.gpu

WIDTHS = [32, 96, 160, 224, 288, 352]   # 32 past a multiple of 64


def _draw(g, *shape):
    """Code bytes without NaN (0x7f, 0xff), on the device."""
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    return torch.where((c & 127) == 127, c - 1, c)


def _scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") + 0.5


def _value(codes):
    return codes.view(torch.float8_e4m3fn).double()


def _check(call, out, ref, mag, kb):
    """The call, several times over; every element of every result."""
    first = None
    for turn in range(6):
        out.fill_(7.0)
        call()
        got = out.double()
        assert bool(((got - ref).abs() <= 1.01 * R.product_bound(mag, kb)).all()), turn
        first = got if first is None else first
        assert torch.equal(got, first), turn


# one tile row a group on 128 x 128 tiles, several tiles to an SM; CTA pairs, several tiles to each
@pytest.mark.parametrize("groups,rows_each", [(500, 20), (1, 256 * 240)])
@pytest.mark.parametrize("n", WIDTHS)
def test_product(groups, rows_each, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = groups * rows_each
    a, sa = _draw(g, rows, 128), _scales(g, 1, rows)
    b, sb = _draw(g, groups, n, 128), _scales(g, groups, ctr.fp8_blocks(n), 1)
    off = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * rows_each
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, groups, n, 128))
    out = torch.empty((rows, n), device="cuda")
    av = (_value(a) * sa[0].double()[:, None]).view(groups, rows_each, 128)
    bv = _value(b) * sb.double().repeat_interleave(128, 1)[:, :n]
    ref = torch.bmm(av, bv.transpose(1, 2)).view(rows, n)
    mag = torch.bmm(av.abs(), bv.abs().transpose(1, 2)).view(rows, n)
    _check(lambda: ctr.ctr_fp8_matmul(a, sa, b, sb, off, out, ws), out, ref, mag, 1)
    assert ctr.ctr_check_status(ws) == 0


# half of the groups are empty: their tiles follow the others' at once, and are zeros
@pytest.mark.parametrize("n", [512, 352])
@pytest.mark.parametrize("k", WIDTHS)
def test_weight_gradient_beside_empty_groups(n, k):
    rng = np.random.default_rng(k)
    groups = 64
    counts = np.where(np.arange(groups) % 2 == 0, rng.choice([128, 256], size=groups), 0)
    rng.shuffle(counts)
    rows = int(counts.sum())
    padded = ctr.fp8_padded_rows(rows, groups)
    g = torch.Generator(device="cuda").manual_seed(k)
    d, sd = _draw(g, n, padded), _scales(g, padded // 128, n)
    x, sx = _draw(g, k, padded), _scales(g, ctr.fp8_blocks(k), padded // 128)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, groups, n, k))
    out = torch.empty((groups, n, k), device="cuda")
    dv = _value(d) * sd.double().repeat_interleave(128, 0).t()
    xv = _value(x) * sx.double().repeat_interleave(128, 0)[:k].repeat_interleave(128, 1)
    ref, mag = (torch.zeros((groups, n, k), dtype=torch.float64, device="cuda") for _ in range(2))
    for i, c in enumerate(counts):                 # whole blocks: a group's place is its first row
        r = slice(int(off[i]), int(off[i]) + int(c))
        ref[i], mag[i] = dv[:, r] @ xv[:, r].t(), dv[:, r].abs() @ xv[:, r].abs().t()
    _check(lambda: ctr.ctr_fp8_matmul_wgrad(d, sd, x, sx, off, out, ws, rows=rows), out, ref, mag, 2)
    assert ctr.ctr_check_status(ws) == 0
