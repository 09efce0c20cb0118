"""Block-scaled e4m3 codes and their products, against 64-bit plain forms.

Codes and scales must match bit for bit (they are defined by fp32 operations);
products are held to the bound derived in _experts_ref, and to equality where
every sum is exact.
"""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _draw(rng, shape, dtype, spread=True):
    x = rng.normal(size=shape)
    if spread:  # columns of different sizes, a few outliers, an all-zero patch and tiny values
        x = x * np.exp(rng.normal(size=shape[-1:]) * 2)
        flat = x.reshape(-1)
        flat[rng.integers(0, flat.size, size=max(1, flat.size // 500))] *= 1e4
        x[..., :min(2, shape[-1])] *= 1e-20
        if len(shape) == 2 and shape[0] > 3:
            x[3] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


def _u8(*shape):
    return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.full(shape, -7.0, device="cuda")


def _ws():
    return ctr.workspace(256)


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _tiles(counts):
    return [-(-c // 128) for c in counts]


# ---------------------------------------------------------------------------
# codes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 479, 0), (3, 128, 0), (7, 129, 3), (130, 64, 8),
                                           (257, 1024, 0), (1000, 300, 4)])
def test_row_codes(rows, cols, pad, dtype):
    rng = np.random.default_rng(rows + cols)
    x = _draw(rng, (rows, cols), dtype)
    buf = torch.zeros((rows, cols + pad), dtype=DT[dtype], device="cuda")
    buf[:, :cols] = x
    kb = ctr.fp8_blocks(cols)
    q, s = _u8(rows, kb * 128), _f32(kb, rows + 5)[:, :rows]
    ws = _ws()
    ctr.ctr_fp8_quantize_rows(buf[:, :cols], q, s, ws)
    ref, rs = R.quantize(x.double().numpy(), 1, 128)
    got = R.e4m3_values(_np(q))
    np.testing.assert_array_equal(got[:, :cols], ref)
    assert np.all(got[:, cols:] == 0)
    np.testing.assert_array_equal(_np(s).T, rs)
    # the same through a map, with rows that have no source
    idx = rng.integers(-1, rows, size=rows + 9).astype(np.int32)
    q2, s2 = _u8(rows + 9, kb * 128), _f32(kb, rows + 9)
    ctr.ctr_fp8_quantize_rows(buf[:, :cols], q2, s2, ws, row_index=torch.from_numpy(idx).cuda())
    ref2 = np.where((idx >= 0)[:, None], ref[idx], 0.0)
    np.testing.assert_array_equal(R.e4m3_values(_np(q2))[:, :cols], ref2)
    rs2 = np.where((idx >= 0)[:, None], rs[idx], R.scale_of(0.0)[0])
    np.testing.assert_array_equal(_np(s2).T, rs2)
    assert ctr.ctr_check_status(ws) == 0


def test_row_codes_of_every_e4m3_boundary():
    # every code's value, every midpoint between neighbours and their fp32 neighbours, in a block
    # whose largest value is 448 (scale 1)
    v = np.unique(np.abs(R.e4m3_values(np.arange(127, dtype=np.uint8))))
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid]).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))])
    x = np.concatenate([x, -x])
    x = x[np.abs(x) <= 448]
    x = np.concatenate([x, np.zeros(-len(x) % 127)]).reshape(-1, 127)
    x = np.concatenate([x, np.full((len(x), 1), 448.0)], axis=1).astype(np.float32)
    q, s = _u8(len(x), 128), _f32(1, len(x))
    ctr.ctr_fp8_quantize_rows(torch.from_numpy(x).cuda(), q, s, _ws())
    assert np.all(_np(s) == 1.0)
    np.testing.assert_array_equal(R.e4m3_values(_np(q)), R.e4m3_round(x))


def test_nan_and_infinity_stay_visible():
    x = torch.ones((4, 300), device="cuda")
    x[1, 200], x[2, 5] = float("nan"), float("inf")
    w = torch.ones((1, 16, 300), device="cuda")
    q, s, wq, wsc = _u8(4, 384), _f32(3, 4), _u8(1, 16, 384), _f32(1, 1, 3)
    ws = _ws()
    ctr.ctr_fp8_quantize_rows(x, q, s, ws)
    ctr.ctr_fp8_quantize_blocks(w, wq, wsc, ws)
    out = torch.empty((4, 16), device="cuda")
    ctr.ctr_fp8_matmul(q, s, wq, wsc, None, out, ws)
    bad = torch.isnan(out).all(dim=1).cpu().numpy()
    np.testing.assert_array_equal(bad, [False, True, True, False])
    assert np.allclose(_np(out)[[0, 3]], 300.0, rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("groups,n,k", [(1, 1, 1), (1, 128, 128), (3, 130, 479), (2, 64, 257), (5, 200, 96)])
def test_block_codes_and_their_transpose(groups, n, k, dtype):
    rng = np.random.default_rng(n + k)
    w = _draw(rng, (groups, n, k), dtype)
    nb, kb = ctr.fp8_blocks(n), ctr.fp8_blocks(k)
    q, s, qt, st = _u8(groups, n, kb * 128), _f32(groups, nb, kb), _u8(groups, k, nb * 128), _f32(groups, kb, nb)
    ws = _ws()
    ctr.ctr_fp8_quantize_blocks(w.cuda(), q, s, ws, qt, st)
    q1, s1 = _u8(groups, n, kb * 128), _f32(groups, nb, kb)
    ctr.ctr_fp8_quantize_blocks(w.cuda(), q1, s1, ws)
    assert torch.equal(q, q1) and torch.equal(s, s1)
    for g in range(groups):
        ref, rs = R.quantize(w[g].double().numpy(), 128, 128)
        got, gt = R.e4m3_values(_np(q[g])), R.e4m3_values(_np(qt[g]))
        np.testing.assert_array_equal(got[:, :k], ref)
        np.testing.assert_array_equal(gt[:, :n], ref.T)
        assert np.all(got[:, k:] == 0) and np.all(gt[:, n:] == 0)
        np.testing.assert_array_equal(_np(s[g]), rs)
        np.testing.assert_array_equal(_np(st[g]), rs.T)


GROUPED = [([0], 40), ([1], 1), ([5, 0, 130, 128], 479), ([0, 0, 300], 64), ([127, 129, 1, 0, 0, 256, 3], 200)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,cols", GROUPED)
@pytest.mark.parametrize("extra", [0, 7])
def test_row_and_column_codes_of_groups(counts, cols, extra, dtype):
    rng = np.random.default_rng(sum(counts) + cols)
    off = _offsets(counts)
    rows = int(off[-1]) + extra                   # `extra` rows belong to no group
    src = _draw(rng, (max(rows, 2), cols), dtype)
    idx = rng.integers(0, max(rows, 2), size=rows).astype(np.int32)
    x = src.double().numpy()[idx]
    G, kb, Rp = len(counts), ctr.fp8_blocks(cols), ctr.fp8_padded_rows(rows, len(counts))
    ref, rs = R.quantize(x, 1, 128) if rows else (np.zeros((0, cols)), np.zeros((0, kb)))
    ws = _ws()
    for by in (ctr.FP8_COLS_BY_COLUMN, ctr.FP8_COLS_BY_BLOCK):
        q, s, qc = _u8(rows, kb * 128), _f32(kb, rows), _u8(cols, Rp)
        sc = _f32(Rp // 128, cols) if by == ctr.FP8_COLS_BY_COLUMN else _f32(kb, Rp // 128)
        ctr.ctr_fp8_quantize_rows_cols(src.cuda(), torch.from_numpy(off).cuda(), q, s, qc, sc, by, ws,
                                       row_index=torch.from_numpy(idx).cuda())
        used = int(off[-1])
        got = R.e4m3_values(_np(q))[:used]
        np.testing.assert_array_equal(got[:, :cols], ref[:used])
        assert np.all(got[:, cols:] == 0)
        np.testing.assert_array_equal(_np(s).T[:used], rs[:used])
        gc, gs = R.e4m3_values(_np(qc)), _np(sc)
        tile = 0
        for g, c in enumerate(counts):
            for r0 in range(0, c, 128):
                part = x[off[g] + r0:off[g] + min(c, r0 + 128)]
                full = np.zeros((128, cols))
                full[:len(part)] = part
                per_col = by == ctr.FP8_COLS_BY_COLUMN
                rq, rsc = R.quantize(full, 128, 1 if per_col else 128)
                np.testing.assert_array_equal(gc[:, tile * 128:(tile + 1) * 128], rq.T)
                np.testing.assert_array_equal(gs[tile] if per_col else gs[:, tile], rsc[0])
                tile += 1
    assert ctr.ctr_check_status(ws) == 0


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def _product_case(counts, n, k, dtype, seed=0, extra=0):
    rng = np.random.default_rng(seed + n + k + sum(counts))
    off = _offsets(counts)
    rows = int(off[-1]) + extra
    x, w = _draw(rng, (max(rows, 1), k), dtype)[:rows], _draw(rng, (len(counts), n, k), dtype, spread=False)
    return off, rows, x, w


def _values(x, w):
    """Values that row codes of x and block codes of w stand for (fp64)."""
    k = x.shape[1]
    q, s = R.quantize(x, 1, 128) if len(x) else (np.zeros((0, k)), np.zeros((0, -(-k // 128))))
    a = q * R.spread(s, 1, 128, *x.shape)
    b = []
    for g in range(len(w)):
        q, s = R.quantize(w[g], 128, 128)
        b.append(q * R.spread(s, 128, 128, *w[g].shape))
    return a, b


def _codes(x, w, ws):
    rows, k = x.shape
    G, n, _ = w.shape
    kb, nb = ctr.fp8_blocks(k), ctr.fp8_blocks(n)
    q, s, wq, wsc = _u8(rows, kb * 128), _f32(kb, rows), _u8(G, n, kb * 128), _f32(G, nb, kb)
    ctr.ctr_fp8_quantize_rows(x.cuda(), q, s, ws)
    ctr.ctr_fp8_quantize_blocks(w.cuda(), wq, wsc, ws)
    return q, s, wq, wsc


PRODUCTS = [([1], 1, 1), ([1], 1024, 479), ([3], 16, 130), ([130], 129, 128), ([64, 0, 1, 63], 96, 300),
            ([0, 0, 5], 200, 128), ([300, 129, 0, 255], 257, 500), ([1000], 520, 1100), ([128] * 9, 64, 64),
            ([2] * 40, 300, 200), ([33] * 3, 640, 256), ([5000, 1, 3000], 700, 260)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,n,k", PRODUCTS)
def test_product(counts, n, k, out, dtype):
    off, rows, x, w = _product_case(counts, n, k, dtype, extra=3)
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, len(counts), n, k))
    codes = _codes(x, w, ws)
    a, b = _values(x.double().numpy(), w.double().numpy())
    for pad in (0, 5, -n % 32):
        buf = torch.full((rows, n + pad), 7.0, dtype=DT[out], device="cuda")
        ctr.ctr_fp8_matmul(*codes, torch.from_numpy(off).cuda(), buf[:, :n], ws)
        assert ctr.ctr_check_status(ws) == 0
        got = _np(buf)
        assert np.all(got[:, n:] == 7.0), "a write left its row"
        assert np.all(got[off[-1]:, :n] == 0.0), "rows of no group"
        for g in range(len(counts)):
            r = slice(off[g], off[g + 1])
            ref, mag = a[r] @ b[g].T, np.abs(a[r]) @ np.abs(b[g]).T
            assert R.within(got[r, :n], ref, R.product_bound(mag, ctr.fp8_blocks(k)) * 1.01, out)


@pytest.mark.parametrize("rows,n,k", [(1, 300, 700), (16, 130, 256), (200, 256, 384), (1500, 1300, 640)])
def test_product_of_exact_sums_is_exact(rows, n, k):
    # small integers, and one 448 in each block that meets zeros: scales are 1, every sum below 2^24
    rng = np.random.default_rng(rows)
    x = rng.integers(-8, 9, size=(rows, k)).astype(np.float32)
    w = rng.integers(-8, 9, size=(1, n, k)).astype(np.float32)
    x[:, 0::128], w[:, :, 0::128] = 448, 0
    w[:, 0::128, 1::128], x[:, 1::128] = 448, 0
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 1, n, k))
    xt, wt = torch.from_numpy(x), torch.from_numpy(w)
    codes = _codes(xt, wt, ws)
    assert torch.all(codes[1] == 1.0) and torch.all(codes[3] == 1.0)
    out = torch.empty((rows, n), device="cuda")
    ctr.ctr_fp8_matmul(*codes, None, out, ws)
    np.testing.assert_array_equal(_np(out), x @ w[0].T)
    again = torch.empty_like(out)
    ctr.ctr_fp8_matmul(*codes, None, again, ws)
    assert torch.equal(out, again)


def test_product_of_no_rows_and_bad_offsets():
    off, rows, x, w = _product_case([4, 6], 40, 200, "f32")
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 2, 40, 200))
    q, s, wq, wsc = _codes(x, w, ws)
    e = torch.empty
    ctr.ctr_fp8_matmul(e((0, 256), dtype=torch.uint8, device="cuda"), e((2, 0), device="cuda"), wq, wsc,
                       torch.zeros(3, dtype=torch.int32, device="cuda"), e((0, 40), device="cuda"), ws)
    assert ctr.ctr_check_status(ws) == 0
    for bad in ([0, 7, 3], [1, 4, 10], [0, 4, 11], [0, -1, 10]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = torch.full((rows, 40), 7.0, device="cuda")
        ctr.ctr_fp8_matmul(q, s, wq, wsc, o, out, ws)
        assert ctr.ctr_check_status(ws) == ctr.ERR_BAD_OFFSETS
        assert torch.all(out == 0)
        qc, sc = _u8(200, ctr.fp8_padded_rows(rows, 2)), _f32(2, ctr.fp8_padded_rows(rows, 2) // 128)
        q2, s2 = _u8(rows, 256), _f32(2, rows)
        ctr.ctr_fp8_quantize_rows_cols(x.cuda(), o, q2, s2, qc, sc, ctr.FP8_COLS_BY_BLOCK, ws)
        assert ctr.ctr_check_status(ws) == ctr.ERR_BAD_OFFSETS
        assert torch.all(qc == 0x55) and torch.all(q2 == 0x55)


def _train(off, rows, x, dy, w, out):
    G, n, k = w.shape
    kb, nb, Rp = ctr.fp8_blocks(k), ctr.fp8_blocks(n), ctr.fp8_padded_rows(rows, G)
    ws = ctr.workspace(max(ctr.ctr_fp8_matmul_workspace_size(rows, G, n, k),
                           ctr.ctr_fp8_matmul_workspace_size(rows, G, k, n)))
    o = torch.from_numpy(off).cuda()
    xq, xs, xc, xcs = _u8(rows, kb * 128), _f32(kb, rows), _u8(k, Rp), _f32(kb, Rp // 128)
    dq, ds, dc, dcs = _u8(rows, nb * 128), _f32(nb, rows), _u8(n, Rp), _f32(Rp // 128, n)
    wq, wsc, wt, wts = _u8(G, n, kb * 128), _f32(G, nb, kb), _u8(G, k, nb * 128), _f32(G, kb, nb)
    ctr.ctr_fp8_quantize_rows_cols(x.cuda(), o, xq, xs, xc, xcs, ctr.FP8_COLS_BY_BLOCK, ws)
    ctr.ctr_fp8_quantize_rows_cols(dy.cuda(), o, dq, ds, dc, dcs, ctr.FP8_COLS_BY_COLUMN, ws)
    ctr.ctr_fp8_quantize_blocks(w.cuda(), wq, wsc, ws, wt, wts)
    dx = torch.full((rows, k), 7.0, dtype=DT[out], device="cuda")
    dw = torch.full((G, n, k), 7.0, dtype=DT[out], device="cuda")
    ctr.ctr_fp8_matmul(dq, ds, wt, wts, o, dx, ws)
    ctr.ctr_fp8_matmul_wgrad(dc, dcs, xc, xcs, o, dw, ws, rows=rows)
    assert ctr.ctr_check_status(ws) == 0
    return _np(dx), _np(dw)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("counts,n,k", [([1], 1, 1), ([40, 0, 200], 130, 479), ([128, 256, 1], 64, 128),
                                        ([700], 300, 257), ([9] * 20, 520, 96), ([3000, 2, 900], 512, 640)])
def test_gradients_are_the_formulas(counts, n, k, dtype, out):
    off, rows, x, w = _product_case(counts, n, k, dtype, seed=5)
    dy = _draw(np.random.default_rng(1), (rows, n), dtype)
    dx, dw = _train(off, rows, x, dy, w, out)
    xv, dv, wv = (t.double().numpy() for t in (x, dy, w))
    a, b = _values(dv, wv)
    for g in range(len(counts)):
        r = slice(off[g], off[g + 1])
        ref, mag = a[r] @ b[g], np.abs(a[r]) @ np.abs(b[g])
        assert R.within(dx[r], ref, R.product_bound(mag, ctr.fp8_blocks(n)) * 1.01, out)
        c = counts[g]
        if c == 0:
            assert np.all(dw[g] == 0)
            continue
        q, s = R.quantize(dv[r], 128, 1)
        d_val = q * R.spread(s, 128, 1, c, n)
        q, s = R.quantize(xv[r], 128, 128)
        x_val = q * R.spread(s, 128, 128, c, k)
        ref, mag = d_val.T @ x_val, np.abs(d_val).T @ np.abs(x_val)
        assert R.within(dw[g], ref, R.product_bound(mag, _tiles([c])[0]) * 1.01, out)


# sums long enough to be taken in parts: a few columns; one part of a block; uneven, empty and tiny groups;
# rows past the last group; result rows that are not 16-byte aligned
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,spare,n,k", [([5000], 0, 64, 70), ([16384], 0, 200, 479), ([2049], 300, 300, 260),
                                              ([9000, 0, 3, 7000], 0, 300, 257), ([1, 6000], 100, 130, 128),
                                              ([3000, 0, 2500, 40, 4000, 0, 900, 700], 0, 129, 300),
                                              ([5000, 0, 40, 300, 2500] + [200] * 8, 50, 300, 260),
                                              ([0] * 39 + [4000], 0, 260, 130)])
def test_weight_gradient_of_long_sums(counts, spare, n, k, out):
    rng = np.random.default_rng(6)
    off, rows, G = _offsets(counts), sum(counts) + spare, len(counts)
    x, dy = _draw(rng, (rows, k), "bf16"), _draw(rng, (rows, n), "bf16")
    Rp = ctr.fp8_padded_rows(rows, G)
    kb, nb = ctr.fp8_blocks(k), ctr.fp8_blocks(n)
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, G, n, k))
    o = torch.from_numpy(off).cuda()
    xc, xcs, dc, dcs = _u8(k, Rp), _f32(kb, Rp // 128), _u8(n, Rp), _f32(Rp // 128, n)
    ctr.ctr_fp8_quantize_rows_cols(x.cuda(), o, _u8(rows, kb * 128), _f32(kb, rows), xc, xcs, ctr.FP8_COLS_BY_BLOCK, ws)
    ctr.ctr_fp8_quantize_rows_cols(dy.cuda(), o, _u8(rows, nb * 128), _f32(nb, rows), dc, dcs, ctr.FP8_COLS_BY_COLUMN,
                                   ws)
    got = []
    for _ in range(2):
        dw = torch.full((G, n, k), 7.0, dtype=DT[out], device="cuda")
        ctr.ctr_fp8_matmul_wgrad(dc, dcs, xc, xcs, o, dw, ws, rows=rows)
        got.append(dw)
    assert ctr.ctr_check_status(ws) == 0
    assert torch.equal(got[0], got[1])
    dw, xv, dv = _np(got[0]), x.double().numpy(), dy.double().numpy()
    for g, c in enumerate(counts):
        if c == 0:
            assert np.all(dw[g] == 0)
            continue
        r = slice(off[g], off[g + 1])
        q, s = R.quantize(dv[r], 128, 1)
        d_val = q * R.spread(s, 128, 1, c, n)
        q, s = R.quantize(xv[r], 128, 128)
        x_val = q * R.spread(s, 128, 128, c, k)
        ref, mag = d_val.T @ x_val, np.abs(d_val).T @ np.abs(x_val)
        assert R.within(dw[g], ref, R.product_bound(mag, _tiles([c])[0]) * 1.01, out)


def test_weight_gradient_of_long_sums_bad_offsets_and_small_workspace():
    rows, n, k = 6000, 64, 64
    Rp = ctr.fp8_padded_rows(rows, 2)
    need = ctr.ctr_fp8_matmul_workspace_size(rows, 2, n, k)
    assert need > 256                             # the sums' parts are in it
    ws = ctr.workspace(need)
    xc, dc = torch.zeros((k, Rp), dtype=torch.uint8, device="cuda"), torch.zeros((n, Rp), dtype=torch.uint8, device="cuda")
    xcs, dcs = torch.ones((1, Rp // 128), device="cuda"), torch.ones((Rp // 128, n), device="cuda")
    for bad in ([0, 7, 3], [1, 4, 10], [0, 4, rows + 1], [0, -1, 10]):
        dw = torch.full((2, n, k), 7.0, device="cuda")
        ctr.ctr_fp8_matmul_wgrad(dc, dcs, xc, xcs, torch.tensor(bad, dtype=torch.int32, device="cuda"), dw, ws, rows=rows)
        assert ctr.ctr_check_status(ws) == ctr.ERR_BAD_OFFSETS
        assert torch.all(dw == 0)
    o = torch.tensor([0, 10, rows], dtype=torch.int32, device="cuda")
    with pytest.raises(ctr.CtrError) as e:
        ctr.ctr_fp8_matmul_wgrad(dc, dcs, xc, xcs, o, dw, ctr.workspace(need - 256), rows=rows)
    assert e.value.status == ctr.ERR_WORKSPACE


def test_gradients_are_the_differences():
    # L = <dy, W x>.  Small integers with a 448 in every scale's block: all scales are 1, the codes hold
    # every value, the sums looked at stay below 2^24, so a difference of L by any step is the gradient
    rng = np.random.default_rng(8)
    counts, n, k = [20, 150], 40, 60
    off, rows = _offsets(counts), sum(counts)
    x, dy, w = (rng.integers(-8, 9, size=sh).astype(np.float32) for sh in ((rows, k), (rows, n), (2, n, k)))
    x[:, 0] = dy[:, 0] = 448
    dy[[0, 20, 148]] = 448                        # the first row of each tile of 128 rows of a group
    w[:, :, 0] = 0
    w[:, 0, 0] = 448
    dx, dw = _train(off, rows, *(torch.from_numpy(v) for v in (x, dy, w)), "f32")

    def loss(xx, ww):
        parts = [(dy[a:b].astype(np.float64) * (xx[a:b].astype(np.float64) @ ww[g].T)).sum()
                 for g, (a, b) in enumerate(zip(off[:-1], off[1:]))]
        return sum(parts)
    base = loss(x, w)
    for r, c in ((0, 3), (19, 59), (20, 1), (169, 30)):
        up = x.copy()
        up[r, c] += 1
        assert loss(up, w) - base == dx[r, c]
    for g, i, c in ((0, 0, 1), (0, 39, 59), (1, 5, 0), (1, 39, 33)):
        up = w.copy()
        up[g, i, c] += 1
        assert loss(x, up) - base == dw[g, i, c]


def test_product_past_32_bits_of_elements():
    rows, n, k = 540_000, 4096, 128               # 2.2e9 results
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 448.0
    x[:, 1] = (torch.arange(rows, device="cuda") % 15 + 1).to(torch.bfloat16)
    w = torch.zeros((1, n, k), dtype=torch.bfloat16, device="cuda")
    w[:, :, 1] = 2.0
    w[:, ::128, 2] = 448.0
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 1, n, k))
    q, s, wq, wsc = _u8(rows, 128), _f32(1, rows), _u8(1, n, 128), _f32(1, n // 128, 1)
    ctr.ctr_fp8_quantize_rows(x, q, s, ws)
    ctr.ctr_fp8_quantize_blocks(w, wq, wsc, ws)
    out = torch.full((rows, n), -1.0, dtype=torch.bfloat16, device="cuda")
    ctr.ctr_fp8_matmul(q, s, wq, wsc, None, out, ws)
    assert ctr.ctr_check_status(ws) == 0
    ref = (x[:, 1] * 2).view(rows, 1)
    for c in range(0, n, 512):
        assert torch.equal(out[:, c:c + 512], ref.expand(rows, 512))


def test_product_on_another_stream_beside_itself():
    # two products at once on two streams, each with its own workspace
    off, rows, x, w = _product_case([2000, 1500], 600, 500, "bf16")
    ws = [ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 2, 600, 500)) for _ in range(2)]
    codes = _codes(x, w, ws[0])
    o = torch.from_numpy(off).cuda()
    ref = torch.empty((rows, 600), device="cuda")
    ctr.ctr_fp8_matmul(*codes, o, ref, ws[0])
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(ref) for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                ctr.ctr_fp8_matmul(*codes, o, outs[i], ws[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)


def test_products_in_a_captured_graph():
    off, rows, x, w = _product_case([40, 50], 96, 300, "bf16")
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 2, 96, 300))
    xd, o = x.cuda(), torch.from_numpy(off).cuda()
    q, s, wq, wsc = _codes(x, w, ws)
    out = torch.empty((rows, 96), device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ctr.ctr_fp8_quantize_rows(xd, q, s, ws)
        ctr.ctr_fp8_matmul(q, s, wq, wsc, o, out, ws)
    for scale in (1.0, 2.0):
        xd.copy_(x * scale)
        out.zero_()
        g.replay()
        eager = torch.empty_like(out)
        ctr.ctr_fp8_matmul(*_codes(x * scale, w, ws), o, eager, ws)
        assert torch.equal(out, eager)


def test_refusals():
    off, rows, x, w = _product_case([4, 6], 40, 200, "f32")
    ws = ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(rows, 2, 40, 200))
    q, s, wq, wsc = _codes(x, w, ws)
    o, out = torch.from_numpy(off).cuda(), torch.empty((rows, 40), device="cuda")
    xd = x.cuda()
    for bad in (
            lambda: ctr.ctr_fp8_quantize_rows(xd.double(), q, s, ws),
            lambda: ctr.ctr_fp8_quantize_rows(xd, q[:, :200], s, ws),
            lambda: ctr.ctr_fp8_quantize_rows(xd[:5], q, s, ws),
            lambda: ctr.ctr_fp8_quantize_rows(xd, q, s[:, :9], ws),
            lambda: ctr.ctr_fp8_quantize_rows(xd, q, s, ws, row_index=torch.zeros(rows, device="cuda")),
            lambda: ctr.ctr_fp8_quantize_blocks(w.cuda(), wq, wsc, ws, qt=wq),
            lambda: ctr.ctr_fp8_quantize_blocks(w.cuda()[0], wq, wsc, ws),
            lambda: ctr.ctr_fp8_matmul(q, s, wq, wsc, o[:2], out, ws),
            lambda: ctr.ctr_fp8_matmul(q, s, wq, wsc[:, :, :1], o, out, ws),
            lambda: ctr.ctr_fp8_matmul(q, s, wq, wsc, o, out[:, :39], ws),
            lambda: ctr.ctr_fp8_matmul(q, s, wq, wsc, o, out.half(), ws),
            lambda: ctr.ctr_fp8_matmul(q[:5], s, wq, wsc, o, out, ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ctr.CtrError) as e:        # two groups need offsets
        ctr.ctr_fp8_matmul(q, s, wq, wsc, None, out, ws)
    assert e.value.status == ctr.ERR_INVALID_ARG
    ctr.ctr_fp8_quantize_rows(xd, q, s, ws, row_index=torch.full((rows,), 10, dtype=torch.int32, device="cuda"))
    assert ctr.ctr_check_status(ws) == ctr.ERR_INDEX_OUT_OF_RANGE
