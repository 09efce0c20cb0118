"""Expert routing and rows into expert order and back, against 64-bit plain forms.

Indices must match exactly; the tolerances of the rest are derived in
_experts_ref.  Sizes cross the kernels' own boundaries (lane groups, tiles of 32
to 256 tokens, one block or several, vector widths) and include zero and one.
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


def _strided(a, dtype, pad, fill=7.0):
    """Rows of a in a wider buffer (stride a.shape[1] + pad) whose other elements hold `fill`; (buffer, view)."""
    T, d = a.shape
    buf = torch.full((max(T, 1), d + pad), fill, dtype=dtype, device="cuda")
    view = buf[:T, :d]
    if T:
        view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dtype))
    return buf, view


def _scores(T, E, dtype, masked, seed):
    rng = np.random.default_rng(seed)
    s = rng.normal(size=(T, E)) + 0.7 * rng.normal(size=(1, E))
    if masked:
        s[rng.random((T, E)) < masked] = -np.inf
        s[rng.random(T) < 0.1] = -np.inf
    t = torch.from_numpy(s).to(DT[dtype])
    return t.double().numpy()


def gpu_route(s, k, renorm, dtype, pad=0):
    T, E = s.shape
    _, x = _strided(s, DT[dtype], pad)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = {"expert": torch.full((T, k), -9, **i32), "weight": torch.full((T, k), -9.0, device="cuda"),
           "slot": torch.full((T, k), -9, **i32), "token": torch.full((T * k,), -9, **i32),
           "offsets": torch.full((E + 1,), -9, **i32)}
    need = ctr.ctr_expert_route_workspace_size(T, E, k)
    full = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    full[:256].zero_()
    ws = full[:need]
    ctr.ctr_expert_route(x, k, renorm, *out.values(), ws)
    st = ctr.ctr_check_status(ws)
    assert np.all(_np(full[need:]) == 0xA5), "a write left the workspace"
    return st, {n: _np(t) for n, t in out.items()}


def check_route(s, k, renorm, dtype, pad=0, status=0):
    st, got = gpu_route(s, k, renorm, dtype, pad)
    assert st == status
    expert, weight, slot, token, offsets, _ = R.route(s, k, renorm)
    np.testing.assert_array_equal(got["expert"], expert)
    np.testing.assert_array_equal(got["offsets"], offsets)
    np.testing.assert_array_equal(got["slot"], slot)
    np.testing.assert_array_equal(got["token"], token)
    assert np.all(np.abs(got["weight"] - weight) <= (s.shape[1] + 8) * R.U * weight + 1e-38)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,masked,pad", [
    (0, 5, 2, 0, 0), (1, 1, 1, 0, 0), (1, 8, 2, 0, 0), (2, 2, 2, 0.5, 3), (31, 7, 3, 0.3, 1), (33, 9, 9, 0.5, 0),
    (256, 64, 4, 0, 0), (257, 64, 5, 0.1, 8), (255, 65, 1, 0, 0), (600, 26, 4, 0.05, 2), (1000, 128, 8, 0, 0),
    (513, 256, 16, 0.2, 0), (700, 257, 4, 0, 7), (300, 512, 16, 0.9, 0), (5000, 16, 2, 0.02, 0),
    (40001, 33, 3, 0.1, 0)])
def test_route(T, E, k, masked, pad, dtype):
    s = _scores(T, E, dtype, masked, 100 * T + E)
    for renorm in (False, True):
        check_route(s, k, renorm, dtype, pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_ties_signed_zeros_and_lowest_values(dtype):
    lowest = float(torch.finfo(DT[dtype]).min)
    s = np.zeros((40, 19))
    s[1::2] = -0.0
    s[4] = lowest                     # the type's lowest value is a score, not a mask
    s[5, :] = lowest
    s[5, 7] = -np.inf
    s[6] = -np.inf                    # nothing left
    s[7, :17] = -np.inf               # fewer left than k
    s[8, 3::4] = 1.0                  # ties at the top
    s[9] = np.where(np.arange(19) % 2, 0.0, -0.0)
    s[10, 18] = float(torch.finfo(DT[dtype]).max)
    for k in (1, 3, 16):
        for renorm in (False, True):
            check_route(s, k, renorm, dtype)


def test_route_nan_and_infinity_are_flagged_and_routed_nowhere():
    s = _scores(300, 20, "f32", 0, 3)
    s[7, 4], s[8, 0], s[299, 19] = np.nan, np.inf, np.nan
    check_route(s, 3, True, "f32", status=ctr.ERR_BAD_VALUE)
    s[8, 0] = 0.5
    s[7, 4] = s[299, 19] = 1.0
    check_route(s, 3, True, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,pad", [(1025, 26, 4, 0), (2049, 26, 4, 0), (3777, 512, 16, 3), (4096, 200, 4, 0), (4097, 40, 1, 0)])
def test_route_around_the_largest_cluster(T, E, k, pad, dtype):
    s = _scores(T, E, dtype, 0.05, T)
    for renorm in (False, True):
        check_route(s, k, renorm, dtype, pad)


@pytest.mark.parametrize("E", [7, 32, 40, 300])
def test_route_every_bf16_number(E):
    # every finite bf16 number, subnormals and both zeros among them, in shuffled rows; a score's distance
    # from the best is rounded once, up to 104 before its exponential leaves fp32
    bits = np.arange(65536, dtype=np.uint32)
    finite = bits[(bits & 0x7f80) != 0x7f80]
    rng = np.random.default_rng(2)
    pick = np.concatenate([rng.permutation(finite), finite[:-len(finite) % E]]).reshape(-1, E)
    s = (pick << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    s[::3] = rng.integers(-2, 3, size=s[::3].shape) * 2.0 ** -133  # ties of the smallest numbers
    for k in (1, 2, 3, 4, 5):
        for renorm in (True, False):
            st, got = gpu_route(s, k, renorm, "bf16")
            assert st == 0
            expert, weight, slot, token, offsets, _ = R.route(s, k, renorm)
            for n, ref in (("expert", expert), ("slot", slot), ("token", token), ("offsets", offsets)):
                np.testing.assert_array_equal(got[n], ref)
            assert np.all(np.abs(got["weight"] - weight) <= (E + 8 + 104) * R.U * weight + 1e-38)


@pytest.mark.parametrize("E", [8, 48])
def test_route_every_bf16_nan_and_infinity_is_flagged_and_routed_nowhere(E):
    bits = np.arange(65536, dtype=np.uint32)
    odd = bits[((bits & 0x7f80) == 0x7f80) & (bits != 0xff80)]   # -inf is a mask
    raw = torch.zeros((2 * len(odd), E), dtype=torch.int16)
    at = np.arange(len(odd))
    raw[2 * at, at % E] = torch.from_numpy(odd.astype(np.uint16).view(np.int16))
    x = raw.view(torch.bfloat16).cuda()
    for k in (1, 3):
        i32 = dict(dtype=torch.int32, device="cuda")
        T = x.shape[0]
        out = [torch.full((T, k), -9, **i32), torch.full((T, k), -9.0, device="cuda"), torch.full((T, k), -9, **i32),
               torch.full((T * k,), -9, **i32), torch.full((E + 1,), -9, **i32)]
        ws = ctr.workspace(ctr.ctr_expert_route_workspace_size(T, E, k))
        ctr.ctr_expert_route(x, k, True, *out, ws)
        assert ctr.ctr_check_status(ws) == ctr.ERR_BAD_VALUE
        assert torch.all(out[0][::2] == -1) and torch.all(out[2][::2] == -1) and torch.all(out[1][::2] == 0)
        assert torch.all(out[0][1::2] == torch.arange(k, device="cuda"))


def test_route_all_tokens_to_one_expert_and_repeats_bit_for_bit():
    s = _scores(30000, 40, "f32", 0, 5)
    s[:, 11] = 50.0
    check_route(s, 2, False, "f32")
    a, b = gpu_route(s, 2, False, "f32")[1], gpu_route(s, 2, False, "f32")[1]
    for n in a:
        np.testing.assert_array_equal(a[n], b[n])


def gpu_route_grad(dw, s, k, renorm, dtype, pad):
    T, E = s.shape
    _, x = _strided(s, DT[dtype], pad)
    expert = torch.from_numpy(R.route(s, k, renorm)[0]).cuda()
    buf, d = _strided(np.full((T, E), -3.0), DT[dtype], pad)
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    ctr.ctr_expert_route_bwd(torch.from_numpy(dw).cuda(), x, renorm, expert, d, ws)
    assert ctr.ctr_check_status(ws) == 0
    if pad and T:
        assert np.all(_np(buf)[:, E:] == 7.0), "a write left its row"
    return _np(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,masked,pad", [
    (1, 1, 1, 0, 0), (1, 8, 2, 0, 0), (37, 9, 4, 0.5, 1), (500, 64, 4, 0.1, 0), (129, 200, 16, 0, 8),
    (65, 300, 5, 0.2, 0), (70, 512, 16, 0, 3), (9000, 26, 3, 0.05, 0)])
def test_route_gradient_is_the_formulas(T, E, k, masked, pad, dtype):
    s = _scores(T, E, dtype, masked, 7 * T + E)
    dw = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    for renorm in (False, True):
        got = gpu_route_grad(dw, s, k, renorm, dtype, pad)
        ref, mag = R.route_grad(dw.astype(np.float64), s, k, renorm)
        assert R.within(got, ref, (2 * E + 24) * R.U * mag + 1e-38, dtype)


def test_route_gradient_is_the_differences():
    # central differences of L = sum dweight * weight in 64 bits; the step leaves every choice as it is
    T, E, k, h = 6, 10, 3, 1e-5
    s = _scores(T, E, "f32", 0.15, 21)
    dw = np.random.default_rng(2).normal(size=(T, k)).astype(np.float32)
    for renorm in (False, True):
        got = gpu_route_grad(dw, s, k, renorm, "f32", 0)
        base = R.route(s, k, renorm)[0]
        for e in range(E):
            step = np.zeros((T, E))
            step[:, e] = h
            lo, hi = R.route(s - step, k, renorm), R.route(s + step, k, renorm)
            assert np.array_equal(lo[0], base) and np.array_equal(hi[0], base)
            diff = ((hi[1] - lo[1]) * dw).sum(axis=1) / (2 * h)
            # third-order term h^2 L''' / 6 < 1e-9, cancellation 1e-16 / h = 1e-11; fp32 as above
            assert np.all(np.abs(got[:, e] - diff) <= 1e-8 + (2 * E + 24) * R.U * 4 * np.abs(dw).sum(axis=1))


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------
ROWS = [(1, 1, 1, "f32", 0), (1, 479, 2, "f32", 0), (7, 3, 4, "bf16", 0), (64, 479, 2, "bf16", 0),
        (65, 480, 2, "bf16", 8), (33, 16, 1, "f32", 0), (500, 130, 3, "f32", 2), (257, 1024, 2, "bf16", 0),
        (100, 1030, 5, "bf16", 2), (40, 2052, 16, "f32", 4), (3000, 64, 2, "bf16", 0)]


def _rows_case(T, d, k, dtype, masked=0.3, seed=0):
    rng = np.random.default_rng(seed + T)
    _, w, slot, token, _, _ = R.route(_scores(T, max(k, 6), "f32", masked, seed), k, True)

    def draw(n):
        return torch.from_numpy(rng.normal(size=(n, d))).to(DT[dtype]).double().numpy()
    return w.astype(np.float32), slot, token, draw(T), draw(T * k), draw(T)


@pytest.mark.parametrize("T,d,k,dtype,pad", ROWS)
def test_rows_into_expert_order_and_back(T, d, k, dtype, pad):
    w, slot, token, x, rows, dy = _rows_case(T, d, k, dtype)
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    sl, tk, wt = (torch.from_numpy(a).cuda() for a in (slot, token, w))
    ref = np.where((token >= 0)[:, None], x[token], 0.0)
    buf, out = _strided(np.full((T * k, d), -5.0), DT[dtype], pad)
    ctr.ctr_expert_dispatch(_strided(x, DT[dtype], pad)[1], sl, tk, out, ws)
    np.testing.assert_array_equal(_np(out), ref)
    assert np.all(_np(buf)[:, d:] == 7.0), "a write left its row"

    live = (slot >= 0)[:, :, None]
    terms = np.where(live, rows[slot], 0.0)
    r_in = _strided(rows, DT[dtype], pad)[1]
    for weight in (wt, None):
        wv = (w if weight is not None else np.ones_like(w)).astype(np.float64)[:, :, None]
        buf, y = _strided(np.full((T, d), -5.0), DT[dtype], pad)
        ctr.ctr_expert_combine(r_in, sl, weight, y, ws)
        ref, mag = (wv * terms).sum(axis=1), np.abs(wv * terms).sum(axis=1)
        assert R.within(_np(y), ref, 1.01 * k * R.U * mag, dtype)
        assert np.all(_np(buf)[:, d:] == 7.0), "a write left its row"

    buf, drows = _strided(np.full((T * k, d), -5.0), DT[dtype], pad)
    dweight = torch.full((T, k), -5.0, device="cuda")
    ctr.ctr_expert_combine_bwd(_strided(dy, DT[dtype], pad)[1], r_in, sl, wt, tk, drows, dweight, ws)
    assert ctr.ctr_check_status(ws) == 0
    dot, mag = (dy[:, None] * terms).sum(axis=2), np.abs(dy[:, None] * terms).sum(axis=2)
    assert np.all(np.abs(_np(dweight) - dot) <= 1.01 * d * R.U * mag)
    ref = np.zeros((T * k, d))
    t, j = np.nonzero(slot >= 0)
    ref[slot[t, j]] = w[t, j][:, None].astype(np.float64) * dy[t]
    assert R.within(_np(drows), ref, 1.01 * R.U * np.abs(ref), dtype)
    assert np.all(_np(buf)[:, d:] == 7.0), "a write left its row"


# enough tokens that a row gets few lanes, down to one
@pytest.mark.parametrize("T,d,k,dtype,pad", [(90001, 1, 1, "bf16", 0), (90001, 7, 2, "f32", 1), (90001, 24, 2, "bf16", 0),
                                             (70003, 64, 2, "f32", 0), (30011, 130, 2, "bf16", 1)])
def test_rows_of_many_tokens(T, d, k, dtype, pad):
    test_rows_into_expert_order_and_back(T, d, k, dtype, pad)


def test_rows_gradients_are_the_differences():
    # L = <dy, combine(rows, weight)> is linear in rows and in weight: a difference of any step is the
    # derivative, up to the rounding of the forward pass (k u |.|) over the step
    T, d, k = 9, 20, 3
    w, slot, token, _, rows, dy = _rows_case(T, d, k, "f32")
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    cu = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (rows.astype(np.float32), slot, w, token,
                                                                     dy.astype(np.float32))]
    drows, dweight = torch.empty_like(cu[0]), torch.empty_like(cu[2])
    ctr.ctr_expert_combine_bwd(cu[4], cu[0], cu[1], cu[2], cu[3], drows, dweight, ws)

    def loss(rw, wt):
        y = torch.empty((T, d), device="cuda")
        ctr.ctr_expert_combine(rw, cu[1], wt, y, ws)
        return (y.double() * cu[4].double()).sum().item()
    size = k * np.abs(rows).max() * np.abs(dy).max() * d
    base = loss(cu[0], cu[2])
    for t, j in ((0, 0), (4, 2), (8, 1)):
        up = cu[2].clone()
        up[t, j] += 1.0
        if slot[t, j] < 0:
            assert dweight[t, j].item() == 0.0 and loss(cu[0], up) == base
            continue
        assert abs(loss(cu[0], up) - base - dweight[t, j].item()) <= 8 * (k + d) * R.U * size
        r = int(slot[t, j])
        up = cu[0].clone()
        up[r, 5] += 1.0
        assert abs(loss(up, cu[2]) - base - drows[r, 5].item()) <= 8 * (k + d) * R.U * size


def test_rows_no_tokens_and_masked_rows_with_nan():
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    e = torch.empty
    ctr.ctr_expert_dispatch(e((0, 4), device="cuda"), e((0, 2), dtype=torch.int32, device="cuda"),
                            e((0,), dtype=torch.int32, device="cuda"), e((0, 4), device="cuda"), ws)
    # a token without rows gets zeros whatever lies in rows nobody refers to
    rows = torch.full((4, 8), float("nan"), device="cuda")
    rows[0] = 1.0
    slot = torch.tensor([[0, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    y = torch.full((2, 8), 5.0, device="cuda")
    ctr.ctr_expert_combine(rows, slot, torch.full((2, 2), float("nan"), device="cuda").nan_to_num_(0.5), y, ws)
    assert torch.equal(y, torch.tensor([[0.5], [0.0]], device="cuda").expand(2, 8))
    assert ctr.ctr_check_status(ws) == 0


def test_rows_slot_out_of_range_is_skipped_and_flagged():
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    rows = torch.ones((4, 8), device="cuda")
    slot = torch.tensor([[0, 4], [1 << 30, 3]], dtype=torch.int32, device="cuda")
    y = torch.empty((2, 8), device="cuda")
    ctr.ctr_expert_combine(rows, slot, None, y, ws)
    assert torch.equal(y, torch.ones_like(y))
    assert ctr.ctr_check_status(ws) == ctr.ERR_INDEX_OUT_OF_RANGE
    assert ctr.ctr_check_status(ws) == 0


def test_rows_past_32_bits_of_elements():
    T, d = 1_100_000, 2048                       # 2.25e9 elements
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16)
    x[:, d - 1] = (torch.arange(T, device="cuda") % 127).to(torch.bfloat16)
    slot = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous().view(T, 1)
    out = torch.full((T, d), -1.0, dtype=torch.bfloat16, device="cuda")
    ws = ctr.workspace(ctr.ctr_expert_workspace_size())
    ctr.ctr_expert_dispatch(x, slot, slot.view(T), out, ws)
    assert torch.equal(out[:, [0, 1, d - 1]].flip(0), x[:, [0, 1, d - 1]])
    y = torch.full_like(out, -1.0)
    ctr.ctr_expert_combine(out, slot, None, y, ws)
    assert torch.equal(y, x)


def test_route_and_rows_on_another_stream():
    s = _scores(4000, 16, "f32", 0, 9)
    x = np.random.default_rng(0).normal(size=(4000, 96)).astype(np.float32)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _, got = gpu_route(s, 2, True, "f32")
        xs = torch.empty((8000, 96), device="cuda")
        ws = ctr.workspace(256)
        ctr.ctr_expert_dispatch(torch.from_numpy(x).cuda(), torch.from_numpy(got["slot"]).cuda(),
                                torch.from_numpy(got["token"]).cuda(), xs, ws)
    side.synchronize()
    np.testing.assert_array_equal(_np(xs), x[got["token"]])
    np.testing.assert_array_equal(got["slot"], R.route(s, 2, True)[2])


def test_refusals_of_shapes_types_and_layouts():
    f, i = torch.empty((4, 8), device="cuda"), torch.empty((4, 2), dtype=torch.int32, device="cuda")
    tok, w, ws = torch.empty(8, dtype=torch.int32, device="cuda"), torch.empty((4, 2), device="cuda"), ctr.workspace(256)
    out = torch.empty((8, 8), device="cuda")
    ctr.ctr_status_reset(ws)
    for bad in (
            lambda: ctr.ctr_expert_dispatch(f.cpu(), i, tok, out, ws),
            lambda: ctr.ctr_expert_dispatch(f.half(), i, tok, out, ws),
            lambda: ctr.ctr_expert_dispatch(f, i.long(), tok, out, ws),
            lambda: ctr.ctr_expert_dispatch(f, i, tok[:7], out, ws),
            lambda: ctr.ctr_expert_dispatch(f, i, tok, out[:7], ws),
            lambda: ctr.ctr_expert_dispatch(f, i, tok, out.bfloat16(), ws),
            lambda: ctr.ctr_expert_dispatch(f.t(), i, tok, out, ws),
            lambda: ctr.ctr_expert_dispatch(f[:1].expand(4, 8), i, tok, out, ws),
            lambda: ctr.ctr_expert_combine(out, i, w[:3], f, ws),
            lambda: ctr.ctr_expert_combine_bwd(f, out, i, w, tok, out, w.double(), ws),
            lambda: ctr.ctr_expert_route(f, 2, True, i, w, i, tok, tok, ws)):
        with pytest.raises(ValueError):
            bad()
    off = torch.empty(9, dtype=torch.int32, device="cuda")
    with pytest.raises(ctr.CtrError) as e:        # the routing needs more than the header
        ctr.ctr_expert_route(f, 2, True, i, w, i, tok, off, ws)
    assert e.value.status == ctr.ERR_WORKSPACE
    with pytest.raises(ctr.CtrError) as e:
        ctr.ctr_expert_dispatch(f, i, tok, out, ws[:128])
    assert e.value.status == ctr.ERR_WORKSPACE
