"""Balanced routing against a 64-bit plain form: indices match exactly, ties and near ties among them."""
import numpy as np
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _experts_ref as R
import _layers_ref as L

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BOTH = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


def _scores(T, E, dtype, masked, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    s = spread * (rng.normal(size=(T, E)) + 0.5 * rng.normal(size=(1, E)))
    if masked:
        s[rng.random((T, E)) < masked] = -np.inf
        s[rng.random(T) < 0.1] = -np.inf
    return torch.from_numpy(s).to(DT[dtype]).double().numpy()


def _bias(E, seed, scale=0.1):
    return (scale * np.random.default_rng(seed).normal(size=E)).astype(np.float32)


def _on(a, dtype, pad=0):
    buf = torch.full((max(a.shape[0], 1), a.shape[1] + pad), 7.0, dtype=DT[dtype], device="cuda")
    buf[:a.shape[0], :a.shape[1]].copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return buf[:a.shape[0], :a.shape[1]]


def gpu(s, k, score, bias, groups, group_k, renorm, factor, dtype, pad=0):
    T, E = s.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((T, k), -9, **i32), torch.full((T, k), -9.0, device="cuda"), torch.full((T, k), -9, **i32),
           torch.full((T * k,), -9, **i32), torch.full((E + 1,), -9, **i32)]
    need = ctr.ctr_expert_route_workspace_size(T, E, k)
    full = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    full[:256].zero_()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ctr.ctr_expert_route_balanced(_on(s, dtype, pad), k, ctr.SCORES[score], b, groups, group_k, renorm, factor, *out,
                                  full[:need])
    st = ctr.ctr_check_status(full[:need])
    assert bool((full[need:] == 0xA5).all()), "a write left the workspace"
    return st, [t.cpu().numpy() for t in out]


def check(s, k, score, bias, groups, group_k, renorm, dtype, factor=1.0, pad=0, status=0):
    st, got = gpu(s, k, score, bias, groups, group_k, renorm, factor, dtype, pad)
    assert st == status
    expert, weight, slot, token, offsets, p = L.balanced(s, k, score, bias, groups, group_k, renorm, factor)
    for a, b in zip((got[0], got[4], got[2], got[3]), (expert, offsets, slot, token)):
        np.testing.assert_array_equal(a, b)
    # softmax: (E + 8) u; an exponent is rounded once, below 104 before it leaves fp32; the factor once
    assert np.all(np.abs(got[1] - weight) <= (s.shape[1] + 113) * L.U * np.abs(weight) + 1e-37)
    return expert, p


SIZES = [(0, 8, 2, 2, 1, 0, 0), (1, 1, 1, 1, 1, 0, 0), (1, 64, 6, 8, 4, 0, 0), (2, 6, 3, 3, 2, 0.3, 1), (33, 26, 4, 1, 1, 0.3, 0),
         (200, 24, 5, 4, 2, 0.2, 3), (255, 64, 8, 8, 1, 0, 0), (256, 32, 16, 32, 16, 0.1, 0), (300, 256, 8, 8, 4, 0, 8),
         (257, 96, 4, 3, 2, 0.1, 0), (1000, 130, 7, 13, 5, 0.5, 0), (513, 512, 16, 16, 8, 0.2, 0), (130, 480, 9, 30, 7, 0, 5),
         (700, 160, 4, 10, 3, 0.05, 0), (3000, 16, 2, 2, 1, 0.9, 0), (4500, 72, 6, 9, 4, 0.1, 1), (20001, 40, 3, 5, 3, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,group_k,masked,pad", SIZES)
def test_routing(T, E, k, groups, group_k, masked, pad, dtype):
    s = _scores(T, E, dtype, masked, T + E)
    for score, renorm in BOTH:
        check(s, k, score, _bias(E, E), groups, group_k, renorm, dtype, factor=2.5, pad=pad)
    check(s, k, "sigmoid", None, groups, group_k, True, dtype, pad=pad)
    check(s, k, "softmax", None, groups, group_k, False, dtype, factor=-0.5, pad=pad)


@pytest.mark.parametrize("cluster", [True, False])
def test_one_launch_and_three_agree(cluster):
    s = _scores(3000, 64, "f32", 0.1, 1)
    before = ctr.ctr_set_route_cluster(cluster)
    try:
        check(s, 6, "sigmoid", _bias(64, 2), 8, 4, True, "f32")
    finally:
        ctr.ctr_set_route_cluster(before)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,group_k,k", [(16, 1, 1, 16), (24, 4, 2, 5), (64, 8, 4, 6), (128, 16, 3, 9), (256, 8, 4, 8)])
def test_keys_a_few_times_1e_8_apart(E, groups, group_k, k, score):
    # biases that bring every expert's key to the same value but for the bias's own rounding: fp32 keys cannot order them
    rng = np.random.default_rng(E)
    base = rng.normal(size=E).astype(np.float32).astype(np.float64)
    p = L.balanced(base[None], 1, score, None, 1, 1, False, 1.0)[5][0]
    bias = (0.9 - p).astype(np.float32)
    s = np.repeat(base[None], 600, axis=0)
    drop = rng.random(s.shape) < 0.3
    if score == "sigmoid":   # a softmax's other values would move
        s[drop] = -np.inf
    check(s, k, score, bias, groups, group_k, True, "f32")
    # the same of the groups' sums alone: two of each group stand out, by as much
    if groups > 1:
        far = np.where(np.arange(E) % (E // groups) < 2, bias + np.float32(2), bias).astype(np.float32)
        check(s, k, score, far, groups, group_k, False, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lower_index(dtype):
    s = np.zeros((40, 48))
    s[1::2] = -0.0
    s[4, 3::4] = 1.0
    s[5] = -np.inf
    s[6, :46] = -np.inf
    s[7] = np.arange(48) // 6 % 2
    s[8] = float(torch.finfo(DT[dtype]).min)
    for bias in (None, np.zeros(48, dtype=np.float32), np.full(48, -0.25, dtype=np.float32)):
        for groups, group_k in ((1, 1), (8, 3), (16, 16), (4, 2)):
            for score, renorm in BOTH:
                check(s, 5, score, bias, groups, group_k, renorm, dtype)


def test_masked_by_bias_and_bad_biases():
    s = _scores(300, 32, "f32", 0.1, 4)
    bias = _bias(32, 5)
    bias[[0, 9, 10, 11]] = -np.inf
    for score, renorm in BOTH:
        check(s, 4, score, bias, 8, 3, renorm, "f32")
    bias[3], bias[20] = np.nan, np.inf
    check(s, 4, "sigmoid", bias, 8, 3, True, "f32", status=ctr.ERR_BAD_VALUE)
    bias[:] = -np.inf
    check(s, 4, "softmax", bias, 1, 1, True, "f32")
    s[7, 4], s[8, 0], s[299, 31] = np.nan, np.inf, np.nan
    check(s, 4, "sigmoid", _bias(32, 6), 8, 3, True, "f32", status=ctr.ERR_BAD_VALUE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,groups,group_k,k", [(32, 1, 1, 1), (32, 8, 3, 4), (64, 4, 2, 6), (256, 8, 4, 8), (256, 16, 3, 16),
                                                (130, 13, 5, 7)])
def test_equal_scores_beside_almost_equal_keys(E, groups, group_k, k, dtype):
    # scores of a few values whose score functions differ by 1e-6 to 1e-14: in fp32 they, and many equal ones, are one key
    rng = np.random.default_rng(E + k)
    tops = [np.array(v) for v in ([20.0, 20.5], [14.0, 14.25, 20.0], [12.0, 30.0, 31.0, 32.0], [-0.5, 20.0, 20.5],
                                  [-20.0, -20.5, -21.0], [-90.0, -60.0, -20.0], [1.0, 1.0 + 2.0 ** -23],
                                  [-86.5, -87.0, -87.5, -88.0], [-87.5, 0.0, -87.0, -88.5, -103.0], [-96.0, 5.0, -100.0, -104.0])]
    for v in tops:
        s = torch.from_numpy(v[rng.integers(0, len(v), size=(200, E))]).to(DT[dtype]).double().numpy()
        s[::2][rng.random((100, E)) < 0.9] = v[0] if dtype == "f32" else float(torch.tensor(v[0]).to(torch.bfloat16))
        s[5::7][rng.random(s[5::7].shape) < 0.3] = -np.inf
        for bias in (None, np.zeros(E, dtype=np.float32), np.repeat(_bias(groups, 7), E // groups)):
            for score, renorm in (("sigmoid", True), ("softmax", True)):
                check(s, k, score, bias, groups, group_k, renorm, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spread", [4.0, 8.0, 16.0, 40.0])
def test_peaked_scores(spread, dtype):
    for T, E, groups, group_k, k in ((400, 256, 8, 4, 8), (400, 64, 8, 4, 6), (300, 96, 3, 2, 4), (300, 32, 16, 5, 9)):
        s = _scores(T, E, dtype, 0.1, E, spread)
        for score in ("sigmoid", "softmax"):
            for bias in (None, _bias(E, 3)):
                check(s, k, score, bias, groups, group_k, True, dtype)


@pytest.mark.parametrize("low", [-50.0, -62.5, -64.0, -1e4, -1e9, float(torch.finfo(torch.float32).min)])
def test_experts_pushed_out_by_finite_biases(low):
    rng = np.random.default_rng(3)
    for E, groups, group_k, k, part in ((32, 1, 1, 4, 0.3), (32, 8, 3, 4, 0.3), (64, 8, 4, 6, 0.9), (16, 4, 4, 16, 0.5),
                                        (256, 8, 4, 8, 0.1), (256, 16, 3, 16, 0.7)):
        s = _scores(400, E, "f32", 0.1, E)
        bias = _bias(E, E + 1)
        out = rng.random(E) < part
        for far in (np.full(E, low), low * (1 - 0.1 * rng.random(E)), low + 0.3 * rng.normal(size=E)):
            b = np.where(out, np.maximum(far, np.finfo(np.float32).min), bias).astype(np.float32)
            for score, renorm in (("softmax", False), ("sigmoid", True)):
                check(s, k, score, b, groups, group_k, renorm, "f32")


@pytest.mark.parametrize("big", [1e6, 1e9, 3e10, 3.3e38])
def test_biases_that_swallow_the_scores(big):
    # keys in 64 bits lose the score's last bits, or all of them: ties then
    s = _scores(300, 32, "f32", 0.1, 5)
    bias = _bias(32, 6)
    for lift in (np.full(32, True), np.arange(32) % 3 == 0, np.arange(32) == 17):
        b = np.where(lift, np.float32(big) + bias, np.where(np.arange(32) % 2, -np.float32(big), bias)).astype(np.float32)
        for groups, group_k in ((1, 1), (8, 3)):
            for score, renorm in (("softmax", True), ("sigmoid", False)):
                check(s, 4, score, b, groups, group_k, renorm, "f32")


def test_sigmoids_that_fp32_cannot_hold():
    # all of a token's scores far below zero: renormalised weights are still in proportion
    s = _scores(64, 20, "f32", 0, 7, 2.0) - 150
    s[::2] += 110
    s = s.astype(np.float32).astype(np.float64)   # the reference has what the call has: shifted scores are rounded
    check(s, 4, "sigmoid", None, 1, 1, True, "f32")
    check(s, 4, "sigmoid", _bias(20, 8), 5, 3, True, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,group_k,masked,pad", SIZES)
def test_gradient_is_the_formulas(T, E, k, groups, group_k, masked, pad, dtype):
    s = _scores(T, E, dtype, masked, 3 * T + E)
    dw = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    for score, renorm in BOTH:
        expert, _, _, _, _, p = L.balanced(s, k, score, _bias(E, 3), groups, group_k, renorm, 1.0)
        buf = torch.full((max(T, 1), E + pad), 7.0, dtype=DT[dtype], device="cuda")
        d = buf[:T, :E]
        ws = ctr.workspace(ctr.ctr_expert_workspace_size())
        ctr.ctr_expert_route_balanced_bwd(torch.from_numpy(dw).cuda(), _on(s, dtype, pad), ctr.SCORES[score], renorm, 1.5,
                                          torch.from_numpy(expert).cuda(), d, ws)
        assert ctr.ctr_check_status(ws) == 0
        ref, mag = L.balanced_grad(dw.astype(np.float64), s, score, renorm, 1.5, expert, p)
        assert R.within(d.double().cpu().numpy(), ref, (2 * E + 40) * L.U * mag + 1e-37, dtype)
        assert bool((buf[:, E:] == 7.0).all())


def test_gradient_is_the_differences():
    # central differences of sum dweight weight in 64 bits, the choices held; third-order term below 1e-9
    T, E, k, h = 5, 12, 4, 1e-5
    s = _scores(T, E, "f32", 0.1, 21)
    dw = np.random.default_rng(2).normal(size=(T, k)).astype(np.float32)
    for score, renorm in BOTH:
        bias = _bias(E, 9)
        expert = L.balanced(s, k, score, bias, 3, 2, renorm, 1.5)[0]
        d = torch.empty((T, E), device="cuda")
        ctr.ctr_expert_route_balanced_bwd(torch.from_numpy(dw).cuda(), _on(s, "f32"), ctr.SCORES[score], renorm, 1.5,
                                          torch.from_numpy(expert).cuda(), d, ctr.workspace(256))
        got = d.double().cpu().numpy()
        for e in range(E):
            step = np.zeros((T, E))
            step[:, e] = h
            lo = L.balanced(s - step, k, score, bias, 3, 2, renorm, 1.5)
            hi = L.balanced(s + step, k, score, bias, 3, 2, renorm, 1.5)
            assert np.array_equal(lo[0], expert) and np.array_equal(hi[0], expert)
            diff = ((hi[1] - lo[1]) * dw).sum(axis=1) / (2 * h)
            assert np.all(np.abs(got[:, e] - diff) <= 1e-8 + (2 * E + 40) * L.U * 6 * np.abs(dw).sum(axis=1))


def test_without_balance_it_is_the_routing_that_was():
    # softmax, no bias, no groups: the same maps and gradient as ctr_expert_route's, bit for bit but for the weights' order of sums
    s = _scores(2000, 64, "bf16", 0.05, 11)
    x = _on(s, "bf16")
    i32 = dict(dtype=torch.int32, device="cuda")

    def outs():
        return [torch.empty((2000, 4), **i32), torch.empty((2000, 4), device="cuda"), torch.empty((2000, 4), **i32),
                torch.empty((8000,), **i32), torch.empty((65,), **i32)]
    ws = ctr.workspace(ctr.ctr_expert_route_workspace_size(2000, 64, 4))
    for renorm in (False, True):
        a, b = outs(), outs()
        ctr.ctr_expert_route(x, 4, renorm, *a, ws)
        ctr.ctr_expert_route_balanced(x, 4, ctr.SCORE_SOFTMAX, None, 1, 1, renorm, 1.0, *b, ws)
        for i in (0, 2, 3, 4):
            assert torch.equal(a[i], b[i])
        assert float((a[1] - b[1]).abs().max()) <= 72 * L.U
        dw = torch.randn((2000, 4), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        da, db = torch.empty_like(x), torch.empty_like(x)
        ctr.ctr_expert_route_bwd(dw, x, renorm, a[0], da, ws)
        ctr.ctr_expert_route_balanced_bwd(dw, x, ctr.SCORE_SOFTMAX, renorm, 1.0, a[0], db, ws)
        assert torch.equal(da, db)
