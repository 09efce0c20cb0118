"""Host-side checks of the expert layer's calls (CPU only): every case is refused before any CUDA call."""
import ctypes as C

import numpy as np
import pytest

import _experts_ref as R


@pytest.fixture(scope="module")
def lib():
    from sparse_embeddings_feature_gb300 import ctr
    return ctr.lib()


P = C.c_void_p(256)
BIG = 1 << 30


def test_route_refusals(lib):
    f = lib.ctr_expert_route

    def call(scores=P, dtype=0, tokens=10, experts=8, ld=8, k=2, expert=P, offsets=P, ws=P, size=BIG):
        return f(scores, dtype, tokens, experts, ld, k, 1, expert, P, P, P, offsets, ws, size, None)
    assert call(scores=None) == -1 and call(expert=None) == -1 and call(offsets=None) == -1
    assert call(dtype=2) == -1 and call(tokens=-1) == -1 and call(experts=0) == -1
    assert call(ld=7) == -1 and call(k=0) == -1 and call(k=9) == -1
    assert call(scores=C.c_void_p(258)) == -1                       # fp32 off its alignment
    assert call(experts=513, ld=513) == -2
    assert call(experts=64, ld=64, k=17) == -2
    assert call(tokens=1 << 31, k=2) == -2
    assert call(size=256) == -3 and call(ws=C.c_void_p(100)) == -3 and call(ws=None) == -3
    g = lib.ctr_expert_route_bwd
    assert g(P, P, 0, 10, 8, 8, 2, 1, None, P, 8, P, 256, None) == -1
    assert g(P, P, 0, 10, 8, 8, 2, 1, P, P, 7, P, 256, None) == -1
    assert g(P, P, 0, 10, 8, 8, 2, 1, P, P, 8, P, 255, None) == -3
    assert g(P, P, 0, 0, 8, 8, 2, 1, None, None, 8, P, 256, None) == 0


def test_row_refusals(lib):
    d = lib.ctr_expert_dispatch
    assert d(None, 0, 4, 8, 8, 2, P, P, P, 8, P, 256, None) == -1
    assert d(P, 0, 4, 8, 7, 2, P, P, P, 8, P, 256, None) == -1
    assert d(P, 0, 4, 8, 8, 2, P, P, P, 7, P, 256, None) == -1
    assert d(P, 0, 4, 0, 8, 2, P, P, P, 8, P, 256, None) == -1
    assert d(P, 0, 4, 8, 8, 17, P, P, P, 8, P, 256, None) == -2
    assert d(C.c_void_p(258), 0, 4, 8, 8, 2, P, P, P, 8, P, 256, None) == -1
    assert d(P, 0, 4, 8, 8, 2, P, P, P, 8, P, 100, None) == -3
    assert d(None, 0, 0, 8, 8, 2, None, None, None, 8, P, 256, None) == 0
    c = lib.ctr_expert_combine
    assert c(P, 1, 4, 8, 8, 2, None, None, P, 8, P, 256, None) == -1
    assert c(P, 5, 4, 8, 8, 2, P, None, P, 8, P, 256, None) == -1
    b = lib.ctr_expert_combine_bwd
    assert b(P, 0, 4, 8, 8, 2, P, 8, P, None, P, P, 8, P, P, 256, None) == -1


def test_code_and_product_refusals(lib):
    q = lib.ctr_fp8_quantize_rows
    assert q(P, 0, 4, 4, 0, 8, None, P, P, 4, P, 256, None) == -1
    assert q(P, 0, 4, 5, 8, 8, None, P, P, 5, P, 256, None) == -1      # more rows than x without a map
    assert q(P, 0, 4, 4, 8, 8, None, P, P, 3, P, 256, None) == -1
    assert q(P, 0, 4, 4, 8, 8, None, C.c_void_p(264), P, 4, P, 256, None) == -1  # codes off 16 bytes
    assert q(P, 0, 4, 4, 8, 8, None, P, P, 4, P, 64, None) == -3
    assert q(None, 0, 0, 0, 8, 8, None, None, None, 0, P, 256, None) == 0
    rc = lib.ctr_fp8_quantize_rows_cols
    assert rc(P, 0, 4, 4, 8, 8, None, None, 1, 0, P, P, 4, P, P, P, 256, None) == -1
    assert rc(P, 0, 4, 4, 8, 8, None, P, 1, 2, P, P, 4, P, P, P, 256, None) == -1
    assert rc(P, 0, 4, 4, 8, 8, None, P, 513, 0, P, P, 4, P, P, P, 256, None) == -2
    bl = lib.ctr_fp8_quantize_blocks
    assert bl(P, 0, 1, 8, 8, P, P, P, None, P, 256, None) == -1
    assert bl(P, 0, 0, 8, 8, P, P, None, None, P, 256, None) == -1
    m = lib.ctr_fp8_matmul

    def mm(a=P, lds=4, offsets=P, rows=4, groups=2, n=8, k=8, out=P, dt=0, ldo=8, size=BIG):
        return m(a, P, lds, P, P, offsets, rows, groups, n, k, out, dt, ldo, P, size, None)
    assert mm(a=None) == -1 and mm(a=C.c_void_p(264)) == -1 and mm(out=None) == -1 and mm(dt=3) == -1
    assert mm(lds=3) == -1 and mm(ldo=7) == -1 and mm(offsets=None) == -1 and mm(n=0) == -1
    assert mm(groups=513) == -2 and mm(n=1 << 31) == -2 and mm(size=0) == -3
    w = lib.ctr_fp8_matmul_wgrad
    assert w(P, P, P, P, None, 4, 1, 8, 8, P, 0, P, BIG, None) == -1
    assert w(P, P, P, P, P, -1, 1, 8, 8, P, 0, P, BIG, None) == -1
    assert w(P, P, P, P, P, 4, 1, 8, 8, None, 0, P, BIG, None) == -1


def test_clip_refusals(lib):
    f = lib.ctr_clip_grads
    ptr, bad = (C.c_void_p * 1)(256), (C.c_void_p * 1)(258)
    dt, n = (C.c_int32 * 1)(0), (C.c_int64 * 1)(4)
    need = lib.ctr_clip_grads_workspace_size()
    assert f(ptr, ptr, dt, n, 1, C.c_float(1), None, P, need, None) == -1
    assert f(None, None, dt, n, 1, C.c_float(1), P, P, need, None) == -1
    assert f(bad, None, dt, n, 1, C.c_float(1), P, P, need, None) == -1
    assert f(ptr, bad, dt, n, 1, C.c_float(1), P, P, need, None) == -1
    assert f(ptr, None, (C.c_int32 * 1)(9), n, 1, C.c_float(1), P, P, need, None) == -1
    assert f(ptr, None, dt, (C.c_int64 * 1)(-4), 1, C.c_float(1), P, P, need, None) == -1
    assert f(ptr, None, dt, n, 1, C.c_float(-1), P, P, need, None) == -1
    assert f(ptr, None, dt, n, 1, C.c_float(float("nan")), P, P, need, None) == -1
    assert f(ptr, None, dt, n, 1, C.c_float(1), P, P, need - 1, None) == -3


def test_padded_rows_cover_every_grouping(lib):
    from sparse_embeddings_feature_gb300 import ctr
    rng = np.random.default_rng(0)
    for _ in range(300):
        counts = rng.integers(0, rng.choice([2, 130, 1000]), size=rng.integers(1, 20))
        rows = int(counts.sum()) + int(rng.integers(0, 3))
        need = 128 * int((-(-counts // 128)).sum())
        padded = ctr.fp8_padded_rows(rows, len(counts))
        assert padded % 128 == 0 and need <= padded <= max(128, rows + 127 * len(counts))
        back = ctr._rows_of_padding(padded, len(counts))
        assert back >= rows and ctr.fp8_padded_rows(back, len(counts)) == padded
        assert ctr.fp8_padded_rows(back + 1, len(counts)) > padded


def test_plain_forms_agree_with_their_definitions():
    # the reference rounding against a search over all code values
    codes = R.e4m3_values(np.arange(256, dtype=np.uint8))
    grid = np.unique(codes[np.isfinite(codes)])
    v = np.random.default_rng(1).normal(size=2000) * np.exp(np.random.default_rng(2).normal(size=2000) * 4)
    v = np.clip(v, -448, 448)
    near = np.abs(grid[None] - v[:, None]).min(axis=1)
    np.testing.assert_allclose(np.abs(R.e4m3_round(v) - v), near, rtol=0, atol=1e-12)
    expert, weight, slot, token, offsets, _ = R.route(np.array([[1.0, 3.0, 3.0], [-np.inf] * 3, [0.0, -np.inf, 5.0]]),
                                                      2, True)
    assert expert.tolist() == [[1, 2], [-1, -1], [2, 0]]
    assert slot.tolist() == [[1, 2], [-1, -1], [3, 0]] and token.tolist() == [2, 0, 0, 2, -1, -1]
    assert offsets.tolist() == [0, 1, 2, 4] and weight[0].tolist() == [0.5, 0.5]
