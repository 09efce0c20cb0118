"""Host-side checks of the layers around the experts (CPU only): every case is refused before any CUDA call."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_embeddings_feature_gb300 import ctr
    return ctr.lib()


P = C.c_void_p(256)
ODD = C.c_void_p(258)


def test_norm_refusals(lib):
    def call(x=P, dt=0, rows=4, d=8, ldx=8, r=None, ldr=8, gamma=P, eps=1e-6, s=None, lds=8, y=P, ldy=8, q=None, scale=None,
             ldc=4, ws=P, size=256):
        return lib.ctr_rms_norm(x, dt, rows, d, ldx, r, ldr, gamma, C.c_float(eps), s, lds, y, ldy, q, scale, ldc, ws,
                                size, None)
    assert call(x=None) == -1 and call(dt=2) == -1 and call(rows=-1) == -1 and call(d=0) == -1 and call(ldx=7) == -1
    assert call(r=P, ldr=7) == -1 and call(s=P, lds=7) == -1 and call(ldy=7) == -1
    assert call(x=ODD) == -1 and call(r=ODD) == -1 and call(s=ODD) == -1 and call(y=ODD) == -1 and call(gamma=ODD) == -1
    assert call(eps=0.0) == -1 and call(eps=-1.0) == -1 and call(eps=float("nan")) == -1 and call(eps=float("inf")) == -1
    assert call(y=None) == -1 and call(q=P) == -1 and call(scale=P) == -1
    assert call(q=C.c_void_p(264), scale=P) == -1 and call(q=P, scale=P, ldc=3) == -1
    assert call(d=16385, ldx=16385, ldy=16385) == -2 and call(rows=1 << 31) == -2
    assert call(size=255) == -3 and call(ws=C.c_void_p(100)) == -3 and call(ws=None) == -3
    assert call(rows=0, x=None, y=None) == 0

    def back(dy=P, dt=0, rows=4, d=8, ld=8, ds=None, ldd=8, s=P, lds=8, gamma=P, eps=1e-6, dx=P, ldx=8, dg=P, size=1 << 20):
        return lib.ctr_rms_norm_bwd(dy, dt, rows, d, ld, ds, ldd, s, lds, gamma, C.c_float(eps), dx, ldx, dg, P, size, None)
    assert back(dy=None) == -1 and back(s=None) == -1 and back(dx=None) == -1 and back(dt=9) == -1 and back(d=0) == -1
    assert back(ld=7) == -1 and back(ds=P, ldd=7) == -1 and back(lds=7) == -1 and back(ldx=7) == -1 and back(eps=0.0) == -1
    assert back(dy=ODD) == -1 and back(ds=ODD) == -1 and back(s=ODD) == -1 and back(dx=ODD) == -1 and back(dg=ODD) == -1
    assert back(size=256) == -3 and back(dg=None, size=255) == -3
    assert lib.ctr_rms_norm_workspace_size(-1, 8) == 0 and lib.ctr_rms_norm_workspace_size(4, 16385) == 0


def test_dense_refusals(lib):
    big = 1 << 30

    def call(x=P, dt=1, rows=40, k=16, ldx=16, w=P, n=24, ldw=16, bias=None, act=0, r=None, ldr=24, y=P, ldy=24, pre=None,
             ldp=24, ws=P, size=big):
        return lib.ctr_dense(x, dt, rows, k, ldx, w, n, ldw, bias, act, r, ldr, y, ldy, pre, ldp, ws, size, None)
    assert call(x=None) == -1 and call(w=None) == -1 and call(y=None) == -1 and call(dt=2) == -1 and call(rows=-1) == -1
    assert call(k=0) == -1 and call(n=0) == -1 and call(act=5) == -1 and call(act=-1) == -1
    assert call(ldx=15) == -1 and call(ldw=15) == -1 and call(ldy=23) == -1
    assert call(r=P, ldr=23) == -1 and call(pre=P, ldp=23) == -1
    odd = C.c_void_p(257)
    for name in ("x", "w", "bias", "r", "y", "pre"):
        assert call(**{name: odd}) == -1, name
        assert call(dt=0, **{name: ODD}) == -1, name
    assert call(rows=1 << 31) == -2 and call(n=1 << 30, ldy=1 << 30) == -2 and call(k=1 << 30, ldx=1 << 30, ldw=1 << 30) == -2
    assert call(size=100) == -3 and call(ws=None) == -3 and call(ws=C.c_void_p(100)) == -3
    assert call(dt=0, size=256) == -3                                   # no room for the planes
    assert call(k=15, ldx=15, ldw=15, size=256) == -3                   # nor for rows off 16 bytes
    assert call(rows=0, x=None, y=None) == 0

    def back(dy=P, dt=1, rows=40, n=24, ld=24, x=P, k=16, ldx=16, w=P, ldw=16, pre=P, ldp=24, act=1, dx=P, ldd=16, gt=0, dw=P,
             ldg=16, db=P, ws=P, size=big):
        return lib.ctr_dense_bwd(dy, dt, rows, n, ld, x, k, ldx, w, ldw, pre, ldp, act, dx, ldd, gt, dw, ldg, db, ws, size, None)
    assert back(dy=None) == -1 and back(x=None) == -1 and back(w=None) == -1 and back(pre=None) == -1
    assert back(dt=0, gt=1) == -1 and back(gt=2) == -1 and back(act=9) == -1
    assert back(ld=23) == -1 and back(ldx=15) == -1 and back(ldw=15) == -1 and back(ldp=23) == -1 and back(ldd=15) == -1
    assert back(ldg=15) == -1
    for name in ("dy", "x", "w", "pre", "dx", "dw", "db"):
        assert back(**{name: odd}) == -1, name
    assert back(dw=ODD) == -1 and back(db=ODD) == -1                    # fp32 gradients of a bf16 layer
    assert back(size=256) == -3 and back(ws=None) == -3
    size = lib.ctr_dense_workspace_size
    assert size(-1, 24, 16, 0, 0, 0) == 0 and size(4, 0, 16, 0, 0, 0) == 0 and size(4, 24, 16, 7, 0, 0) == 0
    assert size(40, 24, 16, 1, 0, 0) == 256 and size(40, 24, 16, 1, 0, 1) > 256 and size(40, 24, 16, 0, 0, 0) > 256
    assert size(40, 24, 16, 1, 1, 0) < size(40, 24, 16, 0, 1, 0)


def test_dense_workspace_sizes_without_a_device(lib):
    size = lib.ctr_dense_workspace_size
    for n, k in ((1, 3), (128, 128), (264, 512), (1024, 1024), (4096, 300)):
        for dt in (0, 1):
            last = 0
            for rows in (0, 1, 9, 63, 511, 512, 1000, 4095, 4096, 29185, 65536, 100000):   # more rows never take less
                now = size(rows, n, k, dt, 1, 0)
                assert now >= max(last, 256)
                last = now
            assert last >= 100000 * n * (2 if dt else 6)   # dz


def test_balanced_routing_refusals(lib):
    def call(scores=P, dt=0, tokens=10, experts=8, ld=8, k=2, score=1, bias=P, groups=4, kept=2, factor=1.0, expert=P,
             offsets=P, size=1 << 30):
        return lib.ctr_expert_route_balanced(scores, dt, tokens, experts, ld, k, score, bias, groups, kept, 1,
                                             C.c_float(factor), expert, P, P, P, offsets, P, size, None)
    assert call(scores=None) == -1 and call(expert=None) == -1 and call(offsets=None) == -1 and call(dt=2) == -1
    assert call(score=2) == -1 and call(score=-1) == -1 and call(bias=ODD) == -1 and call(ld=7) == -1 and call(k=0) == -1
    assert call(groups=3) == -1 and call(groups=0) == -1 and call(kept=0) == -1 and call(kept=5) == -1
    assert call(k=5) == -1                                              # two groups of two hold four
    assert call(factor=float("nan")) == -1 and call(factor=float("inf")) == -1
    assert call(experts=66, ld=66, groups=33, kept=2) == -2 and call(experts=513, ld=513, groups=1, kept=1) == -2
    assert call(size=256) == -3

    def back(dw=P, scores=P, score=1, k=2, factor=1.0, expert=P, out=P, ldd=8, size=256, tokens=10):
        return lib.ctr_expert_route_balanced_bwd(dw, scores, 0, tokens, 8, 8, k, score, 1, C.c_float(factor), expert, out,
                                                 ldd, P, size, None)
    assert back(dw=None) == -1 and back(scores=None) == -1 and back(expert=None) == -1 and back(out=None) == -1
    assert back(score=2) == -1 and back(k=9) == -1 and back(factor=float("nan")) == -1 and back(ldd=7) == -1
    assert back(size=255) == -3 and back(tokens=0, dw=None, scores=None, expert=None, out=None) == 0
