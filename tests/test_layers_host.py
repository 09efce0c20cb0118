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
