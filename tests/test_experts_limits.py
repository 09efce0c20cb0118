"""Sizes at the ends of the expert layer's index types (CPU only: refused before any CUDA call)."""
import ctypes as C

import pytest

P = C.c_void_p(256)
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    from sparse_embeddings_feature_gb300 import ctr
    return ctr.lib()


@pytest.mark.parametrize("rows", [TOP, TOP - 126, TOP - 65535])
def test_rows_whose_tiles_leave_32_bits(lib, rows):
    # tiles are counted as (rows of a group + 127) / 128 and (+ 255) / 256 in 32 bits
    rc = lib.ctr_fp8_quantize_rows_cols(P, 0, rows, rows, 1, 1, None, P, 1, 0, P, P, rows, P, P, P, 256, None)
    mm = lib.ctr_fp8_matmul(P, P, rows, P, P, P, rows, 1, 8, 8, P, 0, 8, P, 1 << 40, None)
    wg = lib.ctr_fp8_matmul_wgrad(P, P, P, P, P, rows, 1, 8, 8, P, 0, P, 1 << 40, None)
    assert (rc, mm, wg) == (-2, -2, -2)
