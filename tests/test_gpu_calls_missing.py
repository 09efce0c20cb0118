"""A tensor that is missing is refused by name, whichever it is."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu

I32, U8 = torch.int32, torch.uint8


def _e(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _calls(T=8, E=4, k=2, d=16, n=32):
    """(call, its arguments, the optional ones' places)"""
    R, P = T * k, ctr.fp8_padded_rows(T * k, E)
    ws = ctr.workspace(1 << 20)
    i = lambda *s: _e(*s, dtype=I32)      # noqa: E731
    u = lambda *s: _e(*s, dtype=U8)       # noqa: E731
    return [
        (ctr.ctr_expert_route, [_e(T, E), k, True, i(T, k), _e(T, k), i(T, k), i(R), i(E + 1), ws], {1, 2}),
        (ctr.ctr_expert_route_bwd, [_e(T, k), _e(T, E), True, i(T, k), _e(T, E), ws], {2}),
        (ctr.ctr_expert_dispatch, [_e(T, d), i(T, k), i(R), _e(R, d), ws], set()),
        (ctr.ctr_expert_combine, [_e(R, d), i(T, k), _e(T, k), _e(T, d), ws], {2}),
        (ctr.ctr_expert_combine_bwd, [_e(T, d), _e(R, d), i(T, k), _e(T, k), i(R), _e(R, d), _e(T, k), ws], set()),
        (ctr.ctr_fp8_quantize_rows, [_e(R, d), u(R, 128), _e(1, R), ws, i(R)], {4}),
        (ctr.ctr_fp8_quantize_rows_cols, [_e(R, d), i(E + 1), u(R, 128), _e(1, R), u(d, P), _e(1, P // 128),
                                          ctr.FP8_COLS_BY_BLOCK, ws, i(R)], {6, 8}),
        (ctr.ctr_fp8_quantize_blocks, [_e(E, n, d), u(E, n, 128), _e(E, 1, 1), ws, u(E, d, 128), _e(E, 1, 1)], set()),
        (ctr.ctr_fp8_matmul, [u(R, 128), _e(1, R), u(E, n, 128), _e(E, 1, 1), i(E + 1), _e(R, n), ws], {4}),
        (ctr.ctr_fp8_matmul_wgrad, [u(n, P), _e(P // 128, n), u(d, P), _e(1, P // 128), i(E + 1), _e(E, n, d), ws, R], {7}),
    ]


def test_missing_tensors_are_refused():
    for call, args, optional in _calls():
        call(*args)
        call(*args, stream=torch.cuda.current_stream())
        for at in range(len(args)):
            if at in optional:
                continue
            for other in (None, 3, args[at].cpu()):
                with pytest.raises(ValueError):
                    call(*args[:at], other, *args[at + 1:])
