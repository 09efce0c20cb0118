"""The expert layer's calls in their usual layouts (csrc/calls.cpp) against the same calls through the
general binding, which takes strided rows, other streams, and refusals."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

I32, F32, U8 = torch.int32, torch.float32, torch.uint8


def _e(*shape, dtype=F32):  # zeros: column codes past the last group's rows are nobody's, and not written
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_both_ways_give_the_same(dtype):
    T, E, k, d, n = 300, 12, 2, 96, 160
    g = torch.Generator(device="cuda").manual_seed(1)
    scores, x = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((T, E), (T, d)))
    w, dy = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((E, n, d), (T * k, n)))
    dwt = torch.randn((T, k), generator=g, device="cuda")
    ws = ctr.workspace(max(ctr.ctr_expert_route_workspace_size(T, E, k), ctr.ctr_clip_grads_workspace_size(),
                           ctr.ctr_fp8_matmul_workspace_size(T * k, E, n, d)))
    kb, nb, P = ctr.fp8_blocks(d), ctr.fp8_blocks(n), ctr.fp8_padded_rows(T * k, E)

    def steps(stream):
        o = {"expert": _e(T, k, dtype=I32), "weight": _e(T, k), "slot": _e(T, k, dtype=I32),
             "token": _e(T * k, dtype=I32), "offsets": _e(E + 1, dtype=I32), "ds": _e(T, E, dtype=dtype),
             "xs": _e(T * k, d, dtype=dtype), "y": _e(T, d, dtype=dtype), "dr": _e(T * k, d, dtype=dtype),
             "dw": _e(T, k), "q": _e(T * k, kb * 128, dtype=U8), "s": _e(kb, T * k), "qc": _e(d, P, dtype=U8),
             "sc": _e(kb, P // 128), "dq": _e(T * k, nb * 128, dtype=U8), "dqs": _e(nb, T * k),
             "dc": _e(n, P, dtype=U8), "dcs": _e(P // 128, n), "r": _e(T * k, kb * 128, dtype=U8), "rs": _e(kb, T * k),
             "wq": _e(E, n, kb * 128, dtype=U8), "wsc": _e(E, nb, kb), "wt": _e(E, d, nb * 128, dtype=U8),
             "wts": _e(E, kb, nb), "p": _e(T * k, n), "g": _e(E, n, d), "norm": _e(1), "clip": _e(E, n, d)}
        z = dict(stream=stream)
        ctr.ctr_expert_route(scores, k, True, o["expert"], o["weight"], o["slot"], o["token"], o["offsets"], ws, **z)
        ctr.ctr_expert_route_bwd(dwt, scores, True, o["expert"], o["ds"], ws, **z)
        ctr.ctr_expert_dispatch(x, o["slot"], o["token"], o["xs"], ws, **z)
        ctr.ctr_expert_combine(o["xs"], o["slot"], o["weight"], o["y"], ws, **z)
        ctr.ctr_expert_combine_bwd(x, o["xs"], o["slot"], o["weight"], o["token"], o["dr"], o["dw"], ws, **z)
        ctr.ctr_fp8_quantize_rows(x, o["r"], o["rs"], ws, row_index=o["token"], **z)
        ctr.ctr_fp8_quantize_rows_cols(x, o["offsets"], o["q"], o["s"], o["qc"], o["sc"], ctr.FP8_COLS_BY_BLOCK, ws,
                                       row_index=o["token"], **z)
        ctr.ctr_fp8_quantize_rows_cols(dy, o["offsets"], o["dq"], o["dqs"], o["dc"], o["dcs"], ctr.FP8_COLS_BY_COLUMN,
                                       ws, **z)
        ctr.ctr_fp8_quantize_blocks(w, o["wq"], o["wsc"], ws, o["wt"], o["wts"], **z)
        ctr.ctr_fp8_matmul(o["q"], o["s"], o["wq"], o["wsc"], o["offsets"], o["p"], ws, **z)
        ctr.ctr_fp8_matmul_wgrad(o["dc"], o["dcs"], o["qc"], o["sc"], o["offsets"], o["g"], ws, rows=T * k, **z)
        ctr.ctr_clip_grads(ctr.grad_list([o["g"]], [o["clip"]]), 0.5, o["norm"], ws, **z)
        torch.cuda.synchronize()
        assert ctr.ctr_check_status(ws) == 0
        return o
    a, b = steps(None), steps(torch.cuda.current_stream())
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.gpu
def test_other_layouts_are_not_taken():
    calls, ws = ctr._usual(), ctr.workspace(256)
    x, slot, token, out = torch.ones((4, 8), device="cuda"), torch.zeros((4, 1), dtype=I32, device="cuda"), \
        torch.arange(4, dtype=I32, device="cuda"), _e(4, 8)
    slot[:, 0] = token
    assert calls.expert_dispatch(x, slot, token, out, ws) == 0
    assert torch.equal(out, x)
    wide = torch.ones((4, 16), device="cuda")[:, :8]
    for args in ((wide, slot, token, out, ws), (x, slot.long(), token, out, ws), (x, slot, token[:3], out, ws),
                 (x, slot, token, out.bfloat16(), ws), (x, slot, token, _e(4, 9), ws), (x, slot, token, out.cpu(), ws),
                 (x, slot, token, out, ws.int()), (x.double(), slot, token, out, ws), (x, None, token, out, ws),
                 (x, slot, token, out), (x, slot, token, out, ws, 1)):
        assert calls.expert_dispatch(*args) is None
    assert calls.expert_dispatch(x, slot, token, out, ws[:128]) == ctr.ERR_WORKSPACE


def test_no_tensors_are_not_taken():
    calls = ctr._usual()
    for name, n in (("expert_route", 9), ("expert_route_bwd", 6), ("expert_dispatch", 5), ("expert_combine", 5),
                    ("expert_combine_bwd", 8), ("fp8_quantize_rows", 5), ("fp8_quantize_rows_cols", 9),
                    ("fp8_quantize_blocks", 6), ("fp8_matmul", 7), ("fp8_matmul_wgrad", 8), ("clip_grads", 8)):
        f = getattr(calls, name)
        assert f(*[None] * n) is None and f(*[torch.zeros(2, 2)] * n) is None and f() is None and f(*[1.5] * n) is None
