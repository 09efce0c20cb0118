"""The expert layer's calls launch on the current device and refuse tensors of another one, and workspaces that are
no dense bytes on it."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu

I32, U8 = torch.int32, torch.uint8


def _e(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _calls(T=8, E=4, k=2, d=16, n=32):
    """Every call of the layer with arguments that it takes, on the stream given."""
    R, P = T * k, ctr.fp8_padded_rows(T * k, E)
    ws = ctr.workspace(max(ctr.ctr_expert_route_workspace_size(T, E, k), ctr.ctr_clip_grads_workspace_size(),
                           ctr.ctr_fp8_matmul_workspace_size(R, E, n, d)))
    scores, x, rows = torch.randn((T, E), device="cuda"), torch.randn((T, d), device="cuda"), _e(R, d)
    expert, weight, slot, token, off = _e(T, k, dtype=I32), _e(T, k), _e(T, k, dtype=I32), _e(R, dtype=I32), \
        _e(E + 1, dtype=I32)
    q, s, w, wq, wsc = _e(R, 128, dtype=U8), _e(1, R), _e(E, n, d), _e(E, n, 128, dtype=U8), _e(E, 1, 1)
    qc, sc, dc, dsc = _e(d, P, dtype=U8), _e(1, P // 128), _e(n, P, dtype=U8), _e(P // 128, n)
    g = [torch.randn(100, device="cuda")]
    return {
        "route": lambda z, ws=ws: ctr.ctr_expert_route(scores, k, True, expert, weight, slot, token, off, ws, stream=z),
        "route_bwd": lambda z, ws=ws: ctr.ctr_expert_route_bwd(weight, scores, True, expert, _e(T, E), ws, stream=z),
        "dispatch": lambda z, ws=ws: ctr.ctr_expert_dispatch(x, slot, token, rows, ws, stream=z),
        "combine": lambda z, ws=ws: ctr.ctr_expert_combine(rows, slot, weight, _e(T, d), ws, stream=z),
        "combine_bwd": lambda z, ws=ws: ctr.ctr_expert_combine_bwd(x, rows, slot, weight, token, _e(R, d), _e(T, k), ws,
                                                                   stream=z),
        "rows": lambda z, ws=ws: ctr.ctr_fp8_quantize_rows(x, q, s, ws, row_index=token, stream=z),
        "rows_cols": lambda z, ws=ws: ctr.ctr_fp8_quantize_rows_cols(x, off, q, s, qc, sc, ctr.FP8_COLS_BY_BLOCK, ws,
                                                                     row_index=token, stream=z),
        "blocks": lambda z, ws=ws: ctr.ctr_fp8_quantize_blocks(w, wq, wsc, ws, stream=z),
        "matmul": lambda z, ws=ws: ctr.ctr_fp8_matmul(q, s, wq, wsc, off, _e(R, n), ws, stream=z),
        "wgrad": lambda z, ws=ws: ctr.ctr_fp8_matmul_wgrad(dc, dsc, qc, sc, off, _e(E, n, d), ws, rows=R, stream=z),
        "clip": lambda z, ws=ws: ctr.ctr_clip_grads(ctr.grad_list(g, g), 0.5, _e(1), ws, stream=z),
    }


NAMES = ["route", "route_bwd", "dispatch", "combine", "combine_bwd", "rows", "rows_cols", "blocks", "matmul", "wgrad", "clip"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    # with one GPU, another device is current as far as the checks can see
    calls, here = _calls(), torch.cuda.current_stream()
    for first in ("route", "rows_cols", "blocks", name):
        calls[first](None)
        calls[first](here)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        calls[name](here)


@pytest.mark.parametrize("name", NAMES)
def test_only_bytes_on_the_device_are_a_workspace(name):
    calls = _calls()
    wide = torch.zeros((1 << 20, 2), dtype=U8, device="cuda")
    bad = (None, torch.zeros(1 << 20, dtype=U8), torch.zeros(1 << 20, dtype=I32, device="cuda"), wide[:, 0],
           ctr.ctr_expert_workspace_size())
    for stream in (None, torch.cuda.current_stream()):
        for ws in bad:
            with pytest.raises(ValueError, match="ws"):
                calls[name](stream, ws)
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(ctr.CtrError):
            calls[name](stream, torch.zeros(128, dtype=U8, device="cuda"))
