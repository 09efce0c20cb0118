"""The two readers of the expert layer's arguments (csrc/calls.cpp and ctr.py) state the same rules: over drawn
sizes both give the same results, and what one refuses the other does not run."""
import random

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu

I32, U8, F32 = torch.int32, torch.uint8, torch.float32


def _z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _log(rng, lo, hi):
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))


def _case(seed):
    """(name, arguments) of every call, in both readers' order, on maps and codes that belong together."""
    rng = random.Random(seed)
    dt = rng.choice([torch.float32, torch.bfloat16])
    T, E, d, n = _log(rng, 1, 700), _log(rng, 1, 40), _log(rng, 1, 400), _log(rng, 1, 300)
    k = rng.randint(1, min(E, 4))
    R, kb, nb, P = T * k, ctr.fp8_blocks(d), ctr.fp8_blocks(n), ctr.fp8_padded_rows(T * k, E)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    ws = ctr.workspace(max(ctr.ctr_expert_route_workspace_size(T, E, k), ctr.ctr_clip_grads_workspace_size(),
                           ctr.ctr_fp8_matmul_workspace_size(R, E, n, d)))
    scores, x, w, dy, y, dw = draw(T, E), draw(T, d), draw(E, n, d), draw(R, n), draw(T, d), draw(T, k, dtype=F32)
    expert, weight, slot, token, off = (_z(T, k, dtype=I32), _z(T, k), _z(T, k, dtype=I32), _z(R, dtype=I32),
                                        _z(E + 1, dtype=I32))
    xs, q, s, qc, sc = _z(R, d, dtype=dt), _z(R, kb * 128, dtype=U8), _z(kb, R), _z(d, P, dtype=U8), _z(kb, P // 128)
    dq, ds, dc, dsc = _z(R, nb * 128, dtype=U8), _z(nb, R), _z(n, P, dtype=U8), _z(P // 128, n)
    wq, wsc, wt, wts = _z(E, n, kb * 128, dtype=U8), _z(E, nb, kb), _z(E, d, nb * 128, dtype=U8), _z(E, kb, nb)
    renorm, out = rng.random() < 0.5, rng.choice([torch.float32, torch.bfloat16])
    rows = rng.choice([R, None])
    return [("expert_route", [scores, k, renorm, expert, weight, slot, token, off, ws]),
            ("expert_route_bwd", [dw, scores, renorm, expert, _z(T, E, dtype=dt), ws]),
            ("expert_dispatch", [x, slot, token, xs, ws]),
            ("expert_combine", [xs, slot, rng.choice([weight, None]), _z(T, d, dtype=dt), ws]),
            ("expert_combine_bwd", [y, xs, slot, weight, token, _z(R, d, dtype=dt), _z(T, k), ws]),
            ("fp8_quantize_rows", [x, q.clone(), s.clone(), ws, token]),
            ("fp8_quantize_rows_cols", [x, off, q, s, qc, sc, ctr.FP8_COLS_BY_BLOCK, ws, token]),
            ("fp8_quantize_rows_cols", [dy, off, dq, ds, dc, dsc, ctr.FP8_COLS_BY_COLUMN, ws, None]),
            ("fp8_quantize_blocks", [w, wq, wsc, ws, wt, wts]),
            ("fp8_quantize_blocks", [w, wq.clone(), wsc.clone(), ws, None, None]),
            ("fp8_matmul", [q, s, wq, wsc, off, _z(R, n, dtype=out), ws]),
            ("fp8_matmul_wgrad", [dc, dsc, qc, sc, off, _z(E, n, d, dtype=out), ws, rows])]


def _general(name, args):
    return getattr(ctr, "ctr_" + name)(*args, stream=torch.cuda.current_stream())


def _tensors(args):
    return [a for a in args if isinstance(a, torch.Tensor)]


@pytest.mark.parametrize("seed", range(30))
def test_both_give_the_same_over_drawn_sizes(seed):
    for name, args in _case(seed):
        _general(name, args)
        ref = [a.clone() for a in _tensors(args)]
        assert getattr(ctr._usual(), name)(*args) == 0, name
        for a, b in zip(_tensors(args), ref):
            assert torch.equal(a.view(U8) if a.is_floating_point() else a, b.view(U8) if b.is_floating_point() else b), name
        ws = next(a for a in args if isinstance(a, torch.Tensor) and a.dtype == U8 and a.dim() == 1)
        assert ctr.ctr_check_status(ws) == 0


def _others(t):
    """Tensors that t must not be taken for: other types, one more or less in every direction, other layouts."""
    yield None
    yield t.cpu()
    yield t.to(torch.int64 if not t.is_floating_point() else torch.float64)
    yield t.to(torch.bfloat16 if t.dtype != torch.bfloat16 else torch.float32)
    yield t.unsqueeze(0)
    yield t.reshape(-1)
    for i in range(t.dim()):
        for m in (-1, 1):
            shape = list(t.shape)
            shape[i] += m
            yield torch.zeros(shape, dtype=t.dtype, device="cuda")
    if t.dim() > 1:
        wide = torch.zeros((*t.shape[:-1], t.shape[-1] + 3), dtype=t.dtype, device="cuda")[..., :t.shape[-1]]
        yield wide.copy_(t)
        yield t.transpose(-1, -2)


@pytest.mark.parametrize("seed", [1, 4, 7, 11])
def test_what_one_refuses_the_other_does_not_run(seed):
    refused = 0
    for name, args in _case(seed):
        for at, arg in enumerate(args):
            for other in _others(arg) if isinstance(arg, torch.Tensor) else ():
                changed = [*args[:at], other, *args[at + 1:]]
                st = getattr(ctr._usual(), name)(*changed)
                try:
                    _general(name, changed)
                except (ValueError, ctr.CtrError):
                    refused += 1
                    assert st != 0, (name, at, None if other is None else tuple(other.shape))
    torch.cuda.synchronize()
    assert refused > 300
