"""The calls of the layers around the experts as a program makes them: both readers of their arguments (csrc/calls.cpp and
ctr.py) state the same rules, and what is missing, on another device or no workspace is refused."""
import random

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu

I32, U8, F32 = torch.int32, torch.uint8, torch.float32
EPS = 1e-6


def _z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _log(rng, lo, hi):
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))


def _case(seed):
    """(name, arguments, places that may be None) of every call, in both readers' order."""
    rng = random.Random(seed)
    dt = rng.choice([torch.float32, torch.bfloat16])
    T, k, n, E = _log(rng, 1, 600), _log(rng, 1, 300), _log(rng, 1, 300), 4 * _log(rng, 1, 20)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    ws = ctr.workspace(max(ctr.ctr_dense_workspace_size(T, n, k, dt, True, packed=True), ctr.ctr_rms_norm_workspace_size(T, k),
                           ctr.ctr_expert_route_workspace_size(T, E, 4)))
    grad = rng.choice([dt, F32])
    act = rng.choice(list(ctr.ACTIVATIONS.values()))
    choices = rng.randint(1, 4)
    i = lambda *s: _z(*s, dtype=I32)   # noqa: E731
    scores, expert = draw(T, E), i(T, choices)
    score, renorm = rng.choice([0, 1]), rng.random() < 0.5
    codes = [_z(T, ctr.fp8_padded(k), dtype=U8), _z(ctr.fp8_blocks(k), T)]
    return [("dense", [draw(T, k), draw(n, k), draw(n), act, draw(T, n), _z(T, n, dtype=dt), _z(T, n, dtype=dt), ws], {2, 4, 6}),
            ("dense", [draw(T, k), draw(n, k), None, act, None, _z(T, n, dtype=dt), None, ws], {2, 4, 6}),
            ("dense_bwd", [draw(T, n), draw(T, k), draw(n, k), draw(T, n), act, _z(T, k, dtype=dt), _z(n, k, dtype=grad),
                           _z(n, dtype=grad), ws], {3, 5, 6, 7} if act == 0 else {5, 6, 7}),
            ("rms_norm", [draw(T, k), draw(T, k), draw(k, dtype=F32), EPS, _z(T, k, dtype=dt), _z(T, k, dtype=dt), *codes, ws],
             {1, 2, 4, 5}),
            ("rms_norm", [draw(T, k), None, None, EPS, None, _z(T, k, dtype=dt), None, None, ws], {1, 2, 4, 6, 7}),
            ("rms_norm_bwd", [draw(T, k), draw(T, k), draw(T, k), draw(k, dtype=F32), EPS, _z(T, k, dtype=dt), _z(k), ws],
             {1, 3, 6}),
            ("expert_route_balanced", [scores, choices, score, draw(E, dtype=F32), 4, 4, renorm, 1.5, expert, _z(T, choices),
                                       i(T, choices), i(T * choices), i(E + 1), ws], {3}),
            ("expert_route_balanced_bwd", [draw(T, choices, dtype=F32), scores, score, renorm, 1.5, expert, _z(T, E, dtype=dt),
                                           ws], set())]


def _general(name, args):
    return getattr(ctr, "ctr_" + name)(*args, stream=torch.cuda.current_stream())


def _bits(t):
    return t.view(U8) if t.is_floating_point() else t


@pytest.mark.parametrize("seed", range(30))
def test_both_give_the_same_over_drawn_sizes(seed):
    for name, args, _ in _case(seed):
        tensors = [a for a in args if isinstance(a, torch.Tensor)]
        before = [a.clone() for a in tensors[:-1]]   # but the workspace
        _general(name, args)
        ref = [a.clone() for a in tensors[:-1]]
        for a, b in zip(tensors[:-1], before):
            a.copy_(b)
        assert getattr(ctr._usual(), name)(*args) == 0, name
        for a, b in zip(tensors[:-1], ref):
            assert torch.equal(_bits(a), _bits(b)), name
        assert ctr.ctr_check_status(args[-1]) == 0


def _others(t):
    """What t must not be taken for: other types, one more or less in every direction, other layouts."""
    yield None
    yield 3
    yield t.cpu()
    yield t.to(torch.int64 if not t.is_floating_point() else torch.float64)
    yield t.to(torch.bfloat16 if t.dtype != torch.bfloat16 else torch.float32)
    yield t.unsqueeze(0)
    yield t.reshape(-1)
    for d in range(t.dim()):
        for m in (-1, 1):
            shape = list(t.shape)
            shape[d] += m
            yield torch.zeros(shape, dtype=t.dtype, device="cuda")
    if t.dim() > 1:
        wide = torch.zeros((*t.shape[:-1], t.shape[-1] + 3), dtype=t.dtype, device="cuda")[..., :t.shape[-1]]
        yield wide.copy_(t)
        yield t.transpose(-1, -2)


@pytest.mark.parametrize("seed", [1, 4, 7])
def test_what_one_refuses_the_other_does_not_run(seed):
    refused = 0
    for name, args, _ in _case(seed):
        for at, arg in enumerate(args):
            for other in _others(arg) if isinstance(arg, torch.Tensor) else ():
                changed = [*args[:at], other, *args[at + 1:]]
                st = getattr(ctr._usual(), name)(*changed)
                try:
                    _general(name, changed)
                except (ValueError, ctr.CtrError):
                    refused += 1
                    assert st != 0, (name, at, None if other is None else other)
    torch.cuda.synchronize()
    assert refused > 300


def test_missing_tensors_are_refused():
    for name, args, optional in _case(2):
        call = getattr(ctr, "ctr_" + name)
        for at, arg in enumerate(args):
            if not isinstance(arg, torch.Tensor):
                continue
            for other in ([] if at in optional else [None]) + [3, arg.cpu()]:
                with pytest.raises((ValueError, ctr.CtrError)):
                    call(*args[:at], other, *args[at + 1:])
    args = _case(2)[3][1]
    with pytest.raises(ValueError, match="go together"):
        ctr.ctr_rms_norm(*args[:6], None, *args[7:])


def test_tensors_of_another_device_are_refused(monkeypatch):
    cases = _case(5)
    for name, args, _ in cases:
        _general(name, args)
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)   # as far as the checks can see
    for name, args, _ in cases:
        with pytest.raises(ValueError, match="cuda:1"):
            getattr(ctr, "ctr_" + name)(*args, stream=here)


def test_only_bytes_on_the_device_are_a_workspace():
    wide = torch.zeros((1 << 20, 2), dtype=U8, device="cuda")
    for name, args, _ in _case(6):
        call = getattr(ctr, "ctr_" + name)
        for stream in (None, torch.cuda.current_stream()):
            for ws in (None, torch.zeros(1 << 20, dtype=U8), torch.zeros(1 << 20, dtype=I32, device="cuda"), wide[:, 0], 256):
                with pytest.raises(ValueError, match="ws"):
                    call(*args[:-1], ws, stream=stream)
            with pytest.raises(ctr.CtrError):
                call(*args[:-1], torch.zeros(128, dtype=U8, device="cuda"), stream=stream)


def test_calls_of_two_threads_at_once():
    import threading
    cases = [_case(s) for s in (11, 12)]
    for c in cases:
        for name, args, _ in c:
            getattr(ctr, "ctr_" + name)(*args)
    torch.cuda.synchronize()
    ref = [[[a.clone() for a in args[:-1] if isinstance(a, torch.Tensor)] for _, args, _ in c] for c in cases]

    def work(c):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                for name, args, _ in c:
                    getattr(ctr, "ctr_" + name)(*args)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for c, r in zip(cases, ref):
        for (name, args, _), tensors in zip(c, r):
            for a, b in zip([a for a in args[:-1] if isinstance(a, torch.Tensor)], tensors):
                assert torch.equal(_bits(a), _bits(b)), name
