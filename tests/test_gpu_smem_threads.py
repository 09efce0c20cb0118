"""Calls whose kernels ask for shared memory by their sizes, made with two sizes from two threads at once."""
import threading

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu


def _both(make, sizes, calls=400):
    """make(size) gives a call and a check; every thread repeats its own."""
    wrong, start = [], threading.Barrier(len(sizes))

    def work(size):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                call, check = make(size)
                call()
                stream.synchronize()
                start.wait(timeout=120)
                for _ in range(calls):
                    call()
                stream.synchronize()
                if not check():
                    wrong.append((size, "result"))
        except Exception as e:   # noqa: BLE001
            wrong.append((size, repr(e)))
            start.abort()
    threads = [threading.Thread(target=work, args=(s,)) for s in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_interactions_of_three_sizes():
    def make(size):
        n, d = size
        x = torch.randn((64, n, d), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(torch.bfloat16)
        out = torch.empty((64, ctr.ctr_interaction_width(n, d, 0)), device="cuda", dtype=torch.bfloat16)
        ws = ctr.workspace(ctr.ctr_interaction_workspace_size())
        first = torch.empty_like(out)
        ctr.ctr_dot_interaction(x, n, d, first, ws)

        def check():
            return torch.equal(out, first) and ctr.ctr_check_status(ws) == 0
        return lambda: ctr.ctr_dot_interaction(x, n, d, out, ws), check
    _both(make, [(27, 256), (27, 128), (12, 256)])


def test_norm_gradients_of_three_widths():
    def make(d):
        g = torch.Generator(device="cuda").manual_seed(d)
        s, dy = (torch.randn((64, d), generator=g, device="cuda") for _ in range(2))
        dx, dg, first = torch.empty_like(s), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        ws = ctr.workspace(ctr.ctr_rms_norm_workspace_size(64, d))
        ctr.ctr_rms_norm_bwd(dy, None, s, None, 1e-6, dx, first, ws)
        return (lambda: ctr.ctr_rms_norm_bwd(dy, None, s, None, 1e-6, dx, dg, ws)), (lambda: torch.equal(dg, first))
    _both(make, [16384, 14000, 12800])
