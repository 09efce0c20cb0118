"""Norms of two widths called from two threads at once."""
import threading

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

from test_gpu_norm import EPS

pytestmark = pytest.mark.gpu


def test_gradients_of_two_widths_from_two_threads():
    # both widths want more shared memory than a kernel has without asking, one more than the other
    widths, rows = (16384, 12800), 64
    wrong, start = [], threading.Barrier(2)

    def work(d):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                g = torch.Generator(device="cuda").manual_seed(d)
                s, dy = (torch.randn((rows, d), generator=g, device="cuda") for _ in range(2))
                dx, dg = torch.empty_like(s), torch.empty(d, device="cuda")
                ws = ctr.workspace(ctr.ctr_rms_norm_workspace_size(rows, d))
                stream.synchronize()
                start.wait(timeout=60)
                for _ in range(400):
                    ctr.ctr_rms_norm_bwd(dy, None, s, None, EPS, dx, dg, ws)
                stream.synchronize()
                ref = (dy.double() * s.double() / torch.sqrt(s.double().square().mean(1, keepdim=True) + EPS)).sum(0)
                if not bool(((dg.double() - ref).abs() <= 1e-3).all()):
                    wrong.append((d, "dgamma"))
        except Exception as e:   # noqa: BLE001
            wrong.append((d, repr(e)))
    threads = [threading.Thread(target=work, args=(d,)) for d in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
