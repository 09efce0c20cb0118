"""The expert layer's calls beside other Python threads."""
import threading
import time

import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_call_waits_for_the_launch_queue():
    T, d = 64, 64
    x, out = torch.ones((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    slot = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    token, ws = slot.view(-1), ctr.workspace(256)
    ctr.ctr_expert_dispatch(x, slot, token, out, ws)
    a = torch.randn((6144, 6144), device="cuda", dtype=torch.float64)
    b = torch.empty_like(a)
    torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    gaps, done = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now
    t = threading.Thread(target=tick)
    t.start()
    torch.mm(a, a, out=b)          # one kernel of some tenths of a second: the launch queue fills up behind it
    t1 = time.perf_counter()
    for _ in range(3000):
        ctr.ctr_expert_dispatch(x, slot, token, out, ws)
    t2 = time.perf_counter()
    torch.cuda.synchronize()
    done.set()
    t.join()
    assert t2 - t1 > 0.1, "the calls did not wait"
    assert max(gaps) < 0.5 * (t2 - t1), (max(gaps), t2 - t1)
