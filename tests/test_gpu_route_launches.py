"""Routing of mid-sized batches gives the same with and without thread-block clusters."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

pytestmark = pytest.mark.gpu


def _route(s, k, renorm):
    T, E = s.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = [torch.full((T, k), -9, **i32), torch.full((T, k), -9.0, device="cuda"), torch.full((T, k), -9, **i32),
         torch.full((T * k,), -9, **i32), torch.full((E + 1,), -9, **i32)]
    ws = ctr.workspace(ctr.ctr_expert_route_workspace_size(T, E, k))
    before = ctr.ctr_launch_count()
    ctr.ctr_expert_route(s, k, renorm, *o, ws)
    assert ctr.ctr_check_status(ws) == 0
    return o, ctr.ctr_launch_count() - before


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(33, 512, 4), (257, 8, 2), (600, 26, 4), (2048, 26, 4), (4096, 64, 8), (4096, 512, 16)])
def test_three_launches_give_what_a_cluster_gives(T, E, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    s = torch.randn((T, E), generator=g, device="cuda").to(dtype)
    s[torch.rand((T, E), generator=g, device="cuda") < 0.1] = -float("inf")
    s[::9] = -float("inf")
    prev = ctr.ctr_set_route_cluster(False)
    try:
        assert prev
        for renorm in (True, False):
            ctr.ctr_set_route_cluster(True)
            a, one = _route(s, k, renorm)
            ctr.ctr_set_route_cluster(False)
            b, three = _route(s, k, renorm)
            assert (one, three) == (1, 3)
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    finally:
        ctr.ctr_set_route_cluster(True)
