"""Balanced routing at the ends of the score functions, where 64 bits still tell values apart."""
import numpy as np
import pytest

from test_gpu_balance import gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 3)])
def test_sigmoids_at_the_end_of_64_bits(groups, group_k):
    # down to e^-744 a score function's value is a number of its own: beside equal biases of zero the scores' order
    rng = np.random.default_rng(5)
    E, k = 32, 6
    s = np.stack([rng.permutation(-744.0 + 2.0 * np.arange(E)) for _ in range(200)])
    for score, top in (("sigmoid", None), ("softmax", 0.0)):
        t = s.copy()
        if top is not None:
            t[:, 5] = top   # a row's largest: the others' values are e^score over it
        per = E // groups
        best = t.reshape(200, groups, per).max(axis=2)   # at least e^2 above any other of a group: the larger sum
        stay = np.argsort(-best, axis=1, kind="stable")[:, :group_k]
        kept = np.zeros((200, groups), dtype=bool)
        np.put_along_axis(kept, stay, True, axis=1)
        want = np.argsort(-np.where(np.repeat(kept, per, axis=1), t, -np.inf), axis=1, kind="stable")[:, :k]
        for bias in (np.zeros(E, dtype=np.float32), None):
            st, got = gpu(t, k, score, bias, groups, group_k, False, 1.0, "f32")
            assert st == 0
            np.testing.assert_array_equal(got[0], want)
