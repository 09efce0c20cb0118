"""Balanced routing under biases of any spread: choices are those of 64-bit keys wherever the biases lie."""
import numpy as np
import pytest

import _layers_ref as L
from test_gpu_balance import BOTH, _bias, _scores, check

pytestmark = pytest.mark.gpu

LAYOUTS = [(8, 1, 1, 2), (16, 1, 1, 8), (32, 1, 1, 16), (32, 8, 3, 4), (64, 8, 4, 6), (256, 8, 4, 8), (256, 16, 3, 16),
           (130, 13, 5, 7), (512, 1, 1, 16)]


def test_two_neighbours_of_a_border():
    # keys 0.5, -5.88, -5.12, -5.6 ..: the score decides between biases 0.2 apart, far below the largest
    s = np.array([[0.0, -4, 4, 0, 0, 0, 0, 0]])
    b = np.array([0, -5.9] + [-6.1] * 6, dtype=np.float32)
    expert, _ = check(s, 2, "sigmoid", b, 1, 1, False, "f32")
    assert expert.tolist() == [[0, 2]]
    expert, _ = check(np.array([[0.0, -2, 2]]), 2, "sigmoid", np.array([0, -5.9, -6.1], dtype=np.float32), 1, 1, True, "f32")
    assert expert.tolist() == [[0, 2]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [4.0, 5.0, 5.9, 6.1, 7.0, 8.0, 12.0, 40.0, 300.0])
def test_biases_spread_evenly(width, dtype):
    rng = np.random.default_rng(int(10 * width))
    for E, groups, group_k, k in LAYOUTS:
        s = _scores(300, E, dtype, 0.1, E, 2.0)
        for b in (width * rng.random(E), width * np.arange(E) / E, width / 4 * rng.normal(size=E) - 100):
            for score, renorm in (("softmax", False), ("sigmoid", True)):
                check(s, k, score, b.astype(np.float32), groups, group_k, renorm, dtype)


@pytest.mark.parametrize("E,groups,group_k,k", LAYOUTS)
def test_steps_around_six_below_the_largest(E, groups, group_k, k):
    # one expert at 0, the others from -5 to -7 in steps of a tenth and from the top again
    s = _scores(400, E, "f32", 0.0, E, 3.0)
    b = (-5 - 0.1 * (np.arange(E) % 21)).astype(np.float32)
    for at in (0, E // 2, E - 1):
        one = b.copy()
        one[at] = 0
        for score, renorm in BOTH:
            check(s, k, score, one, groups, group_k, renorm, "f32")


@pytest.mark.parametrize("lift", [1.5, 6.5, 10.0, 1e3, 1e9, 2e9, 3e38])
def test_lifted_experts(lift):
    # a few experts above the rest; the rest is still chosen from by its own keys
    rng = np.random.default_rng(7)
    for E, groups, group_k, k in LAYOUTS:
        s = _scores(300, E, "f32", 0.05, E, 2.0)
        few = rng.random(E) < 0.1
        few[E // 3] = True
        for far in (np.full(E, lift), lift * (1 - 0.2 * rng.random(E))):
            b = np.where(few, far, _bias(E, E)).astype(np.float32)
            for score, renorm in (("softmax", True), ("sigmoid", False)):
                check(s, k, score, b, groups, group_k, renorm, "f32")


@pytest.mark.parametrize("gap", [0.9, 1.0, 1.0 + 2.0 ** -20, 1.05, 1.0625, 1.07, 1.5, 3.0, 1e4])
def test_steps_of_biases(gap):
    # equal biases in steps of about what a score can add, scores at both ends of their function among them
    for E, groups, group_k, k in LAYOUTS:
        s = _scores(200, E, "f32", 0.0, E, 30.0)
        s[::3] = _scores(67, E, "f32", 0.0, E, 1.0)
        b = (gap * (np.arange(E) * 7 % 11)).astype(np.float32)
        for score, renorm in (("softmax", True), ("sigmoid", False)):
            check(s, k, score, b, groups, group_k, renorm, "f32")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,group_k,k", [(16, 1, 1, 16), (24, 4, 2, 5), (64, 8, 4, 6), (256, 8, 4, 8)])
def test_keys_a_few_times_1e_8_apart_in_each_stretch(E, groups, group_k, k, score):
    # as where all keys lie together, a third of the experts 20 lower and a third 40 higher
    rng = np.random.default_rng(E)
    base = rng.normal(size=E).astype(np.float32).astype(np.float64)
    p = L.balanced(base[None], 1, score, None, 1, 1, False, 1.0)[5][0]
    bias = (0.9 - p + np.array([0, -20, 40])[np.arange(E) % 3]).astype(np.float32)
    s = np.repeat(base[None], 400, axis=0)
    if score == "sigmoid":   # a softmax's other values would move
        s[rng.random(s.shape) < 0.3] = -np.inf
    check(s, k, score, bias, groups, group_k, True, "f32")


def test_groups_sums_from_different_stretches():
    # groups of 4 whose two best keys add up to nearly the same: 10 + 0, 5 + 5, 7 + 3, 2 + 8, each group a few 2^-20 more
    rng = np.random.default_rng(3)
    E, groups = 64, 16
    pairs = [(10.0, 0.0), (5.0, 5.0), (7.0, 3.0), (8.0, 2.0)]
    for trial in range(6):
        b = np.full(E, -30.0)
        more = rng.permutation(groups) * 2.0 ** -20
        for g in range(groups):
            large, small = pairs[(g + trial) % 4]
            b[4 * g:4 * g + 2] = large + more[g], small
        b = b.astype(np.float32)
        two = rng.normal(size=(300, 2)).astype(np.float32).astype(np.float64)
        s = np.zeros((300, E))
        s[:, 0::4], s[:, 1::4], s[:, 2::4], s[:, 3::4] = two[:, :1], two[:, 1:], -1.0, 0.5
        for score, renorm in (("sigmoid", True), ("softmax", False)):
            check(s, 6, score, b, groups, 5, renorm, "f32")


def test_a_lifted_expert_alone_in_its_group():
    # the group has one key, others two; then all of them one
    rng = np.random.default_rng(11)
    s = rng.normal(size=(300, 32))
    b = (0.1 * rng.normal(size=32)).astype(np.float32)
    b[9] = 10
    s[:, [8, 10, 11]] = -np.inf
    for score, renorm in BOTH:
        check(s.astype(np.float32).astype(np.float64), 5, score, b, 8, 3, renorm, "f32")
    s[:, np.arange(32) % 4 != 1] = -np.inf
    for score, renorm in BOTH:
        check(s.astype(np.float32).astype(np.float64), 3, score, b, 8, 3, renorm, "f32")
