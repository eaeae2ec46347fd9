"""Borders of the expert choice that FP32 leaves open: the last expert chosen and
the first one left out are equal and a third key lies within FP32's reach of them;
sums of two keys that cancel.  The ids must be those of the binary64 keys
(oracle/moe.py), whatever the FP32 keys say."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_b200 as fq
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _same_ids(dev, l, k, dtype=torch.float32, bias=None, **kw):
    """l must be values that dtype holds."""
    t = torch.from_numpy(np.ascontiguousarray(l, dtype=np.float32)).to(dtype)
    assert np.array_equal(t.float().numpy(), l)
    bias = None if bias is None else np.asarray(bias, dtype=np.float32)
    ids, _ = fq.fp8_moe_route(t.to(dev), k, bias=None if bias is None else torch.from_numpy(bias).to(dev), **kw)
    oi, _ = moe.route(l.astype(np.float64), k, bias=bias, **kw)
    got = ids.cpu().numpy()
    wrong = np.flatnonzero((got != oi).any(axis=1))
    assert wrong.size == 0, (wrong.size, l.shape[0], got[wrong[0]], oi[wrong[0]])


@pytest.mark.parametrize("E", [32, 64, 256, 512, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_keys_at_the_border_and_a_larger_one_in_reach(dev, score, E):
    """Every FP32 key is 0.25 (but the dominant one's); experts 0 and 1 are equal,
    expert 2 is larger by 1e-13: it is chosen, not expert 0."""
    l = np.full((3, E), -40.0, np.float32)
    l[:, :2] = -30.0
    l[:, 2] = -29.0
    l[1, 2], l[1, E - 1] = -30.0, -29.0          # the larger one last
    l[2, 2] = -31.0                              # a smaller one in reach: the lower of the equal two stays
    bias = np.full(E, 0.25)
    _same_ids(dev, l, 1, bias=bias, score=score)
    l[:, 20] = 0.0                               # dominant: the first place, and of a softmax nearly the whole sum
    for k in (2, 3):
        _same_ids(dev, l, k, bias=bias, score=score)
        _same_ids(dev, l, k, bias=bias, score=score, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,KG,GT", [(64, 4, 2, 2), (64, 4, 2, 1), (256, 8, 4, 2), (60, 5, 2, 2), (768, 3, 2, 2)])
def test_equal_keys_at_the_border_inside_a_kept_group(dev, score, E, G, KG, GT):
    size = E // G
    l = np.full((2, E), -40.0, np.float32)
    l[:, size] = l[:, size + 1] = 0.0            # group 1 and the last group lead
    l[:, E - 1] = l[:, E - 2] = -0.5
    l[:, size + 3] = l[:, size + 4] = -30.0
    l[:, size + 6] = -29.0
    l[1, size + 6], l[1, E - 3] = -40.0, -29.0   # the larger key in the other kept group
    l[:, 2] = -28.0                              # larger still, in a group that is dropped
    for k in (5, 6):
        _same_ids(dev, l, k, bias=np.full(E, 0.25), score=score, n_group=G, topk_group=KG, group_top=GT)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(32, 1), (32, 8), (60, 2), (64, 1), (256, 1), (256, 8), (512, 3), (64, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_saturated_scores_with_a_uniform_bias(dev, score, E, k, dtype):
    """Scores that a bias leaves without FP32 digits, from logits of few distinct
    values: many equal keys, and others in reach, at the border of the choice."""
    rng = np.random.default_rng(E + k)
    mean = {"sigmoid": 22.0, "softmax": -24.0}[score]
    l = torch.from_numpy((mean + rng.standard_normal((300, E))).astype(np.float32)).to(torch.bfloat16).float().numpy()
    if score == "softmax":
        l[:, E // 2] = 0.0
    for b in (0.0, 0.25, -3.0):
        _same_ids(dev, l, k, dtype, bias=np.full(E, b), score=score)


@pytest.mark.parametrize("E,k", [(32, 1), (256, 8), (512, 8)])
def test_rows_of_equal_logits_go_to_the_lowest_indices(dev, E, k):
    l = np.zeros((5, E), np.float32)
    l[1] = -7.5
    l[2, E // 2:] = 1.0
    for bias in (np.zeros(E), np.where(np.arange(E) % 3, 0.5, 0.25)):
        for score in ("softmax", "sigmoid"):
            _same_ids(dev, l, k, bias=bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,KG", [(32, 4, 2), (256, 8, 4), (60, 5, 1), (1024, 2, 1), (64, 32, 5)])
@pytest.mark.parametrize("size_of_bias", [4.0, 1000.0, 3e5])
def test_group_sums_that_cancel(dev, score, E, G, KG, size_of_bias):
    """The best two keys of each group are + and - a large bias: their FP32 sum is
    off by the bias's rounding, far more than the sum's."""
    rng = np.random.default_rng(E + G)
    size = E // G
    T = 200
    bias = np.full(E, -np.inf)
    l = rng.standard_normal((T, E)).astype(np.float32)
    for g in range(G):
        a, b = rng.choice(size, 2, replace=False)
        bias[g * size + a], bias[g * size + b] = size_of_bias, -size_of_bias
        # sums of two scores that differ between the groups by a few FP32 steps of the bias at most
        step = 2.0 ** -22 * size_of_bias if size_of_bias < 1e4 else 0.05
        l[:, g * size + a] = (0.25 + step * rng.standard_normal(T)).astype(np.float32)
        l[:, g * size + b] = (-0.5 + step * rng.standard_normal(T)).astype(np.float32)
    _same_ids(dev, l, 2 * KG, bias=bias, score=score, n_group=G, topk_group=KG, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_of_very_large_and_infinite_biases(dev, score):
    """Sums beyond FP32's largest value, infinite ones, and groups with one expert
    or none left."""
    rng = np.random.default_rng(3)
    E, G, size = 64, 8, 8
    l = rng.standard_normal((40, E)).astype(np.float32)
    l[:, 7 * size:] = -np.inf                    # no expert
    l[::2, 6 * size + 1:7 * size] = -np.inf      # one expert
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[:2] = 3.4e38
    bias[size:size + 2] = 3.3e38
    bias[2 * size] = np.inf
    bias[3 * size:3 * size + 2] = 3.4e38
    bias[4 * size:4 * size + 2] = -3.4e38
    for KG in (1, 2, 3, 4, 5, 7, 8):
        _same_ids(dev, l, 2, bias=bias, score=score, n_group=G, topk_group=KG, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (60, 15), (512, 8), (1024, 8)])
def test_group_sums_below_the_range_come_before_groups_without_experts(dev, score, E, G):
    """Two biases of -3.4e38 make a sum that only binary64 holds; a group whose
    experts are all masked has none."""
    rng = np.random.default_rng(E)
    size = E // G
    for low in (-3.4e38, -2e38):
        l = rng.standard_normal((30, E)).astype(np.float32)
        bias = np.full(E, low, np.float32)
        l[:, np.arange(E) % size > 2] = -np.inf                 # three experts a group
        bias[2 * size:3 * size] = 0.1
        l[:, :size] = -np.inf                                   # the first group is empty
        bias[size + 1:2 * size] = -np.inf                       # one expert left in the second
        l[::3, (G - 1) * size:] = -np.inf                       # the last is empty too
        for KG in range(1, G + 1):
            _same_ids(dev, l, min(KG * size, 3 * G, 32), bias=bias, score=score, n_group=G, topk_group=KG, group_top=2)
