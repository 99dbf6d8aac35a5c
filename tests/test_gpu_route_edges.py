"""Keys at the edges of what fp32 can tell: infinite and overflowing biases,
infinite logits, and near-ties that lie behind the last place. Ids have to be
those of 64-bit arithmetic (the bounds of weights are those of test_gpu_route)."""
import numpy as np
import pytest
import torch

from test_gpu_route import DEV, INF, check, draw, draw_bias

pytestmark = pytest.mark.gpu
MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    return m


# ---- group counts that are infinite or overflow

@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,topk_groups", [(16, 4, 1), (64, 8, 2), (256, 8, 3), (60, 6, 2), (96, 32, 4)])
def test_infinite_bias_forces_an_expert(moe, e, groups, topk_groups, score, group_score):
    per = e // groups
    x = draw(21, 24, e, False)
    # as many forced groups as are taken, fewer, more, and two experts of one group
    for forced in ([g * per + 1 for g in range(groups - topk_groups, groups)], [e - 1],
                   [g * per for g in range(groups)], [e - 1, e - 2, per]):
        bias = draw_bias(21, e)
        bias[forced] = INF
        check(moe, x, bias, 2, score, groups, topk_groups, group_score, grad=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(32, 4), (64, 8), (256, 8), (24, 4)])
def test_group_sums_that_overflow(moe, e, groups, score):
    per = e // groups
    x = draw(22, 16, e, False)
    bias = draw_bias(22, e)
    bias[per:per + 2] = 2e38
    bias[2 * per:2 * per + 2] = 3e38  # the larger sum, in 64 bits
    for topk_groups in (1, 2, 3):
        check(moe, x, bias, 4, score, groups, topk_groups, "top2", grad=False)
    # experts masked by the lowest value stay before those that are taken out
    bias = draw_bias(22, e)
    bias[(groups - 1) * per:] = -MOST
    x[:, :(groups - 2) * per] = -INF
    check(moe, x, bias, 4, score, groups, 2, "top2", grad=False)


@pytest.mark.parametrize("e,groups", [(32, 4), (256, 8), (12, 3)])
def test_infinite_logits_tie_with_the_largest(moe, e, groups):
    x = draw(23, 8, e, False)
    x[:, 1] = MOST
    x[:, e - 1] = INF
    for score in ("softmax", "sigmoid"):
        check(moe, x, None, 2, score, groups, 1, "max", grad=False)


# ---- keys beyond the fixed-point range in every lane

@pytest.mark.parametrize("e", [128, 256, 1000])
def test_a_largest_key_in_every_lane(moe, e):
    x = draw(24, 6, e, False)
    inf = x.clone()
    inf[:, 1::4] = INF
    check(moe, inf, None, 5, "sigmoid", grad=False)
    inf[:, 2::4] = MOST
    check(moe, inf, None, 5, "sigmoid", grad=False)
    bias = draw_bias(24, e)
    bias[1::4] = INF
    for score in ("softmax", "sigmoid"):
        check(moe, x, bias, 5, score, grad=False)
    # all but a few
    few = torch.full_like(x, INF)
    few[:, 3:80:4] = x[:, 3:80:4]
    check(moe, few, None, 5, "sigmoid", grad=False)
    bias.fill_(INF)
    bias[3:80:4] = 0.1
    check(moe, x, bias, 5, "softmax", grad=False)


# ---- what lies behind the last place

def from_keys(key, bias):
    """Logits (fp32) whose sigmoid + bias is about key (float64 [N, E])."""
    s = key - bias.astype(np.float64)
    x = torch.tensor(np.log(s / (1 - s)), dtype=torch.float32, device=DEV)
    return x, torch.from_numpy(bias).to(DEV)


@pytest.mark.parametrize("e", [128, 256, 1024])
def test_the_thirty_third_key_behind_thirty_two_lanes(moe, e):
    # the 32 largest keys lie one to a lane (experts 4 l), and the next one is
    # within an fp32 step or so of the smallest of them
    g, n = np.random.default_rng(25), 300
    bias = (0.02 * g.standard_normal(e)).astype(np.float32)
    key = 0.6 + 0.01 * g.random((n, e))
    tops = 0.75 + 1e-3 * g.random((n, 32))
    key[:, 0:128:4] = tops
    rows = np.arange(n)
    low = 4 * tops.argmin(1)
    rival = (4 * g.integers(0, 32, n) + 1)
    key[rows, rival] = key[rows, low] + g.uniform(-1, 1, n) * 2.0 ** -25
    x, b = from_keys(key, bias)
    true = 1 / (1 + np.exp(-x.double().cpu().numpy())) + bias.astype(np.float64)
    gap = true[rows, rival] - true[rows, low]
    assert 0.2 < (gap > 0).mean() < 0.8 and (np.abs(gap) > 1e-14).all()  # decided either way, and defined
    check(moe, x, b, 32, "sigmoid", grad=False)


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("k", [1, 3])
def test_a_larger_key_behind_an_equal_one(moe, k, groups):
    # two equal keys, one of them at the last place, and a third that is larger
    # only in 64 bits
    e = 128
    for bf16 in (False, True):
        x = draw(26, 40, e, bf16).clamp(-4, 4)
        for r in range(40):
            at = [2 + r % 20, 23 + r % 5, 90 + r % 20]
            x[r, 100:100 + k - 1] = 30.0 + r % 2
            x[r, at[:2]] = 20.0
            x[r, at[2]] = 21.0
            if k > 1:
                x[r, 120:120 + k - 1] = 9.0  # in the way of nothing
        for b in (torch.zeros(e, device=DEV), torch.full((e,), 0.25, device=DEV)):
            check(moe, x, b, k, "sigmoid", groups, groups, "max", grad=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_larger_logit_behind_an_equal_one_in_one_step(moe, score):
    # an outlier stretches the range, so that 0.5 and 0.50001 are one step
    x = torch.zeros(3, 256, device=DEV)
    x[:, 200] = 1000.0
    x[:, [10, 11]] = 0.5
    x[:, 30] = 0.50001
    x[1, 31] = 0.50002
    x[2, 9] = 0.49999
    for k in (2, 3):
        check(moe, x, None, k, score, grad=False)


def test_equal_keys_in_plenty(moe):
    # ties alone stay with the lower index, however many there are
    for bf16 in (False, True):
        x = (draw(27, 60, 256, bf16) * 2).round() / 2
        for b in (None, torch.zeros(256, device=DEV)):
            check(moe, x, b, 8, "sigmoid", grad=False)
            check(moe, x, b, 32, "softmax", grad=False)
            check(moe, x, b, 8, "sigmoid", 8, 4, "top2", grad=False)


def test_masks_of_large_finite_values(moe):
    for mask in (-1e4, -1e9, -1e30, -3e38):
        for e in (128, 256):
            x = draw(28, 20, e, False)
            x[:, 4:8] = mask
            x[3:, 64:] = mask
            check(moe, x, None, 6, "softmax", grad=False)
            check(moe, x, draw_bias(28, e), 6, "softmax", 8, 4, "top2", grad=False)
