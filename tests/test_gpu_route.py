"""The router against plain 64-bit loops.

Ids have to be equal. Weights and gradients are fp32 from a handful of
operations: expf (2 units), the argument's rounding (|x - top| <= 32 units for
these draws), sums over at most 1024 terms in a tree (11), divisions and
products (6): under 64 units of 2^-24 relative to the largest term."""
import numpy as np
import pytest
import torch

from layer_reference import HALF_BF16, UNIT, clean, route, route_weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    return m


def desc_of(moe, n, e, k, score, groups, topk_groups, group_score, renorm, scale, bf16, stride=0):
    return moe.MoeRouteDesc(n, e, k, moe.MOE_SCORE_SIGMOID if score == "sigmoid" else moe.MOE_SCORE_SOFTMAX, groups,
                            topk_groups, moe.MOE_GROUP_MAX if group_score == "max" else moe.MOE_GROUP_TOP2_SUM, renorm,
                            scale, moe.MOE_LOGITS_BF16 if bf16 else moe.MOE_LOGITS_F32, stride)


def check(moe, logits, bias, k, score="softmax", groups=1, topk_groups=1, group_score="max", renorm=True, scale=1.0,
          grad=True):
    n, e = logits.shape
    d = desc_of(moe, n, e, k, score, groups, topk_groups, group_score, renorm, scale, logits.dtype == torch.bfloat16,
                logits.stride(0) if n > 1 else 0)
    idx, w = moe.moe_route(d, logits, bias)
    ids, ref = route(logits, bias, k, score, groups, topk_groups, group_score, renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), ids)
    got = w.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 64 * UNIT * np.abs(ref) + 1e-37)
    assert np.all(got[ids < 0] == 0)
    if not grad:
        return
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    gw = torch.randn(n, k, generator=g, device=DEV)
    dl = moe.moe_route_backward(d, logits, idx, gw)
    x = torch.from_numpy(np.where(np.isinf(clean(logits)), -1e300, clean(logits))).requires_grad_()
    tid = torch.from_numpy(ids)
    weights = route_weights(x, tid, score, renorm, scale)
    upstream = torch.where(tid >= 0, gw.double().cpu(), torch.zeros((), dtype=torch.float64))
    (ref_grad,) = torch.autograd.grad((weights * upstream).sum(), x)
    ref_grad = torch.nan_to_num(ref_grad)
    # each term is a product of weights and gradients, of which one sum is subtracted
    size = (weights.detach().abs() * upstream.abs()).sum(1, keepdim=True) + weights.detach().abs().amax(1, keepdim=True) * upstream.abs().amax(1, keepdim=True)
    lim = 64 * UNIT * size + (HALF_BF16 if logits.dtype == torch.bfloat16 else 4 * UNIT) * ref_grad.abs() + 1e-37
    assert bool(((dl.double().cpu() - ref_grad).abs() <= lim).all())


def draw(seed, n, e, bf16, scale=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, e, generator=g, device=DEV) * scale
    return x.to(torch.bfloat16) if bf16 else x


def draw_bias(seed, e, scale=0.1):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 + seed)
    return torch.randn(e, generator=g, device=DEV) * scale


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (3, 7, 7), (33, 33, 4), (1, 256, 8), (257, 256, 8), (20, 1000, 10), (5, 1024, 32), (64, 60, 6)])
def test_scores(moe, n, e, k, score, biased, bf16, renorm):
    check(moe, draw(1, n, e, bf16), draw_bias(1, e) if biased else None, k, score, renorm=renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,e,k,groups,topk_groups", [(70, 256, 8, 8, 4), (9, 96, 6, 32, 6), (9, 32, 3, 32, 3), (40, 1024, 9, 4, 1),
                                                      (13, 160, 6, 8, 3), (7, 6, 2, 2, 1), (11, 9, 3, 3, 3)])
def test_groups(moe, n, e, k, groups, topk_groups, score, biased, group_score):
    for bf16 in (False, True):
        check(moe, draw(2, n, e, bf16), draw_bias(2, e) if biased else None, k, score, groups, topk_groups, group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_experts_taken_out(moe, score, biased):
    e, k = 48, 6
    x = draw(3, 40, e, False)
    x[torch.rand(40, e, device=DEV) < 0.5] = -INF
    x[0] = -INF                 # nobody left
    x[1] = -INF
    x[1, 40] = 0.25             # one left
    x[2, 5] = float("nan")
    x[3] = float("nan")
    x[4, 7] = INF               # the largest finite value
    x[5] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[6, 3] = 1.0
    x[7] = -INF
    x[7, 8:12] = torch.finfo(torch.float32).min
    b = None
    if biased:
        b = draw_bias(3, e)
        b[9], b[10] = -INF, float("nan")
    rows = slice(0, 40)
    for groups, topk_groups, gs in ((1, 1, "max"), (8, 3, "max"), (8, 3, "top2")):
        for renorm in (False, True):
            if renorm and score == "sigmoid":  # a sum of sigmoids of the lowest value has no ratio in 64 bits either
                rows = torch.tensor([i for i in range(40) if i not in (5, 6, 7)], device=DEV)
            check(moe, x[rows].contiguous(), b, k, score, groups, topk_groups, gs, renorm, grad=False)
    keep = torch.tensor([i for i in range(40) if i not in (4, 5, 6, 7)], device=DEV)
    for renorm in (False, True):
        check(moe, x[keep].contiguous(), b, k, score, renorm=renorm)


@pytest.mark.parametrize("bf16", [False, True])
def test_ties_go_to_the_lower_index(moe, bf16):
    t = torch.bfloat16 if bf16 else torch.float32
    flat = torch.zeros(4, 64, dtype=t, device=DEV)
    flat[1, 60:] = 1.0
    flat[2, ::2] = -1.0
    for score in ("softmax", "sigmoid"):
        for b in (None, torch.zeros(64, device=DEV)):
            check(moe, flat, b, 8, score)
            for gs in ("max", "top2"):
                check(moe, flat, b, 8, score, 8, 4, gs)


def test_order_that_fp32_cannot_tell(moe):
    # sigmoid(x) + b equal to within 2^-30: the sums are ordered as in 64 bits
    g = np.random.default_rng(5)
    e, rows = 64, []
    base = 0.75
    b = (0.02 * g.standard_normal(e)).astype(np.float32)
    for _ in range(50):
        s = base + g.uniform(-1, 1, e) * 2.0 ** -28 - b.astype(np.float64)
        rows.append(np.log(s / (1 - s)))
    x = torch.tensor(np.array(rows), dtype=torch.float32, device=DEV)
    bias = torch.from_numpy(b).to(DEV)
    key = 1 / (1 + np.exp(-clean(x))) + b.astype(np.float64)
    gaps = np.diff(np.sort(key, 1), axis=1)
    assert (gaps < 2.0 ** -26).mean() > 0.5 and (gaps > 1e-14).all()  # hard, and defined
    check(moe, x, bias, 8, "sigmoid", grad=False)
    check(moe, x, bias, 8, "sigmoid", 8, 4, "top2", grad=False)
    check(moe, x, bias, 8, "sigmoid", 8, 4, "max", grad=False)


def test_a_few_rows_among_many_that_fp32_cannot_tell(moe):
    x = draw(6, 3000, 256, False)
    bias = draw_bias(6, 256)
    s = torch.sigmoid(x.double())
    order = (s + bias.double()).sort(1, descending=True).indices
    for place in (0, 3, 7):  # pull the next expert's key up to the one before it
        at, to = order[::3, place + 1], order[::3, place]
        rows = torch.arange(0, 3000, 3, device=DEV)
        want = (s[rows, to] + bias.double()[to] - bias.double()[at]).clamp(1e-3, 1 - 1e-6)
        x[rows, at] = torch.log(want / (1 - want)).float()
    check(moe, x, bias, 8, "sigmoid", grad=False)
    check(moe, x, bias, 8, "sigmoid", 8, 4, "top2", grad=False)


def test_strided_and_unaligned_logits(moe):
    for bf16 in (False, True):
        wide = draw(7, 21, 300, bf16)
        for off in (0, 1, 3, 8):
            check(moe, wide[:, off:off + 256], draw_bias(7, 256), 8, "sigmoid", 8, 4, "top2")
            check(moe, wide[:, off:off + 37], None, 5, "softmax", renorm=False)


def test_many_tokens(moe):
    check(moe, draw(8, 5000, 128, True), None, 4, "softmax", renorm=False)


def test_far_logits_keep_their_ratios(moe):
    x = draw(9, 16, 64, False) - 200.0
    for score in ("softmax", "sigmoid"):
        check(moe, x, None, 6, score, grad=False)


def test_gradient_against_differences(moe):
    x = draw(10, 6, 40, False)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            d = desc_of(moe, 6, 40, 5, score, 1, 1, "max", renorm, 1.5, False)
            idx, _ = moe.moe_route(d, x)
            gw = draw(11, 6, 5, False)
            got = moe.moe_route_backward(d, x, idx, gw).double().cpu()
            v = draw(12, 6, 40, False).double().cpu()
            ids, up = idx.long().cpu(), gw.double().cpu()
            loss = lambda a: (route_weights(a, ids, score, renorm, 1.5) * up).sum()  # noqa: E731
            h = 1e-5
            by = (loss(x.double().cpu() + h * v) - loss(x.double().cpu() - h * v)) / (2 * h)
            assert abs((got * v).sum() - by) <= 1e-5 * (got * v).abs().sum()


def test_ids_feed_the_layout(moe):
    # rows without a full set of experts go through the layout as -1
    x = draw(13, 50, 32, False)
    x[:, 4:] = -INF
    x[7] = -INF
    d = desc_of(moe, 50, 32, 6, "sigmoid", 1, 1, "max", True, 1.0, False)
    idx, _ = moe.moe_route(d, x)
    lay = moe.moe_layout(moe.MoeDesc(50, 6, 32, 4, 8), idx)
    assert moe.moe_layout_status(lay["workspace"]) == moe.MOE_OK
    assert int(lay["expert_offset"][-1]) == 49 * 4


def test_other_stream_and_graph(moe):
    x = draw(14, 100, 64, False)
    d = desc_of(moe, 100, 64, 4, "softmax", 1, 1, "max", True, 1.0, False)
    idx = torch.empty(100, 4, dtype=torch.int32, device=DEV)
    w = torch.empty(100, 4, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = moe.prepare_route(d, x, None, idx, w, stream=s)
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    s.synchronize()
    x.copy_(draw(15, 100, 64, False))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(idx.cpu().numpy(), route(x, None, 4, "softmax", 1, 1, "max", True, 1.0)[0])
