"""A layer served with 8-bit experts: the calls one by one give what forward_i8
gives, and it stays near the bf16 layer."""
import pytest
import torch

from layer_reference import HALF_BF16, swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(n, h, f, e, f32=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    r = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale  # noqa: E731
    w1, w2 = r(e, 2 * f, h, scale=h ** -0.5), r(e, h, f, scale=f ** -0.5)
    return r(n, h).bfloat16(), r(n, e, scale=1.5), w1 if f32 else w1.bfloat16(), w2 if f32 else w2.bfloat16(), r(e, scale=0.05)


def reference(layer, x, logits, bias, experts):
    """float64 [N, H]: 64-bit products of the same codes, token by token."""
    from combine_moe_layout_03_gb300 import moe
    n, h, f, e, k = x.shape[0], layer.hidden, layer.width, layer.num_experts, layer.topk
    q1, s1, q2, s2 = experts
    idx, weights = moe.moe_route(layer._descs(n, logits)[0], logits, bias)
    rows = lambda t: moe.moe_quantize_rows(moe.MoeQuantDesc(t.shape[0], t.shape[1]), t)  # noqa: E731
    q, s = rows(x)
    ref = torch.zeros(n, h, dtype=torch.float64, device=DEV)
    for j in range(k):
        for i in range(e):
            t = (idx[:, j] == i).nonzero().view(-1)
            if len(t):
                v = (q[t].double() @ q1[i].double().t()) * s[t].double() * s1[i].double()
                a, sa = rows(swiglu(v[:, :f], v[:, f:]).to(torch.bfloat16))
                ref[t] += weights[t, j].double()[:, None] * ((a.double() @ q2[i].double().t()) * sa.double() * s2[i].double())
    return ref


@pytest.mark.parametrize("n,h,f,e,k,groups,f32", [(200, 256, 144, 16, 4, 1, False), (1, 512, 128, 32, 8, 8, True), (515, 1024, 256, 64, 2, 4, False)])
def test_layer(n, h, f, e, k, groups, f32):
    from combine_moe_layout_03_gb300 import moe
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, bias = make(n, h, f, e, f32)
    logits[0] = float("-inf")  # a token that no expert takes
    layer = MoeLayer(h, f, e, k, num_ranks=4, score=moe.MOE_SCORE_SIGMOID, num_groups=groups, topk_groups=max(1, groups // 2), scale=2.5)
    experts = layer.quantize(w1, w2)
    out = layer.forward_i8(x, logits, experts, bias)
    q1, s1, q2, s2 = experts
    assert q1.shape == w1.shape and s1.shape == w1.shape[:2] and q2.shape == w2.shape and s2.shape == w2.shape[:2]
    ref = reference(layer, x, logits, bias, experts)
    assert not out[0].any() and not ref[0].any()
    if n > 1:
        # the experts' outputs and the sum are rounded to bf16 once each; an activation that rounds to the neighbouring
        # bf16 may change a code by one of some 36
        assert float((out.double() - ref).norm() / ref.norm()) < 2 * HALF_BF16
        plain, _ = layer.forward(x, logits, w1.bfloat16(), w2.bfloat16(), bias)
        assert float((out.double() - plain.double()).norm() / plain.double().norm()) < 0.04


@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("h,f,e,k", [(512, 128, 32, 8), (1024, 272, 8, 2), (7168, 256, 256, 8), (256, 64, 1, 1)])
def test_single_tokens(n, h, f, e, k):
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, bias = make(n, h, f, e)
    layer = MoeLayer(h, f, e, k, scale=2.5)
    experts = layer.quantize(w1, w2)
    out, ref = layer.forward_i8(x, logits, experts, bias), reference(layer, x, logits, bias, experts)
    # as above: two roundings to bf16, and a code of the activation that may be the neighbouring one
    assert float((out.double() - ref).norm() / ref.norm()) < 2 * HALF_BF16


def test_layer_in_a_graph_follows_the_routing():
    from combine_moe_layout_03_gb300.layer import MoeLayer
    n, h, f, e, k = 24, 256, 128, 16, 2
    x, logits, w1, w2, _ = make(n, h, f, e)
    layer = MoeLayer(h, f, e, k)
    experts = layer.quantize(w1, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward_i8(x, logits, experts)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward_i8(x, logits, experts)
    for seed in range(3):
        x2, logits2, *_ = make(n + 100 + seed, h, f, e)
        x.copy_(x2[:n])
        logits.copy_(logits2[:n])
        graph.replay()
        assert torch.equal(out, layer.forward_i8(x, logits, experts))


def test_no_tokens():
    from combine_moe_layout_03_gb300.layer import MoeLayer
    _, _, w1, w2, _ = make(3, 64, 32, 4)
    layer = MoeLayer(64, 32, 4, 2)
    out = layer.forward_i8(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 4, device=DEV), layer.quantize(w1, w2))
    assert out.shape == (0, 64)
