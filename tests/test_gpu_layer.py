"""A whole MoE layer, forward and backward, against 64-bit autograd.

Every value that a call hands to the next is rounded to bf16 once (2^-8 at
most), so the output is within a few of those of the 64-bit one in the 2-norm;
the experts' gradients also carry the checkpoint's e4m3 rounding, at most 2^-4
of gate and of up each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(x, logits, w1, w2, idx, renorm, scale, score):
    p = torch.sigmoid(logits) if score else torch.softmax(logits, -1)
    got = idx >= 0
    w = torch.where(got, p.gather(1, idx.clamp(min=0)), torch.zeros((), dtype=p.dtype, device=p.device))
    if renorm:
        w = w / w.sum(1, keepdim=True)
    w = scale * w
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            gu = x[t] @ w1[e].t()
            f = gu.shape[1] // 2
            y = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ w2[e].t()
            out = out.index_add(0, t, w[t, j][:, None] * y)
    return out


def make(n, h, f, e, bf16):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    r = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale  # noqa: E731
    logits = r(n, e, scale=1.5)
    return (r(n, h).bfloat16(), logits.bfloat16() if bf16 else logits, r(e, 2 * f, h, scale=h ** -0.5).bfloat16(),
            r(e, h, f, scale=f ** -0.5).bfloat16(), r(e, scale=0.05), r(n, h).bfloat16())


def far(a, b):
    return float((a.double() - b.detach()).norm() / b.detach().norm())


@pytest.mark.parametrize("n,h,f,e,k,groups,score,bf16", [(200, 256, 136, 16, 4, 1, 0, False), (1, 512, 128, 32, 8, 8, 1, False),
                                                         (515, 1024, 256, 64, 2, 4, 1, True)])
def test_layer(n, h, f, e, k, groups, score, bf16):
    from combine_moe_layout_03_gb300 import moe
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, bias, go = make(n, h, f, e, bf16)
    layer = MoeLayer(h, f, e, k, num_ranks=4, score=score, num_groups=groups, topk_groups=max(1, groups // 2),
                     renormalize=bool(score), scale=2.5)
    out, kept = layer.forward(x, logits, w1, w2, bias if score else None, train=True)
    served, none = layer.forward(x, logits, w1, w2, bias if score else None)
    assert none is None and torch.equal(out, served)
    leaves = [t.double().requires_grad_() for t in (x, logits, w1, w2)]
    ref = reference(*leaves, kept["idx"].long(), bool(score), 2.5, score)
    assert far(out, ref) < 4 * 2.0 ** -8
    grads = layer.backward(kept, go, w1, w2)
    refs = torch.autograd.grad((ref * go.double()).sum(), leaves)
    assert far(grads["logits"], refs[1]) < 8 * 2.0 ** -8
    for name, want in (("x", refs[0]), ("w1", refs[2]), ("w2", refs[3])):
        assert far(grads[name], want) < 2 * 2.0 ** -4, name
    assert moe.moe_device_status() == moe.MOE_OK
    # a second micro-batch adds to the first one's gradients
    again = layer.backward(kept, go, w1, w2, moe.MOE_GRAD_F32_ADD, grads["w1"].clone(), grads["w2"].clone())
    assert torch.equal(again["w1"], 2 * grads["w1"]) and torch.equal(again["w2"], 2 * grads["w2"])


def test_tokens_without_experts():
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, _, go = make(40, 256, 64, 8, False)
    logits[3] = float("-inf")
    logits[:, 5] = float("-inf")
    layer = MoeLayer(256, 64, 8, 3)
    out, kept = layer.forward(x, logits, w1, w2, train=True)
    grads = layer.backward(kept, go, w1, w2)
    assert bool((out[3] == 0).all()) and bool((grads["x"][3] == 0).all()) and bool((grads["logits"][3] == 0).all())
    assert bool((grads["w1"][5] == 0).all()) and all(bool(torch.isfinite(g).all()) for g in grads.values())


def test_captured_step():
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, _, go = make(64, 256, 128, 16, False)
    layer = MoeLayer(256, 128, 16, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.backward(layer.forward(x, logits, w1, w2, train=True)[1], go, w1, w2)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, kept = layer.forward(x, logits, w1, w2, train=True)
        grads = layer.backward(kept, go, w1, w2)
    x2, l2 = make(65, 256, 128, 16, False)[:2]
    x.copy_(x2[:64])
    logits.copy_(l2[:64])
    g.replay()
    torch.cuda.synchronize()
    want, kept2 = layer.forward(x, logits, w1, w2, train=True)
    more = layer.backward(kept2, go, w1, w2)
    assert torch.equal(out, want) and all(torch.equal(grads[k], more[k]) for k in grads)
