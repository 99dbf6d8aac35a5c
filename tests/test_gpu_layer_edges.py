"""Calls of a layer at the ends of their range."""
import pytest
import torch

from test_gpu_layer import DEV, make

pytestmark = pytest.mark.gpu


def test_no_tokens():
    from combine_moe_layout_03_gb300 import moe
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, bias, go = make(4, 256, 64, 8, False)
    layer = MoeLayer(256, 64, 8, 3)
    out, kept = layer.forward(x[:0], logits[:0], w1, w2, bias, train=True)
    grads = layer.backward(kept, go[:0], w1, w2)
    assert out.shape == (0, 256) and grads["x"].shape == (0, 256) and grads["logits"].shape == (0, 8)
    assert bool((grads["w1"] == 0).all()) and bool((grads["w2"] == 0).all())
    assert moe.moe_device_status() == moe.MOE_OK


def test_every_token_on_one_expert():
    from combine_moe_layout_03_gb300.layer import MoeLayer
    x, logits, w1, w2, _, go = make(300, 256, 64, 8, True)
    logits[:] = float("-inf")
    logits[:, 6] = 0.0
    layer = MoeLayer(256, 64, 8, 2, scale=2.0)
    out, kept = layer.forward(x, logits, w1, w2, train=True)
    grads = layer.backward(kept, go, w1, w2)
    gu = x.double() @ w1[6].double().t()
    ref = 2.0 * (torch.nn.functional.silu(gu[:, :64]) * gu[:, 64:]) @ w2[6].double().t()
    assert float((out.double() - ref).norm() / ref.norm()) < 4 * 2.0 ** -8
    idle = [e for e in range(8) if e != 6]
    assert bool((grads["w1"][idle] == 0).all()) and bool((grads["w2"][idle] == 0).all())
    # a lone expert's renormalised weight is constant: its gradient is what rounding leaves of a difference of
    # equals, 2 (G - 2 G / 2) with a handful of roundings of 2^-24 (and bf16's own)
    y = kept["y"][:300].double()
    size = 2 * (go.double() * y[kept["lay"]["slot_of"][:, 0].long()]).sum(1).abs()
    assert bool((grads["logits"][:, 6].double().abs() <= 16 * 2.0 ** -24 * size + 1e-30).all())
