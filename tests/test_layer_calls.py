"""What the Python calls of the router, the activation, the experts' products and
the layer do around the library (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import build
    build.build_library()
    from combine_moe_layout_03_gb300 import moe as m
    return m


def test_a_weight_gradient_without_a_buffer_is_not_filled_first(moe, monkeypatch):
    # a fill would cost as much as the result's stores, and stand in another
    # stream's order than the call
    seen = []

    def prepare(desc, grad_y, x, row_begin, row_end, grad_w, grad_kind, stream):
        return lambda: seen.append((grad_w, grad_kind))

    def fill(*args, **kw):
        raise AssertionError("filled")

    monkeypatch.setattr(moe, "prepare_expert_product_backward_weight", prepare)
    for name in ("zeros", "zeros_like", "full"):
        monkeypatch.setattr(torch, name, fill)
    ids = torch.empty(3, dtype=torch.int32)
    for kind, dtype, used in ((moe.MOE_GRAD_BF16, torch.bfloat16, moe.MOE_GRAD_BF16), (moe.MOE_GRAD_F32, torch.float32, moe.MOE_GRAD_F32),
                              (moe.MOE_GRAD_F32_ADD, torch.float32, moe.MOE_GRAD_F32)):
        got = moe.moe_expert_product_backward_weight(moe.MoeExpertDesc(3, 5, 16, 8), None, None, ids, ids, grad_kind=kind)
        assert got.shape == (3, 8, 16) and got.dtype == dtype and seen[-1][0] is got and seen[-1][1] == used
        mine = torch.empty(3, 8, 16)
        assert moe.moe_expert_product_backward_weight(moe.MoeExpertDesc(3, 5, 16, 8), None, None, ids, ids, mine, kind) is mine
        assert seen[-1][0] is mine and seen[-1][1] == kind
