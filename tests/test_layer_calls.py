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


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on the GPU (nothing is launched)."""
    is_cuda = property(lambda self: True)


def test_the_layer_refuses_tokens_that_are_not_dense_rows(moe, monkeypatch):
    # dispatch, combine and their backward take pointers: an expanded gradient
    # (of a sum) would be read behind its one element
    from combine_moe_layout_03_gb300.layer import MoeLayer

    def launched(*args, **kw):
        raise AssertionError("launched")

    for name in ("moe_route", "moe_layout_dispatch", "moe_combine_backward"):
        monkeypatch.setattr(moe, name, launched)
    n, h = 6, 16
    layer = MoeLayer(h, 8, 4, 2)
    kept = dict(d=moe.MoeDesc(n, 2, 4, 1, h), lay=dict(expert_offset=torch.zeros(5, dtype=torch.int32), slot_of=None), rows=None, weights=None, y=None)
    bf16 = lambda t: t.bfloat16().as_subclass(OnGpu)  # noqa: E731
    wide = bf16(torch.zeros(n, 2 * h))
    bad = [bf16(torch.ones(())).expand(n, h), bf16(torch.zeros(h)).expand(n, h), wide[:, :h], bf16(torch.zeros(h, n)).t(),
           torch.zeros(n, h).as_subclass(OnGpu), torch.zeros(n, h).bfloat16()]
    for t in bad:
        for call in (lambda: layer.forward(t, torch.zeros(n, 4), None, None), lambda: layer.backward(kept, t, None, None)):
            with pytest.raises(moe.MoeError) as err:
                call()
            assert err.value.code == moe.MOE_ERR_INVALID_ARG
    for t in (wide, bf16(torch.zeros(n * h))):
        with pytest.raises(moe.MoeError) as err:
            layer.forward(t, torch.zeros(n, 4), None, None)
        assert err.value.code == moe.MOE_ERR_SHAPE
    with pytest.raises(moe.MoeError) as err:
        layer.backward(kept, bf16(torch.zeros(n - 1, h)), None, None)
    assert err.value.code == moe.MOE_ERR_SHAPE
    good = bf16(torch.zeros(n, h))
    for call in (lambda: layer.forward(good, torch.zeros(n, 4), None, None), lambda: layer.backward(kept, good, None, None)):
        with pytest.raises(AssertionError, match="launched"):
            call()
