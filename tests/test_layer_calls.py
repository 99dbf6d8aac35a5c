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


def test_rows_that_lie_as_the_descriptor_says(moe):
    t = torch.zeros(4, 3, 24)
    on = lambda v: v.as_subclass(OnGpu)  # noqa: E731
    want = lambda v, rows, width, stride: moe._want_rows("x", on(v), torch.float32, rows, width, stride)  # noqa: E731
    # dense, whatever the shape; padded rows; a batch of padded rows; one row; a column of width 1
    for args in ((t, 12, 24, 24), (t.view(12, 24), 12, 24, 24), (t.view(-1), 12, 24, 24), (t.view(24, 12), 12, 24, 24),
                 (t.view(12, 2, 12), 12, 24, 24), (t.view(1, 12, 24), 5, 24, 24),
                 (t.view(12, 24)[:, 8:], 12, 16, 24), (t[..., 8:], 12, 16, 24), (t[:, :, :16], 11, 16, 24), (t, 12, 16, 24),
                 (t.view(12, 24)[5:6, :8], 1, 8, 8), (t.view(12, 24)[::2], 6, 24, 48), (t.view(12, 24)[:, 7:8], 12, 1, 24),
                 (t.view(1, 288).t(), 288, 1, 1), (torch.zeros(0, 24), 0, 24, 24)):
        want(*args)
    # rows further apart than the descriptor says, uneven ones, columns, repeated rows
    for args in ((t[..., 8:], 12, 16, 16), (t[..., :16], 12, 16, 16), (t[:, :2], 8, 24, 24), (t[:, ::2, 8:], 8, 16, 24),
                 (t.transpose(0, 1), 12, 24, 24), (t.view(12, 24).t(), 24, 12, 12), (torch.zeros(24).expand(12, 24), 12, 24, 24),
                 (t.view(12, 24)[:, ::2], 12, 12, 24), (t.view(4, 72), 12, 24, 24), (t.view(12, 24), 12, 16, 16), (t.view(12, 24)[:, 8:], 12, 16, 16),
                 (torch.zeros(()).expand(12, 1), 12, 1, 1)):
        with pytest.raises(moe.MoeError) as err:
            want(*args)
        assert err.value.code == moe.MOE_ERR_INVALID_ARG, args[1:]
    # too few rows in the view, whatever its storage holds
    for args in ((t.view(12, 24)[:5], 6, 24, 24), (t[..., 8:], 13, 16, 24), (t.view(-1)[:280], 12, 24, 24), (torch.zeros(0, 24), 1, 24, 24)):
        with pytest.raises(moe.MoeError) as err:
            want(*args)
        assert err.value.code == moe.MOE_ERR_CAPACITY, args[1:]
    # through the calls: a batch of padded rows needs its stride named
    x = on(torch.zeros(2, 3, 72, dtype=torch.bfloat16))[..., 8:]
    ids = on(torch.zeros(2, dtype=torch.int32))
    w, y = on(torch.zeros(2, 8, 64, dtype=torch.bfloat16)), on(torch.zeros(6, 8, dtype=torch.bfloat16))
    with pytest.raises(moe.MoeError):
        moe.prepare_expert_product(moe.MoeExpertDesc(2, 6, 64, 8), x, ids, ids, w, y, stream=0)
    moe.prepare_expert_product(moe.MoeExpertDesc(2, 6, 64, 8, x_stride=72), x, ids, ids, w, y, stream=0)
    logits = on(torch.zeros(2, 3, 20))[..., :16]
    out, weights = on(torch.zeros(6, 2, dtype=torch.int32)), on(torch.zeros(6, 2))
    with pytest.raises(moe.MoeError):
        moe.prepare_route(moe.MoeRouteDesc(6, 16, 2), logits, None, out, weights, stream=0)
    moe.prepare_route(moe.MoeRouteDesc(6, 16, 2, logits_stride=20), logits, None, out, weights, stream=0)
