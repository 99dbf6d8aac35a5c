"""What the 8-bit calls refuse, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

INVALID, ALIGN, SHAPE, CAPACITY = -1, -2, -3, -4


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import build
    build.build_library()
    from combine_moe_layout_03_gb300 import moe as m
    return m


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on the GPU (nothing is launched)."""
    is_cuda = property(lambda self: True)


def gpu(*shape, dtype=torch.int8):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def code_of(moe, call, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        call(*args, **kw)
    return e.value.code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(width=0), SHAPE), (dict(width=8), SHAPE), (dict(width=24), SHAPE),
    (dict(width=65552), SHAPE), (dict(x_stride=48), SHAPE), (dict(x_stride=68), SHAPE), (dict(x_stride=-8), SHAPE),
    (dict(x_stride=1 << 36), SHAPE), (dict(scale_stride=2), SHAPE), (dict(scale_stride=-1), SHAPE), (dict(x_kind=2), INVALID),
    (dict(x_kind=-1), INVALID)])
def test_quantize_shapes(moe, kw, code):
    d = moe.MoeQuantDesc(**{**dict(rows=4, width=64), **kw})
    assert moe._lib.moe_quantize_rows(ctypes.byref(d.c()), None, 16, 16, 16, None) == code


def test_quantize_arguments(moe):
    f = moe._lib.moe_quantize_rows
    assert f(None, None, 16, 16, 16, None) == INVALID
    d = ctypes.byref(moe.MoeQuantDesc(4, 64).c())
    for i in range(3):
        a = [16, 16, 16]
        a[i] = None
        assert f(d, None, *a, None) == INVALID
    for a in ((2, 16, 16, 16), (None, 24, 16, 16), (None, 16, 24, 16), (None, 16, 16, 18)):
        assert f(d, *a, None) == ALIGN
    assert f(ctypes.byref(moe.MoeQuantDesc(4, 64, scale_stride=4).c()), None, 16, 16, 20, None) == ALIGN
    assert f(ctypes.byref(moe.MoeQuantDesc(0, 64).c()), None, None, None, None, None) == 0


@pytest.mark.parametrize("name", ["moe_expert_product_i8", "moe_expert_swiglu_i8"])
def test_product_shapes_and_arguments(moe, name):
    f = getattr(moe._lib, name)
    good = dict(num_experts=4, rows=8, in_features=64, out_features=24)
    full = [16] * 7
    for kw in (dict(num_experts=0), dict(num_experts=1025), dict(rows=-1), dict(rows=(1 << 31) - 128), dict(in_features=0),
               dict(in_features=8), dict(in_features=24), dict(in_features=65552), dict(out_features=0), dict(out_features=4),
               dict(out_features=12), dict(out_features=65544), dict(x_stride=48), dict(x_stride=72), dict(x_stride=-16),
               dict(x_stride=1 << 36), dict(x_scale_stride=-1), dict(x_scale_stride=1 << 36)):
        assert f(ctypes.byref(moe.MoeExpertI8Desc(**{**good, **kw}).c()), *full, None) == SHAPE, kw
    d = ctypes.byref(moe.MoeExpertI8Desc(**good).c())
    assert f(None, *full, None) == INVALID
    for i in range(7):
        a = list(full)
        a[i] = None
        assert f(d, *a, None) == INVALID
        a[i] = 24 if i in (0, 4, 6) else 18
        assert f(d, *a, None) == ALIGN
    empty = ctypes.byref(moe.MoeExpertI8Desc(**{**good, "rows": 0}).c())
    assert f(empty, None, None, 16, 16, None, None, None, None) == 0


def test_python_checks_of_quantize(moe):
    q, s = gpu(4, 64), gpu(4, 1, dtype=torch.float32)
    x = gpu(4, 64, dtype=torch.bfloat16)
    call = moe.prepare_quantize_rows
    d = moe.MoeQuantDesc(4, 64)
    assert code_of(moe, call, d, gpu(4, 64, dtype=torch.float32), q, s) == INVALID     # the desc says bf16
    assert code_of(moe, call, d, gpu(4, 64, dtype=torch.float16), q, s) == INVALID
    assert code_of(moe, call, d, torch.zeros(4, 64, dtype=torch.bfloat16), q, s) == INVALID  # not on the GPU
    assert code_of(moe, call, d, x[:3], q, s) == CAPACITY
    assert code_of(moe, call, d, gpu(4, 72, dtype=torch.bfloat16)[:, :64], q, s) == INVALID  # a stride that the desc does not give
    assert code_of(moe, call, d, x, gpu(3, 64), s) == CAPACITY
    assert code_of(moe, call, d, x, gpu(4, 64, dtype=torch.uint8), s) == INVALID
    assert code_of(moe, call, d, x, gpu(4, 128)[:, :64], s) == INVALID
    assert code_of(moe, call, d, x, q, s[:3]) == CAPACITY
    assert code_of(moe, call, moe.MoeQuantDesc(4, 64, scale_stride=4), x, q, s) == CAPACITY
    assert code_of(moe, call, d, x, q, s, gpu(1, dtype=torch.int64)) == INVALID
    assert code_of(moe, call, d, None, q, s) == INVALID


@pytest.mark.parametrize("halves", [1, 2])
def test_python_checks_of_products(moe, halves):
    call = moe.prepare_expert_product_i8 if halves == 1 else moe.prepare_expert_swiglu_i8
    e, r, k, n = 3, 5, 32, 16
    d = moe.MoeExpertI8Desc(e, r, k, n)
    ids = gpu(e, dtype=torch.int32)
    good = dict(x=gpu(r, k), x_scales=gpu(r, dtype=torch.float32), row_begin=ids, row_end=ids, w=gpu(e, halves * n, k),
                w_scales=gpu(e, halves * n, dtype=torch.float32))
    out = gpu(r, n, dtype=torch.bfloat16)
    last = "y" if halves == 1 else "act"
    for name, bad, code in (
            ("x", gpu(r, k, dtype=torch.uint8), INVALID), ("x", gpu(r - 1, k), CAPACITY), ("x", gpu(r, 2 * k)[:, :k], INVALID),
            ("x", torch.zeros(r, k, dtype=torch.int8), INVALID), ("x_scales", gpu(r, dtype=torch.bfloat16), INVALID),
            ("x_scales", gpu(r - 1, dtype=torch.float32), CAPACITY), ("x_scales", gpu(r, 4, dtype=torch.float32)[:, 0], INVALID),
            ("x_scales", gpu(1, dtype=torch.float32).expand(r), INVALID), ("row_begin", gpu(e - 1, dtype=torch.int32), CAPACITY),
            ("row_end", gpu(e, dtype=torch.int64), INVALID), ("w", gpu(e, halves * n - 1, k), CAPACITY),
            ("w", gpu(e, halves * n, k, dtype=torch.uint8), INVALID), ("w", gpu(e, halves * n, 2 * k)[:, :, :k], INVALID),
            ("w_scales", gpu(e, halves * n - 1, dtype=torch.float32), CAPACITY), ("w_scales", None, INVALID), ("x", None, INVALID),
            (last, gpu(r, n, dtype=torch.float32), INVALID), (last, gpu(r - 1, n, dtype=torch.bfloat16), CAPACITY)):
        assert code_of(moe, call, d, **{**good, last: out, name: bad}) == code, name
    # scales [rows, scale_stride] count as the first of each row, at the stride that the desc gives
    four = moe.MoeExpertI8Desc(e, r, k, n, x_scale_stride=4)
    assert code_of(moe, call, d, **{**good, last: out, "x_scales": gpu(r, 4, dtype=torch.float32)}) == INVALID
    assert code_of(moe, call, four, **{**good, last: out, "x_scales": gpu(r, 1, dtype=torch.float32)}) == INVALID
    assert code_of(moe, call, four, **{**good, last: out, "x_scales": gpu(r - 1, 4, dtype=torch.float32)}) == CAPACITY
    strided = moe.MoeExpertI8Desc(e, r, k, n, x_stride=48, x_scale_stride=12)
    assert code_of(moe, call, strided, **{**good, last: out}) == INVALID


def test_layer_checks(moe, monkeypatch):
    from combine_moe_layout_03_gb300.layer import MoeLayer

    def launched(*args, **kw):
        raise AssertionError("launched")

    for name in ("moe_route", "moe_quantize_rows", "moe_layout_dispatch"):
        monkeypatch.setattr(moe, name, launched)
    layer = MoeLayer(64, 32, 4, 2)
    w1, w2 = gpu(4, 64, 64, dtype=torch.bfloat16), gpu(4, 64, 32, dtype=torch.bfloat16)
    assert code_of(moe, layer.quantize, w2, w1) == SHAPE
    assert code_of(moe, layer.quantize, w1[:3], w2) == SHAPE
    experts = (gpu(4, 64, 64), gpu(4, 64, dtype=torch.float32), gpu(4, 64, 32), gpu(4, 64, dtype=torch.float32))
    logits = gpu(6, 4, dtype=torch.float32)
    assert code_of(moe, layer.forward_i8, gpu(6, 128, dtype=torch.bfloat16)[:, :64], logits, experts) == INVALID
    assert code_of(moe, layer.forward_i8, gpu(6, 32, dtype=torch.bfloat16), logits, experts) == SHAPE
