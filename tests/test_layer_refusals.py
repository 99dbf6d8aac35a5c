"""What the router, the gated activation and the experts' products refuse,
before anything is launched (no GPU)."""
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


def route_desc(moe, **kw):
    base = dict(num_tokens=8, num_experts=16, topk=2, num_groups=4, topk_groups=2)
    base.update(kw)
    return moe.MoeRouteDesc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), SHAPE), (dict(num_experts=0), SHAPE), (dict(num_experts=1028, num_groups=4), SHAPE),
    (dict(topk=0), SHAPE), (dict(topk=33, num_experts=1024), SHAPE), (dict(num_groups=0), SHAPE), (dict(num_groups=3), SHAPE),
    (dict(num_groups=64, num_experts=128), SHAPE), (dict(topk_groups=0), SHAPE), (dict(topk_groups=5), SHAPE),
    (dict(topk=9), SHAPE), (dict(logits_stride=15), SHAPE), (dict(logits_stride=-1), SHAPE), (dict(num_tokens=1 << 30), SHAPE),
    (dict(score=2), INVALID), (dict(group_score=2), INVALID), (dict(logits_kind=2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID)])
def test_route_shapes(moe, kw, code):
    d = ctypes.byref(route_desc(moe, **kw).c())
    assert moe._lib.moe_route(d, 16, None, 16, 16, None) == code
    assert moe._lib.moe_route_backward(d, 16, 16, 16, 16, None) == code


def test_route_arguments(moe):
    f32, bf16 = route_desc(moe).c(), route_desc(moe, logits_kind=moe.MOE_LOGITS_BF16).c()
    f, b = moe._lib.moe_route, moe._lib.moe_route_backward
    assert f(None, 16, None, 16, 16, None) == INVALID and b(None, 16, 16, 16, 16, None) == INVALID
    for i in (0, 2, 3):
        a = [16, None, 16, 16]
        a[i] = None
        assert f(ctypes.byref(f32), *a, None) == INVALID
    for i, v in ((0, 18), (1, 2), (2, 18), (3, 17)):
        a = [16, 16, 16, 16]
        a[i] = v
        assert f(ctypes.byref(f32), *a, None) == ALIGN
    assert f(ctypes.byref(bf16), 17, None, 16, 16, None) == ALIGN
    for i in range(4):
        a = [16] * 4
        a[i] = None
        assert b(ctypes.byref(f32), *a, None) == INVALID
        a[i] = 18
        assert b(ctypes.byref(f32), *a, None) == ALIGN
    assert f(ctypes.byref(route_desc(moe, num_tokens=0).c()), None, None, None, None, None) == 0
    assert b(ctypes.byref(route_desc(moe, num_tokens=0).c()), None, None, None, None, None) == 0


def test_swiglu_arguments(moe):
    f, b = moe._lib.moe_swiglu, moe._lib.moe_swiglu_backward
    for rows, width in ((-1, 8), (1 << 31, 8), (1, 0), (1, 4), (1, 12), (1, 65544)):
        d = ctypes.byref(moe.MoeGluDesc(rows, width).c())
        assert f(d, None, 16, 16, 16, 16, None) == SHAPE and b(d, None, 16, 16, 16, 16, 16, None) == SHAPE
    d = ctypes.byref(moe.MoeGluDesc(4, 64).c())
    assert f(None, None, 16, 16, 16, 16, None) == INVALID and b(None, None, 16, 16, 16, 16, 16, None) == INVALID
    assert f(d, None, None, 16, 16, 16, None) == INVALID       # no input
    assert f(d, None, 16, None, None, None, None) == INVALID   # nothing to write
    assert f(d, None, 16, 16, 16, None, None) == INVALID       # codes without scales
    assert f(d, None, 16, 16, None, 16, None) == INVALID
    for a in ((2, 16, 16, 16, 16), (None, 24, 16, 16, 16), (None, 16, 24, 16, 16), (None, 16, 16, 20, 16), (None, 16, 16, 16, 18)):
        assert f(d, *a, None) == ALIGN
    for i in range(4):
        a = [16] * 5
        a[i] = None
        assert b(d, None, *a, None) == INVALID
    for i, v in ((0, 12), (1, 18), (2, 24), (3, 24), (4, 24)):
        a = [16] * 5
        a[i] = v
        assert b(d, None, *a, None) == ALIGN
    zero = ctypes.byref(moe.MoeGluDesc(0, 64).c())
    assert f(zero, None, None, None, None, None, None) == 0 and b(zero, None, None, None, None, None, None, None) == 0


def expert_calls(moe, d):
    lib = moe._lib
    return [lambda a: lib.moe_expert_product(d, *a[:5], None), lambda a: lib.moe_expert_swiglu(d, *a[:5], 16, 16, None),
            lambda a: lib.moe_expert_product_backward_input(d, *a[:5], None),
            lambda a: lib.moe_expert_product_backward_weight(d, a[0], a[3], a[1], a[2], a[4], moe.MOE_GRAD_F32, None)]


@pytest.mark.parametrize("kw", [
    dict(num_experts=0), dict(num_experts=1025), dict(rows=-1), dict(rows=(1 << 31) - 128), dict(in_features=4), dict(in_features=20),
    dict(in_features=65544), dict(out_features=0), dict(out_features=65544), dict(out_features=12), dict(x_stride=56),
    dict(x_stride=68), dict(x_stride=-64), dict(x_stride=1 << 36)])
def test_expert_shapes(moe, kw):
    base = dict(num_experts=2, rows=4, in_features=64, out_features=64)
    base.update(kw)
    for call in expert_calls(moe, ctypes.byref(moe.MoeExpertDesc(**base).c())):
        assert call([16] * 5) == SHAPE


def test_expert_arguments(moe):
    d = ctypes.byref(moe.MoeExpertDesc(2, 4, 64, 64).c())
    for call in expert_calls(moe, None):
        assert call([16] * 5) == INVALID
    for call in expert_calls(moe, d):
        for i in range(5):
            a = [16] * 5
            a[i] = None
            assert call(a) == INVALID
            a[i] = 18 if i in (1, 2) else 24
            assert call(a) == ALIGN
    lib = moe._lib
    assert lib.moe_expert_swiglu(d, 16, 16, 16, 16, 16, 16, None, None) == INVALID  # codes without scales
    assert lib.moe_expert_swiglu(d, 16, 16, 16, 16, 16, None, 16, None) == INVALID
    assert lib.moe_expert_swiglu(d, 16, 16, 16, 16, 16, 20, 16, None) == ALIGN
    assert lib.moe_expert_swiglu(d, 16, 16, 16, 16, 16, 16, 18, None) == ALIGN
    assert lib.moe_expert_product_backward_weight(d, 16, 16, 16, 16, 16, 3, None) == INVALID
    zero = ctypes.byref(moe.MoeExpertDesc(2, 0, 64, 64).c())
    assert lib.moe_expert_product(zero, None, 16, 16, None, None, None) == 0
    assert lib.moe_expert_product_backward_weight(zero, None, None, 16, 16, None, 0, None) == INVALID
    assert lib.moe_expert_product_backward_weight(zero, None, None, 16, 16, 16, moe.MOE_GRAD_F32_ADD, None) == 0


def test_python_refuses_tensors_that_do_not_fit(moe):
    # CPU tensors, wrong types and missing buffers never reach the library
    x = torch.zeros(8, 16)
    with pytest.raises(moe.MoeError) as err:
        moe.prepare_route(route_desc(moe), x, None, None, None, stream=0)
    assert err.value.code == INVALID
    with pytest.raises(moe.MoeError):
        moe.prepare_swiglu(moe.MoeGluDesc(4, 64), torch.zeros(4, 128), None, stream=0)
    with pytest.raises(moe.MoeError):
        moe.prepare_expert_product(moe.MoeExpertDesc(2, 4, 64, 64), x, None, None, None, None, stream=0)
