"""The gated activation, its checkpoint and the backward from it, against
64-bit forms.

The checkpoint follows the format's fp32 rule, so its codes and scales are
equal bit for bit. act and the gradients are fp32 from about a dozen
operations with __expf (argument error |g| * 2^-24, so under 2^-18 relative
for |g| < 32) and one rounding to bf16; grad_gate has a difference in it,
whose terms are at most |grad * up * sig| * (1 + |g|)."""
import pytest
import torch

from layer_reference import HALF_BF16, kept, kept_values, near, swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROUGH = 2.0 ** -18


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    return m


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def check(moe, gu, da, num_rows=None):
    rows, f = gu.shape[0], gu.shape[1] // 2
    d = moe.MoeGluDesc(rows, f)
    n = d.groups
    act = torch.full((rows, f), 5.0, dtype=torch.bfloat16, device=DEV)
    ckpt = torch.full((rows, 2 * f), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, 2 * n), -3.0, device=DEV)
    count = None if num_rows is None else torch.tensor([num_rows], dtype=torch.int32, device=DEV)
    moe.moe_swiglu(d, gu, act, ckpt, scales, count)
    p = rows if num_rows is None else max(0, min(num_rows, rows))
    g, u = gu[:p, :f].float(), gu[:p, f:].float()
    for h, v in enumerate((g, u)):
        codes, sc = kept(v)
        assert torch.equal(ckpt[:p, h * f:(h + 1) * f], codes.view(torch.uint8))
        assert torch.equal(scales[:p, h * n:(h + 1) * n], sc)
    ref = swiglu(g.double(), u.double())
    assert near(act[:p], ref, (HALF_BF16 + ROUGH) * ref.abs() + 1e-37)
    assert bool((act[p:] == 5.0).all()) and bool((ckpt[p:] == 0x55).all()) and bool((scales[p:] == -3.0).all())
    plain = torch.empty_like(act)
    moe.moe_swiglu(d, gu, plain, num_rows=count)
    assert torch.equal(plain[:p], act[:p])
    # backward from the checkpoint
    dgu = torch.full((rows, 2 * f), 5.0, dtype=torch.bfloat16, device=DEV)
    again = torch.full((rows, f), 5.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_swiglu_backward(d, ckpt, scales, da, dgu, again, count)
    g = kept_values(ckpt[:p, :f].contiguous(), scales[:p, :n], f)
    u = kept_values(ckpt[:p, f:].contiguous(), scales[:p, n:], f)
    sig, a = torch.sigmoid(g), da[:p].double()
    terms = (a * u * sig).abs() * (1 + g.abs())
    ref = a * u * sig * (1 + g * (1 - sig))
    assert near(dgu[:p, :f], ref, HALF_BF16 * ref.abs() + ROUGH * terms + 1e-37)
    ref = a * g * sig
    assert near(dgu[:p, f:], ref, (HALF_BF16 + ROUGH) * ref.abs() + 1e-37)
    ref = swiglu(g, u)
    assert near(again[:p], ref, (HALF_BF16 + ROUGH) * ref.abs() + 1e-37)
    assert bool((dgu[p:] == 5.0).all()) and bool((again[p:] == 5.0).all())
    lean = torch.empty_like(dgu)
    moe.moe_swiglu_backward(d, ckpt, scales, da, lean, num_rows=count)
    assert torch.equal(lean[:p], dgu[:p])


@pytest.mark.parametrize("rows,f", [(1, 8), (1, 128), (3, 136), (77, 1000), (5, 120), (2, 2048), (300, 384), (7, 16), (1, 65536), (1000, 264)])
def test_forward_and_backward(moe, rows, f):
    check(moe, normal(1, rows, 2 * f, scale=2.0), normal(2, rows, f))


@pytest.mark.parametrize("num_rows", [-4, 0, 1, 13, 40, 41])
def test_row_count_on_the_device(moe, num_rows):
    check(moe, normal(1, 40, 400), normal(2, 40, 200), num_rows)


def test_extreme_values(moe):
    gu = normal(3, 6, 512)
    gu[0] = 0.0
    gu[1] = 1e-6
    gu[2] *= 1e4
    gu[3, :256] = -90.0
    gu[4, :256] = 90.0
    gu[5, 7] = 3e38
    check(moe, gu, normal(4, 6, 256))


def test_no_rows(moe):
    d = moe.MoeGluDesc(0, 64)
    empty = torch.empty(0, dtype=torch.bfloat16, device=DEV)
    moe.moe_swiglu(d, empty, empty)
    moe.moe_swiglu_backward(d, torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(0, device=DEV), empty, empty)


def test_gradient_against_differences(moe):
    # differences of the activation at the kept values, in 64 bits
    rows, f = 9, 264
    gu, da = normal(5, rows, 2 * f), normal(6, rows, f)
    d = moe.MoeGluDesc(rows, f)
    ckpt, scales = moe.swiglu_checkpoint(d, DEV)
    moe.moe_swiglu(d, gu, None, ckpt, scales)
    got = moe.moe_swiglu_backward(d, ckpt, scales, da).double()
    n = d.groups
    x = torch.cat([kept_values(ckpt[:, :f].contiguous(), scales[:, :n], f), kept_values(ckpt[:, f:].contiguous(), scales[:, n:], f)], 1)
    v = normal(7, rows, 2 * f).double()
    loss = lambda a: (swiglu(a[:, :f], a[:, f:]) * da.double()).sum()  # noqa: E731
    h = 1e-5
    by = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
    assert abs((got * v).sum() - by) <= (HALF_BF16 + 1e-6) * (got * v).abs().sum()
