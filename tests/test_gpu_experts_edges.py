"""The experts' products where blocks, warps and ranges meet: ragged ends
beside rows that are not finite, ranges outside the buffers, waits. Inputs are
small whole numbers, so every sum is exact (see test_gpu_experts)."""
import pytest
import torch

from layer_reference import ranges
from test_gpu_experts import DEV, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def sums(dy, x, begin, end):
    return torch.stack([dy[b:t].double().t() @ x[b:t].double() for b, t in zip(begin.tolist(), end.tolist())])


@pytest.mark.parametrize("cin,cout", [(520, 264), (1024, 768)])
def test_ragged_ends_beside_rows_that_are_not_finite(moe, cin, cout):
    # every second expert's rows are NaN or infinite; the others' reductions end
    # inside 16 rows that reach into them, in many tiles of every pair of blocks
    g = torch.Generator().manual_seed(1)
    counts = [int(torch.randint(1, 200, (), generator=g)) // 16 * 16 + 1 + i % 15 for i in range(64)]
    begin, end = ranges(counts, DEV)
    rows = sum(counts)
    x, dy = whole(1, rows, cin), whole(2, rows, cout)
    for e in range(1, 64, 2):
        x[begin[e]:end[e]] = float("nan") if e % 4 == 1 else float("inf")
        dy[begin[e]:end[e]] = float("inf") if e % 4 == 1 else float("nan")
    d = moe.MoeExpertDesc(64, rows, cin, cout)
    want = sums(dy, x, begin, end)[::2]
    for kind, t in ((moe.MOE_GRAD_F32, torch.float32), (moe.MOE_GRAD_BF16, torch.bfloat16)):
        dw = torch.empty(64, cout, cin, dtype=t, device=DEV)
        call = moe.prepare_expert_product_backward_weight(d, dy, x, begin, end, dw, kind)
        for _ in range(20):
            dw.fill_(7.0)
            call()
            assert torch.equal(dw[::2], want.to(t))


def test_ranges_that_end_far_below_zero(moe):
    # such an expert has no rows, whatever its begin is
    rows, cin, cout, least = 100, 72, 144, -(1 << 31)
    begin = torch.tensor([5, 0, 99, (1 << 31) - 1, -7], dtype=torch.int32, device=DEV)
    end = torch.tensor([least, 60, least + 50, least, least + 1], dtype=torch.int32, device=DEV)
    x, w, dy = whole(1, rows, cin), whole(2, 5, cout, cin), whole(3, rows, cout)
    d = moe.MoeExpertDesc(5, rows, cin, cout)
    y = torch.full((rows, cout), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product(d, x, begin, end, w, y)
    assert torch.equal(y[:60], (x[:60].double() @ w[1].double().t()).to(torch.bfloat16)) and bool((y[60:] == 7.0).all())
    dx = torch.full((rows, cin), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_backward_input(d, dy, begin, end, w, dx)
    assert torch.equal(dx[:60], (dy[:60].double() @ w[1].double()).to(torch.bfloat16)) and bool((dx[60:] == 7.0).all())
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    want = torch.zeros_like(dw)
    want[1] = (dy[:60].double().t() @ x[:60].double()).float()
    assert torch.equal(dw, want)
    act = torch.full((rows, cout // 2), 7.0, dtype=torch.bfloat16, device=DEV)
    ckpt, scales = moe.swiglu_checkpoint(moe.MoeGluDesc(rows, cout // 2), DEV)
    scales.fill_(-1.0)
    moe.moe_expert_swiglu(moe.MoeExpertDesc(5, rows, cin, cout // 2), x, begin, end, w, act, ckpt, scales)
    assert bool((act[60:] == 7.0).all()) and bool((scales[60:] == -1.0).all()) and bool((scales[:60] > 0).all())


def test_a_long_reduction_outlasts_the_budget_of_a_wait(moe):
    # a million rows of one expert take several times the budget; the ragged
    # expert that the same pair of blocks comes to last waits for two such
    long, e = 1 << 20, 153
    counts = [0] * e
    counts[0] = counts[76] = long
    counts[152] = 5
    begin, end = ranges(counts, DEV)
    x, dy = whole(1, sum(counts), 8), whole(2, sum(counts), 8)
    dw = torch.full((e, 8, 8), 7.0, device=DEV)
    want = sums(dy, x, begin, end).float()
    torch.cuda.synchronize()
    moe.moe_set_wait_limit_ns(1_000_000)
    try:
        moe.moe_expert_product_backward_weight(moe.MoeExpertDesc(e, sum(counts), 8, 8), dy, x, begin, end, dw, moe.MOE_GRAD_F32)
        assert moe.moe_device_status() == moe.MOE_OK
    finally:
        moe.moe_set_wait_limit_ns(0)
    assert torch.equal(dw, want)


def test_a_weight_gradient_without_a_buffer(moe):
    # experts without rows get zeros whatever the memory held; added to nothing is written
    counts = [37, 0, 130, 0]
    begin, end = ranges(counts, DEV)
    x, dy = whole(1, 167, 72), whole(2, 167, 136)
    d = moe.MoeExpertDesc(4, 167, 72, 136)
    want = sums(dy, x, begin, end)
    for kind, t in ((moe.MOE_GRAD_BF16, torch.bfloat16), (moe.MOE_GRAD_F32, torch.float32), (moe.MOE_GRAD_F32_ADD, torch.float32)):
        for _ in range(3):
            junk = torch.full((4, 136, 72), float("nan"), dtype=t, device=DEV)
            del junk
            dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=kind)
            assert torch.equal(dw, want.to(t))
    none = moe.MoeExpertDesc(4, 0, 72, 136)
    dw = moe.moe_expert_product_backward_weight(none, None, None, begin, end, grad_kind=moe.MOE_GRAD_F32_ADD)
    assert bool((dw == 0).all())
