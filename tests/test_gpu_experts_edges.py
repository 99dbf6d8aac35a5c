"""The experts' products where blocks, warps and ranges meet: ragged ends
beside rows that are not finite, ranges outside the buffers, waits. Inputs are
small whole numbers, so every sum is exact (see test_gpu_experts)."""
import pytest
import torch

from layer_reference import HALF_BF16, kept_values, product, ranges, swiglu
from test_gpu_experts import DEV, normal, whole

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


@pytest.mark.parametrize("counts", [[128] * 256, [i % 6 for i in range(1024)], [300, 0, 1, 500, 257] * 12], ids=["256x128", "1024", "60"])
def test_many_experts(moe, counts):
    e, rows, cin, cout = len(counts), sum(counts), 136, 264
    begin, end = ranges(counts, DEV)
    x, w, dy = whole(1, rows, cin), whole(2, e, cout, cin), whole(3, rows, cout)
    d = moe.MoeExpertDesc(e, rows, cin, cout)
    assert torch.equal(moe.moe_expert_product(d, x, begin, end, w), product(x, begin, end, w)[0].to(torch.bfloat16))
    ref = product(dy, begin, end, w.transpose(1, 2))[0].to(torch.bfloat16)
    assert torch.equal(moe.moe_expert_product_backward_input(d, dy, begin, end, w), ref)
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    assert torch.equal(dw, sums(dy, x, begin, end).float())


def test_rows_of_fixed_capacity_buffers(moe):
    # expert e owns [e * capacity, e * capacity + count[e]); what lies behind is left alone and not read
    capacity, cin, cout = 96, 72, 136
    count = torch.tensor([96, 0, 5, 64, 33], dtype=torch.int32, device=DEV)
    begin = torch.arange(5, dtype=torch.int32, device=DEV) * capacity
    end = begin + count
    rows = 5 * capacity
    inside = (torch.arange(rows, device=DEV) % capacity) < count.repeat_interleave(capacity)
    x, w, dy = whole(1, rows, cin), whole(2, 5, cout, cin), whole(3, rows, cout)
    x[~inside], dy[~inside] = float("nan"), float("inf")
    d = moe.MoeExpertDesc(5, rows, cin, cout)
    y = torch.full((rows, cout), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product(d, x, begin, end, w, y)
    assert torch.equal(y[inside], product(x, begin, end, w)[0].to(torch.bfloat16)[inside]) and bool((y[~inside] == 7.0).all())
    dx = torch.full((rows, cin), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_backward_input(d, dy, begin, end, w, dx)
    assert torch.equal(dx[inside], product(dy, begin, end, w.transpose(1, 2))[0].to(torch.bfloat16)[inside])
    assert bool((dx[~inside] == 7.0).all())
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end)
    assert torch.equal(dw, sums(dy, x, begin, end).to(torch.bfloat16))


@pytest.mark.parametrize("call", ["swiglu", "checkpoint", "input", "weight", "weight_add"])
def test_every_product_gives_up_in_time(moe, call):
    # as for the plain product: with no time to wait the kernel says so and ends
    counts, cin, f = [300, 129, 777], 1024, 256
    begin, end = ranges(counts, DEV)
    rows = sum(counts)
    x, w, dy = whole(1, rows, cin), whole(2, 3, 2 * f, cin), whole(3, rows, 2 * f)
    d = moe.MoeExpertDesc(3, rows, cin, 2 * f)
    dw = torch.zeros(3, 2 * f, cin, device=DEV)
    ckpt = moe.swiglu_checkpoint(moe.MoeGluDesc(rows, f), DEV) if call == "checkpoint" else (None, None)
    run = {"swiglu": lambda: moe.moe_expert_swiglu(moe.MoeExpertDesc(3, rows, cin, f), x, begin, end, w),
           "checkpoint": lambda: moe.moe_expert_swiglu(moe.MoeExpertDesc(3, rows, cin, f), x, begin, end, w, None, *ckpt),
           "input": lambda: moe.moe_expert_product_backward_input(d, dy, begin, end, w),
           "weight": lambda: moe.moe_expert_product_backward_weight(d, dy, x, begin, end),
           "weight_add": lambda: moe.moe_expert_product_backward_weight(d, dy, x, begin, end, dw.zero_(), moe.MOE_GRAD_F32_ADD)}[call]
    want = run().clone()
    torch.cuda.synchronize()
    moe.moe_set_wait_limit_ns(1)
    try:
        run()
        assert moe.moe_device_status() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_wait_limit_ns(0)
    again = run()
    assert moe.moe_device_status() == moe.MOE_OK and torch.equal(again, want)


def test_the_activation_over_many_tiles(moe):
    # several tiles a pair of blocks, whose rows differ by up to 2^10 in size, so that a largest magnitude or scale of
    # another tile shows; bounds as in test_gpu_experts
    counts, cin, f = [1500, 37, 0, 2000, 700], 136, 2048
    begin, end = ranges(counts, DEV)
    rows = sum(counts)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    size = torch.exp2(torch.randint(-9, 2, (rows // 32 + 1, 1), generator=g, device=DEV).float()).repeat_interleave(32, 0)[:rows]
    x = (torch.randn(rows, cin, generator=g, device=DEV) * size).to(torch.bfloat16)
    w = normal(8, 5, 2 * f, cin, scale=2 * cin ** -0.5)
    gd = moe.MoeGluDesc(rows, f)
    ckpt, scales = moe.swiglu_checkpoint(gd, DEV)
    act = moe.moe_expert_swiglu(moe.MoeExpertDesc(5, rows, cin, f), x, begin, end, w, None, ckpt, scales)
    v, mag = product(x, begin, end, w)
    off = (cin / 16 + 4) * 2.0 ** -23 * mag * 1.01
    a, u, ao, uo = v[:, :f], v[:, f:], off[:, :f], off[:, f:]
    ref = swiglu(a, u)
    lim = HALF_BF16 * ref.abs() + 1.1 * ao * u.abs() + a.abs() * uo + 2.0 ** -18 * ref.abs() + 1e-30
    assert bool(((act.double() - ref).abs() <= lim).all())
    groups = gd.groups
    for h, (val, o) in enumerate(((a, ao), (u, uo))):
        sc = scales[:, h * groups:(h + 1) * groups].double()
        most = val.view(rows, groups, 128).abs().amax(2).clamp(min=1e-4)
        assert bool(((sc * 448 - most).abs() <= o.view(rows, groups, 128).amax(2) + 2.0 ** -22 * most).all())
        got = kept_values(ckpt[:, h * f:(h + 1) * f], scales[:, h * groups:(h + 1) * groups], f)
        step = sc.repeat_interleave(128, 1) * 2.0 ** -10
        assert bool(((got - val).abs() <= (2.0 ** -4 * val.abs()).maximum(step) * 1.001 + o).all())
    assert torch.equal(act, moe.moe_expert_swiglu(moe.MoeExpertDesc(5, rows, cin, f), x, begin, end, w))


def test_infinity_and_nan_in_a_fused_checkpoint(moe):
    # an infinity takes its group of 128 with it, NaN only itself
    rows, cin, f = 40, 64, 384
    begin, end = ranges([rows], DEV)
    x = whole(1, rows, cin).abs() + 1.0
    w = whole(2, 1, 2 * f, cin)
    w[0, 5, 0] = float("inf")           # gate, group 0
    w[0, 130, 3] = float("nan")         # gate, group 1
    w[0, f + 300, 1] = -float("inf")    # up, group 2
    ckpt, scales = moe.swiglu_checkpoint(moe.MoeGluDesc(rows, f), DEV)
    act = moe.moe_expert_swiglu(moe.MoeExpertDesc(1, rows, cin, f), x, begin, end, w, None, ckpt, scales)
    v = (x.double() @ w[0].double().t()).float()  # whole numbers: exact
    want = torch.nan_to_num(v, nan=0.0, posinf=float("inf"), neginf=-float("inf")).abs().view(rows, 6, 128).amax(2).clamp(min=1e-4)
    # (quotients by a tensor: by a number they are not IEEE divisions on the GPU)
    assert torch.equal(scales, want / torch.full_like(want, 448.0))
    codes = ckpt.view(torch.float8_e4m3fn).float()
    bad = torch.isnan(codes)
    where = torch.zeros(2 * f, dtype=torch.bool, device=DEV)
    where[[5, 130, f + 300]] = True
    assert torch.equal(bad, where.expand(rows, -1))
    assert bool((codes[:, :128][:, ~where[:128]] == 0).all()) and bool((codes[:, f + 256:][:, ~where[f + 256:]] == 0).all())
    keep = ~where
    keep[:128] = keep[f + 256:] = False
    # of 448 / a and its product with a value each rounds once; 2^-4 half a step, 2^-10 of 448 / 448 below the smallest
    kept = codes.double() * scales.double().repeat_interleave(128, 1)
    lim = (2.0 ** -4 * v.abs().double()).maximum(scales.double().repeat_interleave(128, 1) * 2.0 ** -10) * 1.001
    assert bool(((kept - v.double()).abs() <= lim)[:, keep].all())
    bad = torch.isnan(act)
    assert bool(bad[:, 130].all()) and not bool(bad[:, [c for c in range(f) if c not in (5, 130, 300)]].any())
