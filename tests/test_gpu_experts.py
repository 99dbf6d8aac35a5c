"""The experts' products against 64-bit sums.

Two kinds of input. Small whole numbers: every sum is exact in fp32, so the
bf16 result is the correctly rounded one, bit for bit. Normal draws: bf16
products are exact and each tensor-core step of 16 of them adds one rounding
or truncation of the running sum (2^-23 of what it holds, at most the sum of
magnitudes), so a sum over K is within (K / 16 + 4) * 2^-23 of the sum of
magnitudes, plus half a step of the output's type."""
import pytest
import torch

from layer_reference import HALF_BF16, kept_values, product, ranges, swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def whole(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(torch.bfloat16)


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def bound(ref, mag, red):
    return HALF_BF16 * ref.abs() + (red / 16 + 4) * 2.0 ** -23 * mag * 1.01 + 1e-30


COUNTS = [
    [1], [128], [129], [0, 3, 0], [5, 0, 127, 128, 1, 300, 0], [0, 0], [1] * 40, [64, 65, 63, 1],
]
SIZES = [(64, 256), (8, 8), (72, 264), (200, 136), (1024, 520), (320, 1000)]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("cin,cout", SIZES)
def test_product_exact(moe, counts, cin, cout):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w = whole(1, max(rows, 1), cin), whole(2, e, cout, cin)
    y = torch.full((max(rows, 1), cout), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product(moe.MoeExpertDesc(e, rows, cin, cout), x, begin, end, w, y)
    if rows:
        assert torch.equal(y, product(x, begin, end, w)[0].to(torch.bfloat16))


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("cin,cout", SIZES)
def test_backward_exact(moe, counts, cin, cout):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    d = moe.MoeExpertDesc(e, rows, cin, cout)
    x, w, dy = whole(1, max(rows, 1), cin), whole(2, e, cout, cin), whole(3, max(rows, 1), cout)
    dx = torch.full((max(rows, 1), cin), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_backward_input(d, dy, begin, end, w, dx)
    if rows:
        ref = product(dy, begin, end, w.transpose(1, 2))[0].to(torch.bfloat16)
        assert torch.equal(dx, ref)
    sums = torch.stack([dy[b:t].double().t() @ x[b:t].double() for b, t in zip(begin.tolist(), end.tolist())])
    dw = torch.full((e, cout, cin), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_backward_weight(d, dy, x, begin, end, dw)
    assert torch.equal(dw, sums.to(torch.bfloat16))
    dw32 = torch.full((e, cout, cin), 7.0, dtype=torch.float32, device=DEV)
    moe.moe_expert_product_backward_weight(d, dy, x, begin, end, dw32, moe.MOE_GRAD_F32)
    assert torch.equal(dw32, sums.float())
    moe.moe_expert_product_backward_weight(d, dy, x, begin, end, dw32, moe.MOE_GRAD_F32_ADD)
    assert torch.equal(dw32, (2 * sums).float())


@pytest.mark.parametrize("rows,e,cin,cout", [(700, 5, 2048, 1024), (40, 8, 7168, 512), (1, 1, 1024, 2048)])
def test_products_of_normal_draws(moe, rows, e, cin, cout):
    counts = [rows // e] * (e - 1)
    counts.append(rows - sum(counts))
    begin, end = ranges(counts, DEV)
    d = moe.MoeExpertDesc(e, rows, cin, cout)
    x, w, dy = normal(1, rows, cin), normal(2, e, cout, cin, scale=cin ** -0.5), normal(3, rows, cout)
    ref, mag = product(x, begin, end, w)
    y = moe.moe_expert_product(d, x, begin, end, w)
    assert bool(((y.double() - ref).abs() <= bound(ref, mag, cin)).all())
    ref, mag = product(dy, begin, end, w.transpose(1, 2))
    dx = moe.moe_expert_product_backward_input(d, dy, begin, end, w)
    assert bool(((dx.double() - ref).abs() <= bound(ref, mag, cout)).all())
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    for i, (b, t) in enumerate(zip(begin.tolist(), end.tolist())):
        a, c = dy[b:t].double(), x[b:t].double()
        ref, mag = a.t() @ c, a.abs().t() @ c.abs()
        lim = ((t - b) / 16 + 4) * 2.0 ** -23 * mag * 1.01 + 1e-30
        assert bool(((dw[i].double() - ref).abs() <= lim).all())


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("counts", [[1], [130, 0, 5], [0, 300, 1, 128]], ids=str)
@pytest.mark.parametrize("cin,f", [(64, 128), (256, 8), (136, 200), (512, 384), (72, 136)])
def test_expert_swiglu(moe, train, counts, cin, f):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w = normal(1, rows, cin), normal(2, e, 2 * f, cin, scale=2 * cin ** -0.5)
    gd = moe.MoeGluDesc(rows, f)
    ckpt, scales = moe.swiglu_checkpoint(gd, DEV) if train else (None, None)
    act = moe.moe_expert_swiglu(moe.MoeExpertDesc(e, rows, cin, f), x, begin, end, w, None, ckpt, scales)
    v, mag = product(x, begin, end, w)
    off = (cin / 16 + 4) * 2.0 ** -23 * mag * 1.01  # of gate and up before the activation
    g, u, og, ou = v[:, :f], v[:, f:], off[:, :f], off[:, f:]
    ref = swiglu(g, u)
    # |silu'| <= 1.1; __expf and the division stay within 2^-18 for |g| < 32
    lim = HALF_BF16 * ref.abs() + 1.1 * og * u.abs() + g.abs() * ou + 2.0 ** -18 * ref.abs() + 1e-30
    assert bool(((act.double() - ref).abs() <= lim).all())
    if not train:
        return
    groups = gd.groups
    for h, (val, o) in enumerate(((g, og), (u, ou))):
        sc = scales[:, h * groups:(h + 1) * groups].double()
        for q in range(groups):
            part, po = val[:, q * 128:(q + 1) * 128], o[:, q * 128:(q + 1) * 128]
            amax = part.abs().amax(1).clamp(min=1e-4)
            assert bool(((sc[:, q] * 448 - amax).abs() <= po.amax(1) + 2.0 ** -22 * amax).all())
        got = kept_values(ckpt[:, h * f:(h + 1) * f], scales[:, h * groups:(h + 1) * groups], f)
        step = sc.repeat_interleave(128, 1)[:, :f] * 2.0 ** -10  # half of the smallest step
        assert bool(((got - val).abs() <= (2.0 ** -4 * val.abs()).maximum(step) * 1.001 + o).all())


def test_rows_from_records_and_untouched_rows(moe):
    # rows read out of padded records, ranges out of order, a gap, and limits past the buffer
    rows, cin, cout, pad = 300, 136, 264, 40
    rec = whole(5, rows, cin + pad)
    x = rec[:, pad:]
    begin = torch.tensor([200, 10, 50, 290, -5], dtype=torch.int32, device=DEV)
    end = torch.tensor([250, 30, 50, 1000, 4], dtype=torch.int32, device=DEV)
    w, dy = whole(6, 5, cout, cin), whole(7, rows, cout)
    d = moe.MoeExpertDesc(5, rows, cin, cout, x_stride=x.stride(0))
    y = torch.full((rows, cout), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product(d, x, begin, end, w, y)
    b, t = begin.clamp(min=0), end.clamp(max=rows)
    ref = product(x, b, t, w)[0].to(torch.bfloat16)
    inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for lo, hi in zip(b.tolist(), t.tolist()):
        inside[lo:hi] = True
    assert torch.equal(y[inside], ref[inside]) and bool((y[~inside] == 9.0).all())
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    for e, (lo, hi) in enumerate(zip(b.tolist(), t.tolist())):
        assert torch.equal(dw[e], (dy[lo:hi].double().t() @ x[lo:hi].double()).float())


def test_other_experts_rows_do_not_leak(moe):
    # infinities and NaN in one expert's rows stay out of the others' results
    counts, cin, cout = [70, 3, 60], 72, 136
    begin, end = ranges(counts, DEV)
    x, w, dy = whole(1, 133, cin), whole(2, 3, cout, cin), whole(3, 133, cout)
    x[70:73] = float("inf")
    dy[70:73] = float("nan")
    d = moe.MoeExpertDesc(3, 133, cin, cout)
    y = moe.moe_expert_product(d, x, begin, end, w)
    dw = moe.moe_expert_product_backward_weight(d, dy, x, begin, end)
    clean = torch.ones(133, dtype=torch.bool, device=DEV)
    clean[70:73] = False
    assert bool(torch.isfinite(y[clean]).all()) and bool(torch.isfinite(dw[[0, 2]]).all())
    assert torch.equal(dw[2], (dy[73:].double().t() @ x[73:].double()).to(torch.bfloat16))


def test_gradients_against_differences(moe):
    # L = sum(c * y): its differences along random directions of x and w, in 64 bits
    counts, cin, cout = [40, 0, 25], 128, 72
    begin, end = ranges(counts, DEV)
    x, w, c = normal(1, 65, cin), normal(2, 3, cout, cin, scale=0.1), normal(3, 65, cout)
    d = moe.MoeExpertDesc(3, 65, cin, cout)
    dx = moe.moe_expert_product_backward_input(d, c, begin, end, w).double()
    dw = moe.moe_expert_product_backward_weight(d, c, x, begin, end, grad_kind=moe.MOE_GRAD_F32).double()
    vx, vw = normal(4, 65, cin).double(), normal(5, 3, cout, cin).double()
    loss = lambda a, b: (c.double() * product(a, begin, end, b)[0]).sum()  # noqa: E731
    h = 2.0 ** -10
    by_x = (loss(x.double() + h * vx, w.double()) - loss(x.double() - h * vx, w.double())) / (2 * h)
    by_w = (loss(x.double(), w.double() + h * vw) - loss(x.double(), w.double() - h * vw)) / (2 * h)
    assert abs((dx * vx).sum() - by_x) <= HALF_BF16 * (dx * vx).abs().sum()
    assert abs((dw * vw).sum() - by_w) <= 2.0 ** -18 * (dw * vw).abs().sum()


def test_graph_replay_follows_the_ranges(moe):
    rows, e, cin, cout = 200, 4, 128, 256
    x, w = whole(1, rows, cin), whole(2, e, cout, cin)
    begin, end = ranges([50, 50, 50, 50], DEV)
    y = torch.zeros(rows, cout, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    call = moe.prepare_expert_product(moe.MoeExpertDesc(e, rows, cin, cout), x, begin, end, w, y, stream=s)
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    b2, e2 = ranges([0, 130, 7, 63], DEV)
    begin.copy_(b2)
    end.copy_(e2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, product(x, begin, end, w)[0].to(torch.bfloat16))


def test_same_inputs_same_bits(moe):
    counts = [37, 200, 0, 64]
    begin, end = ranges(counts, DEV)
    x, dy = normal(1, 301, 520), normal(2, 301, 264)
    d = moe.MoeExpertDesc(4, 301, 520, 264)
    a = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    b = moe.moe_expert_product_backward_weight(d, dy, x, begin, end, grad_kind=moe.MOE_GRAD_F32)
    assert torch.equal(a, b)


def test_behind_a_kernel_that_fills_the_gpu(moe):
    # calls queued without a pause: the product's pairs of blocks start while
    # blocks of the kernel before still hold part of each SM
    rows, cin, f = 4096, 256, 2048
    begin, end = ranges([1000, 0, 3001, 95], DEV)
    x, w = normal(1, rows, cin), normal(2, 4, 2 * f, cin, scale=cin ** -0.5)
    d, gd = moe.MoeExpertDesc(4, rows, cin, f), moe.MoeGluDesc(rows, f)
    act = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)
    ckpt, scales = moe.swiglu_checkpoint(gd, DEV)
    da, dgu = normal(3, rows, f), torch.empty(rows, 2 * f, dtype=torch.bfloat16, device=DEV)
    again = torch.empty_like(act)
    calls = [moe.prepare_expert_swiglu(d, x, begin, end, w, act, ckpt, scales),
             moe.prepare_swiglu_backward(gd, ckpt, scales, da, dgu, again)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    first = [t.clone() for t in (act, ckpt, dgu, again)]
    for _ in range(100):
        for call in calls:
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (act, ckpt, dgu, again)))


def test_waits_that_run_out_leave_the_context_usable(moe):
    begin, end = ranges([300, 129], DEV)
    x, w = whole(1, 429, 1024), whole(2, 2, 520, 1024)
    d = moe.MoeExpertDesc(2, 429, 1024, 520)
    torch.cuda.synchronize()
    moe.moe_set_wait_limit_ns(1)
    try:
        moe.moe_expert_product(d, x, begin, end, w)
        assert moe.moe_device_status() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_wait_limit_ns(0)
    y = moe.moe_expert_product(d, x, begin, end, w)
    assert moe.moe_device_status() == moe.MOE_OK
    assert torch.equal(y, product(x, begin, end, w)[0].to(torch.bfloat16))


def test_beside_other_work_on_another_stream(moe):
    # blocks of another stream's kernels come and go on the same SMs
    counts, cin, cout = [300, 0, 129, 71], 512, 768
    begin, end = ranges(counts, DEV)
    x, w, dy = whole(1, 500, cin), whole(2, 4, cout, cin), whole(3, 500, cout)
    d = moe.MoeExpertDesc(4, 500, cin, cout)
    want = product(x, begin, end, w)[0].to(torch.bfloat16)
    y = torch.zeros(500, cout, dtype=torch.bfloat16, device=DEV)
    dw = torch.zeros(4, cout, cin, device=DEV)
    sums = torch.stack([dy[b:t].double().t() @ x[b:t].double() for b, t in zip(begin.tolist(), end.tolist())]).float()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    noise = torch.randn(1 << 22, device=DEV)
    torch.cuda.synchronize()
    calls = [moe.prepare_expert_product(d, x, begin, end, w, y, stream=mine),
             moe.prepare_expert_product_backward_weight(d, dy, x, begin, end, dw, moe.MOE_GRAD_F32, stream=mine)]
    for _ in range(30):
        with torch.cuda.stream(other):
            for _ in range(4):
                noise.mul_(1.0001)
        for call in calls:
            call()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(dw, sums)
