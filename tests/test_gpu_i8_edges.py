"""The 8-bit calls where they can go wrong: few rows (a kernel of their own),
ranges of every kind, offsets past 32 bits, streams, graphs, waits that run out."""
import pytest
import torch

from layer_reference import HALF_BF16, ranges, swiglu
from test_gpu_experts_i8 import DEV, codes, factors, scales, sums
from test_gpu_layer_streams import behind_pending_work

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def product_of(x, sx, begin, end, w, sw):
    """bf16 result of whole sums that stay within 2^24."""
    ref, mag = sums(x, begin, end, w)
    assert float(mag.max()) <= 2 ** 24
    return (ref.float() * factors(sx, begin, end, sw, w.shape[1])).to(torch.bfloat16)


def near_swiglu(act, v):
    f = v.shape[1] // 2
    g, u = v[:, :f].double(), v[:, f:].double()
    ref = swiglu(g, u)
    # __expf is within 2 + |1.16 g| steps of fp32 and the quotient within 2
    lim = (HALF_BF16 + 2.0 ** -18 + 2.0 ** -22 * g.abs().clamp(max=128)) * ref.abs() + 1e-30
    return bool(((act.double() - ref).abs() <= lim).all())


# at most 16 rows, and some two for each expert on average: one expert with all of
# them, some with none, one or several units of four rows of w for each warp
FEW = [[1], [6], [0, 2], [8, 0], [0, 0, 1, 0], [1] * 16, [2, 0, 1, 5, 0, 0, 1, 1], [0, 0, 0, 0, 0, 0, 0, 16], [3, 4, 1, 0], [0] * 30 + [1, 3]]


@pytest.mark.parametrize("counts", FEW, ids=str)
@pytest.mark.parametrize("cin,n", [(16, 8), (112, 24), (496, 264), (512, 1024), (528, 2056), (1024, 5128), (1040, 8)])
def test_few_rows(moe, counts, cin, n):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, sx = codes(1, rows, cin, most=126), codes(2, e, 2 * n, cin, most=126), scales(3, rows)
    sw = scales(4, e, 2 * n)
    y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    half, shalf = w[:, :n].contiguous(), sw[:, :n].contiguous()
    moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, n), x, sx, begin, end, half, shalf, y)
    assert torch.equal(y, product_of(x, sx, begin, end, half, shalf))
    act = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    sx = sx * 2.0 ** -4
    moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, cin, n), x, sx, begin, end, w, sw, act)
    assert near_swiglu(act, sums(x, begin, end, w)[0].float() * factors(sx, begin, end, sw, 2 * n))


@pytest.mark.parametrize("counts", [[1], [2, 0, 1, 5, 0, 0, 1, 1], [1] * 16], ids=str)
@pytest.mark.parametrize("cin,n", [(80, 40), (7168, 256)])
def test_few_rows_are_those_of_the_tiles(moe, counts, cin, n):
    # the same rows in buffers of 100, which tiles work on: the same bits
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, 100, cin, most=40), codes(2, e, 2 * n, cin, most=40), scales(3, 100), scales(4, e, 2 * n)
    for name in ("moe_expert_product_i8", "moe_expert_swiglu_i8"):
        call = getattr(moe, name)
        width = n if "swiglu" in name else 2 * n
        few = call(moe.MoeExpertI8Desc(e, rows, cin, width), x[:rows], sx[:rows], begin, end, w, sw)
        many = call(moe.MoeExpertI8Desc(e, 100, cin, width), x, sx, begin, end, w, sw)
        assert torch.equal(few, many[:rows])


def test_few_rows_of_long_sums(moe):
    # 32-bit sums: exact to the last element, with the largest codes
    for cin in (7168, 65536):
        begin, end = ranges([1, 0, 3], DEV)
        x = torch.full((4, cin), -128, dtype=torch.int8, device=DEV)
        w = torch.full((3, 16, cin), -128, dtype=torch.int8, device=DEV)
        w[:, 1::2, -1] = 127
        x[1, ::2] = 127
        one = torch.ones(48, device=DEV)
        y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(3, 4, cin, 16), x, one, begin, end, w, one)
        assert torch.equal(y, sums(x, begin, end, w)[0].float().to(torch.bfloat16))


@pytest.mark.parametrize("rows", [11, 300])
def test_ranges_of_every_kind(moe, rows):
    # out of order, empty, backwards, from before the first row, past the last, far past it; and rows of none
    x, sx = codes(5, rows, 144), scales(6, rows)
    begin = torch.tensor([5, 3, 4, 9, -7, rows, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    end = torch.tensor([7, 3, 2, 2 ** 31 - 1, 2, rows + 5, 2 ** 31 - 1, -1], dtype=torch.int32, device=DEV)
    w, sw = codes(7, 8, 264, 144), scales(8, 8, 264)
    y = torch.full((rows, 264), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_i8(moe.MoeExpertI8Desc(8, rows, 144, 264), x, sx, begin, end, w, sw, y)
    b, t = begin.clamp(min=0, max=rows), end.clamp(min=0, max=rows)
    ref = product_of(x, sx, b, t, w, sw)
    inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for lo, hi in zip(b.tolist(), t.tolist()):
        inside[lo:hi] = True
    assert inside.tolist()[:11] == [True, True, False, False, False, True, True, False, False, True, True]
    assert torch.equal(y[inside], ref[inside]) and bool((y[~inside] == 9.0).all())


def test_few_rows_from_records(moe):
    rows, cin, n = 8, 528, 136
    rec = codes(5, rows, 80 + cin + 16)
    sx = scales(8, rows)
    rec.view(torch.float32)[:, (80 + cin) // 4] = sx
    x, view = rec[:, 80:80 + cin], rec.view(torch.float32)[:, (80 + cin) // 4]
    begin = torch.tensor([6, 0, 2, 5], dtype=torch.int32, device=DEV)
    end = torch.tensor([7, 2, 3, 5], dtype=torch.int32, device=DEV)
    w, sw = codes(6, 4, n, cin), scales(7, 4, n)
    y = torch.full((rows, n), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_i8(moe.MoeExpertI8Desc(4, rows, cin, n, x.stride(0), view.stride(0)), x, view, begin, end, w, sw, y)
    ref = product_of(x, sx, begin, end, w, sw)
    inside = torch.tensor([0, 1, 2, 6], device=DEV)
    outside = torch.tensor([3, 4, 5, 7], device=DEV)
    assert torch.equal(y[inside], ref[inside]) and bool((y[outside] == 9.0).all())


def test_few_rows_with_scales_that_are_not_numbers(moe):
    rows, cin, n = 5, 64, 136
    begin, end = ranges([2, 0, 3], DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 3, n, cin), scales(3, rows), scales(4, 3, n)
    sx[1], sw[2, 9] = float("nan"), float("inf")
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(3, rows, cin, n), x, sx, begin, end, w, sw)
    ref = product_of(x, sx, begin, end, w, sw)
    assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.nan_to_num(), ref.nan_to_num())
    assert bool(y[1].isnan().all()) and not bool(y[[0, 2, 3, 4]].isnan().any(1).all())


def test_a_row_that_is_not_finite_is_nan_to_the_end(moe):
    # quantised to the scale NaN, carried through the product
    for rows in (3, 40):
        x = torch.randn(rows, 128, device=DEV).bfloat16()
        x[1, 17] = float("inf")
        w, sw = codes(2, 2, 64, 128), scales(4, 2, 64)
        begin, end = ranges([2, rows - 2], DEV)
        q, s = moe.moe_quantize_rows(moe.MoeQuantDesc(rows, 128), x)
        y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(2, rows, 128, 64), q, s, begin, end, w, sw)
        assert bool(y[1].isnan().all()) and not bool(y[0].isnan().any()) and not bool(y[2:].isnan().any())


@pytest.mark.parametrize("most", [1, 3, 70])
def test_the_most_experts(moe, most):
    g = torch.Generator()
    g.manual_seed(most)
    counts = torch.randint(0, most + 1, (1024,), generator=g).tolist()
    rows, cin, n = sum(counts), 32, 24
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 1024, n, cin), scales(3, rows), scales(4, 1024, n)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(1024, rows, cin, n), x, sx, begin, end, w, sw)
    assert torch.equal(y, product_of(x, sx, begin, end, w, sw))


@pytest.mark.parametrize("busy", [[0], [31, 32], [33, 500, 1023], [1023], [255, 256, 257, 800]], ids=str)
def test_many_experts_without_rows(moe, busy):
    counts = [0] * 1024
    for i, e in enumerate(busy):
        counts[e] = (20, 220, 570)[i % 3]
    rows, cin, n = sum(counts), 144, 520
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 1024, n, cin), scales(3, rows), scales(4, 1024, n)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(1024, rows, cin, n), x, sx, begin, end, w, sw)
    assert torch.equal(y, product_of(x, sx, begin, end, w, sw))


@pytest.mark.parametrize("width", [32, 64, 96, 128, 160, 192])
def test_every_width_of_tiles(moe, width):
    # the widest tile sets how many stages there are; many steps go around all of them
    counts, cin, n = [width, 1, width - 31], 1000 * 16, 264
    rows = sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin, most=32), codes(2, 3, n, cin, most=32), scales(3, rows), scales(4, 3, n)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(3, rows, cin, n), x, sx, begin, end, w, sw)
    assert torch.equal(y, product_of(x, sx, begin, end, w, sw))


def test_weights_past_32_bits(moe):
    e, n, cin = 41, 8192, 16384  # 5.5 GB
    w = torch.zeros(e, n, cin, dtype=torch.int8, device=DEV)
    w[-1], w[0] = codes(2, n, cin, most=30), codes(3, n, cin, most=30)
    sw = scales(4, e, n)
    for rows in (5, 77):
        begin = torch.zeros(e, dtype=torch.int32, device=DEV)
        end = torch.zeros(e, dtype=torch.int32, device=DEV)
        end[0], begin[-1], end[-1] = 2, 2, rows
        x, sx = codes(1, rows, cin, most=30), scales(5, rows)
        y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, n), x, sx, begin, end, w, sw)
        assert torch.equal(y[:2], product_of(x[:2], sx[:2], begin[:1], end[:1], w[:1], sw[:1]))
        assert torch.equal(y[2:], product_of(x[2:], sx[2:], begin[:1], end[-1:] - 2, w[-1:], sw[-1:]))


def test_rows_past_32_bits(moe):
    # rows 65536 bytes apart, results of 65536 features: 2.6 and 5.2 GB, and rows behind 2^31 bytes of each
    rows, cin, n = 40000, 64, 65536
    buffer = torch.zeros(rows, 65536, dtype=torch.int8, device=DEV)
    x = buffer[:, 48 * 16:48 * 16 + cin]
    at = [0, 16383, 16384, 32767, 32768, 39999]
    x[at] = codes(1, 6, cin)
    sx = scales(2, rows)
    begin = torch.tensor([0, 16383, 32767, 39999], dtype=torch.int32, device=DEV)
    end = torch.tensor([1, 16385, 32769, 40000], dtype=torch.int32, device=DEV)
    w, sw = codes(3, 4, n, cin), scales(4, 4, n)
    y = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_i8(moe.MoeExpertI8Desc(4, rows, cin, n, x_stride=65536), x, sx, begin, end, w, sw, y)
    b, t = ranges([1, 2, 2, 1], DEV)
    assert torch.equal(y[at], product_of(x[at].contiguous(), sx[at], b, t, w, sw))
    assert int((y != 0).any(1).sum()) == 6


def test_graph_follows_ranges_scales_and_rows(moe):
    counts, cin, n = [40, 0, 77, 11], 256, 136
    rows, e = sum(counts), 4
    begin, end = ranges(counts, DEV)
    x16, w, sw = torch.empty(rows, cin, dtype=torch.bfloat16, device=DEV), codes(2, e, n, cin), scales(4, e, n)
    used = torch.tensor([rows], dtype=torch.int32, device=DEV)
    few_begin, few_end = ranges([1, 0, 2, 1], DEV)

    def step():
        q, s = moe.moe_quantize_rows(moe.MoeQuantDesc(rows, cin), x16, num_rows=used)
        return (q, s, moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, n), q, s, begin, end, w, sw),
                moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, 4, cin, n), q, s, few_begin, few_end, w, sw))

    x16.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed, counts in enumerate(([40, 0, 77, 11], [0, 128, 0, 0], [3, 5, 70, 2], [0, 0, 0, 0])):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        x16.copy_(torch.randn(rows, cin, generator=g, device=DEV))
        b, t = ranges(counts, DEV)
        begin.copy_(b)
        end.copy_(t)
        total = sum(counts)
        used.fill_(max(total, 4))
        graph.replay()
        q, s, y, few = (t.clone() for t in got)
        want = step()
        assert torch.equal(q[:total], want[0][:total]) and torch.equal(s[:total], want[1][:total])
        assert torch.equal(y[:total], want[2][:total]) and torch.equal(few, want[3])
        if total:
            assert torch.equal(y[:total], product_of(q[:total], s[:total, 0], b, t, w, sw))


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream(moe, raw):
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    counts, cin, f = [40, 0, 77], 256, 128
    rows = sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 3, 2 * f, cin), scales(3, rows), scales(4, 3, 2 * f)
    x16 = torch.randn(rows, cin, device=DEV).bfloat16()
    few_begin, few_end = ranges([1, 0, 2], DEV)
    calls = [lambda **k: moe.moe_quantize_rows(moe.MoeQuantDesc(rows, cin), x16, **k),
             lambda **k: moe.moe_quantize_rows(moe.MoeQuantDesc(rows, cin, scale_stride=4), x16, **k),
             lambda **k: moe.moe_expert_product_i8(moe.MoeExpertI8Desc(3, rows, cin, 2 * f), x, sx, begin, end, w, sw, **k),
             lambda **k: moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(3, rows, cin, f), x, sx, begin, end, w, sw, **k),
             lambda **k: moe.moe_expert_product_i8(moe.MoeExpertI8Desc(3, 3, cin, 2 * f), x, sx, few_begin, few_end, w, sw, **k)]
    for call in calls:
        want = call()
        want = want if isinstance(want, tuple) else (want,)
        got = behind_pending_work(lambda: call(stream=stream), want)
        got = got if isinstance(got, tuple) else (got,)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_queued_without_a_pause(moe):
    # pairs of blocks start while blocks of the kernel before still hold part of each SM
    rows, cin, f = 4096, 256, 2048
    begin, end = ranges([1000, 0, 3001, 95], DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(rows, cin, generator=g, device=DEV).bfloat16()
    w, sw = codes(2, 4, 2 * f, cin), scales(4, 4, 2 * f) * 2.0 ** -3
    q, s = torch.empty(rows, cin, dtype=torch.int8, device=DEV), torch.empty(rows, 1, device=DEV)
    act = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)
    qa, sa = torch.empty(rows, f, dtype=torch.int8, device=DEV), torch.empty(rows, 1, device=DEV)
    calls = [moe.prepare_quantize_rows(moe.MoeQuantDesc(rows, cin), x, q, s),
             moe.prepare_expert_swiglu_i8(moe.MoeExpertI8Desc(4, rows, cin, f), q, s, begin, end, w, sw, act),
             moe.prepare_quantize_rows(moe.MoeQuantDesc(rows, f), act, qa, sa)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    first = [t.clone() for t in (q, s, act, qa, sa)]
    for _ in range(100):
        for call in calls:
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (q, s, act, qa, sa)))


def test_beside_the_bf16_products_on_another_stream(moe):
    # both hold all of an SM's tensor memory while they run
    rows, cin, n = 1500, 512, 1024
    begin, end = ranges([700, 1, 799], DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 3, n, cin), scales(3, rows), scales(4, 3, n)
    xb, wb = x.bfloat16(), w.bfloat16()
    d8, d16 = moe.MoeExpertI8Desc(3, rows, cin, n), moe.MoeExpertDesc(3, rows, cin, n)
    want8, want16 = moe.moe_expert_product_i8(d8, x, sx, begin, end, w, sw), moe.moe_expert_product(d16, xb, begin, end, wb)
    streams = [torch.cuda.Stream() for _ in range(2)]
    y8, y16 = torch.zeros_like(want8), torch.zeros_like(want16)
    torch.cuda.synchronize()
    for _ in range(50):
        moe.moe_expert_product_i8(d8, x, sx, begin, end, w, sw, y8, stream=streams[0])
        moe.moe_expert_product(d16, xb, begin, end, wb, y16, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(y8, want8) and torch.equal(y16, want16)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("counts", [[300, 129, 777], [8, 8, 20]], ids=str)
def test_waits_that_run_out_leave_the_context_usable(moe, counts, glu):
    cin, f = 4096, 256
    begin, end = ranges(counts, DEV)
    rows = sum(counts)
    x, w, sx, sw = codes(1, rows, cin, most=30), codes(2, 3, 2 * f, cin, most=30), scales(3, rows), scales(4, 3, 2 * f)
    name, n = ("moe_expert_swiglu_i8", f) if glu else ("moe_expert_product_i8", 2 * f)
    run = lambda: getattr(moe, name)(moe.MoeExpertI8Desc(3, rows, cin, n), x, sx, begin, end, w, sw)  # noqa: E731
    want = run().clone()
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    moe.moe_set_wait_limit_ns(1)
    try:
        run()
        assert moe.moe_device_status() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_wait_limit_ns(0)
    again = run()
    assert moe.moe_device_status() == moe.MOE_OK and torch.equal(again, want)
