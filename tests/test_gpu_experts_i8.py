"""The experts' 8-bit products against 64-bit sums of whole numbers.

While a sum and its parts stay within 2^24 it is exact, so that the result is
bf16 of one fp32 product, bit for bit. Beyond, each step of 16 products adds one
rounding or truncation of the running sum (2^-23 of what it holds, at most the
sum of magnitudes)."""
import pytest
import torch

from layer_reference import HALF_BF16, ranges, swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def codes(seed, *shape, most=127):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV, dtype=torch.int8)


def scales(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.exp(torch.randn(shape, generator=g, device=DEV)) * 2.0 ** -10


def sums(x, begin, end, w):
    """float64 sums [rows, N] (exact: below 2^53) and of magnitudes, zero outside the ranges."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e, (b, t) in enumerate(zip(begin.tolist(), end.tolist())):
        if t > b:
            a, m = x[b:t].double(), w[e].double()
            y[b:t], mag[b:t] = a @ m.t(), a.abs() @ m.abs().t()
    return y, mag


def factors(sx, begin, end, sw, n):
    """[rows, n] of the scales' type: sx[s] * sw[e, n]."""
    out = torch.zeros(sx.shape[0], n, dtype=sx.dtype, device=sx.device)
    for e, (b, t) in enumerate(zip(begin.tolist(), end.tolist())):
        out[b:t] = sx[b:t, None] * sw[e][None, :]
    return out


COUNTS = [[1], [32], [191], [192], [193], [0, 3, 0], [5, 0, 127, 128, 1, 300, 0], [0, 0], [1] * 40, [64, 65, 63, 1], [97, 385]]
SIZES = [(64, 256), (16, 8), (80, 264), (208, 136), (1024, 520), (336, 1000)]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("cin,cout", SIZES)
def test_product(moe, counts, cin, cout):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w = codes(1, max(rows, 1), cin), codes(2, e, cout, cin)
    sx, sw = scales(3, max(rows, 1)), scales(4, e, cout)
    y = torch.full((max(rows, 1), cout), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, cout), x, sx, begin, end, w, sw, y)
    if not rows:
        assert bool((y == 7.0).all())
        return
    ref, mag = sums(x, begin, end, w)
    assert float(mag.max()) <= 2 ** 24  # 1024 * 127^2
    assert torch.equal(y, (ref.float() * factors(sx, begin, end, sw, cout)).to(torch.bfloat16))


@pytest.mark.parametrize("cin", [16, 112, 128, 144, 1024])
def test_all_codes(moe, cin):
    # -128 too, in both operands, at every place of a step
    rows, cout = 256, 256
    begin, end = ranges([rows], DEV)
    every = torch.arange(-128, 128, device=DEV).to(torch.int8)
    x = every[:, None].repeat(1, cin)
    x[:, 1::2] = 0
    w = torch.stack([every.roll(k)[:256] for k in range(cin)], 1)[None].contiguous()
    one = torch.ones(256, device=DEV)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(1, rows, cin, cout), x, one, begin, end, w, one)
    assert torch.equal(y, sums(x, begin, end, w)[0].float().to(torch.bfloat16))


@pytest.mark.parametrize("rows,e,cin,cout", [(700, 5, 2048, 1024), (40, 8, 7168, 512), (1, 1, 65536, 2048), (9, 3, 16384, 65536)])
def test_long_sums(moe, rows, e, cin, cout):
    # sums of one sign, far past 2^24
    counts = [rows // e] * (e - 1)
    counts.append(rows - sum(counts))
    begin, end = ranges(counts, DEV)
    x, w = codes(1, rows, cin), codes(2, e, cout, cin).abs()
    x[::2] = x[::2].abs()
    sx, sw = scales(3, rows), scales(4, e, cout)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, cout), x, sx, begin, end, w, sw)
    ref, mag = sums(x, begin, end, w)
    f = sx.double()[:, None] * torch.cat([sw[i].double().expand(c, cout) for i, c in enumerate(counts)])
    lim = (cin / 16 + 4) * 2.0 ** -23 * mag * f * 1.01
    ref = ref * f
    assert bool(((y.double() - ref).abs() <= lim + (HALF_BF16 + 3 * 2.0 ** -24) * ref.abs()).all())


@pytest.mark.parametrize("counts", [[1], [130, 0, 5], [0, 300, 1, 128], [33] * 9], ids=str)
@pytest.mark.parametrize("cin,f", [(64, 128), (256, 8), (144, 200), (512, 384), (80, 136)])
def test_swiglu(moe, counts, cin, f):
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w = codes(1, rows, cin), codes(2, e, 2 * f, cin)
    sx, sw = scales(3, rows) * 2.0 ** -2, scales(4, e, 2 * f) * 2.0 ** -2
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, cin, f), x, sx, begin, end, w, sw)
    v = (sums(x, begin, end, w)[0].float() * factors(sx, begin, end, sw, 2 * f)).double()  # fp32 as the kernel has it
    g, u = v[:, :f], v[:, f:]
    ref = swiglu(g, u)
    # __expf is within 2 + |1.16 g| steps of fp32 and the quotient within 2; beyond |g| = 88 the smaller of the two is zero
    lim = (HALF_BF16 + 2.0 ** -18 + 2.0 ** -22 * g.abs().clamp(max=128)) * ref.abs() + 1e-30
    assert bool(((act.double() - ref).abs() <= lim).all())


def test_swiglu_is_the_product_activated(moe):
    # gate and up from the plain product with scales that leave them exact
    rows, cin, f = 500, 256, 264
    begin, end = ranges([rows], DEV)
    x, w = codes(1, rows, cin, most=3), codes(2, 1, 2 * f, cin, most=2)
    sx, sw = torch.full((rows,), 2.0 ** -3, device=DEV), torch.full((1, 2 * f), 2.0 ** -4, device=DEV)
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(1, rows, cin, f), x, sx, begin, end, w, sw)
    v = sums(x, begin, end, w)[0] * 2.0 ** -7
    ref = swiglu(v[:, :f], v[:, f:])
    assert bool(((act.double() - ref).abs() <= (HALF_BF16 + 2.0 ** -17) * ref.abs() + 1e-30).all())


def test_rows_from_records_and_untouched_rows(moe):
    # rows and scales read out of padded records, ranges out of order, a gap, and limits past the buffer
    rows, cin, cout = 300, 144, 264
    rec = codes(5, rows, 80 + cin + 16)
    sx = scales(8, rows)
    rec.view(torch.float32)[:, (80 + cin) // 4] = sx
    x, view = rec[:, 80:80 + cin], rec.view(torch.float32)[:, (80 + cin) // 4]
    begin = torch.tensor([200, 10, 50, 290, -5], dtype=torch.int32, device=DEV)
    end = torch.tensor([250, 30, 50, 1000, 4], dtype=torch.int32, device=DEV)
    w, sw = codes(6, 5, cout, cin), scales(7, 5, cout)
    d = moe.MoeExpertI8Desc(5, rows, cin, cout, x.stride(0), view.stride(0))
    y = torch.full((rows, cout), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_product_i8(d, x, view, begin, end, w, sw, y)
    b, t = begin.clamp(min=0), end.clamp(max=rows)
    ref = (sums(x, b, t, w)[0].float() * factors(sx, b, t, sw, cout)).to(torch.bfloat16)
    inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for lo, hi in zip(b.tolist(), t.tolist()):
        inside[lo:hi] = True
    assert torch.equal(y[inside], ref[inside]) and bool((y[~inside] == 9.0).all())
    act = torch.full((rows, cout // 2 // 8 * 8), 9.0, dtype=torch.bfloat16, device=DEV)
    f = act.shape[1]
    moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(5, rows, cin, f, x.stride(0), view.stride(0)), x, view, begin, end,
                             w[:, :2 * f].contiguous(), sw[:, :2 * f].contiguous(), act)
    assert bool((act[~inside] == 9.0).all()) and not bool((act[inside] == 9.0).all(1).any())


def test_scales_that_are_not_numbers_stay_in_their_row_and_channel(moe):
    rows, cin, cout = 70, 64, 136
    begin, end = ranges([33, 37], DEV)
    x, w = codes(1, rows, cin), codes(2, 2, cout, cin)
    sx, sw = scales(3, rows), scales(4, 2, cout)
    sx[40], sw[0, 9] = float("nan"), float("inf")
    d = moe.MoeExpertI8Desc(2, rows, cin, cout)
    y = moe.moe_expert_product_i8(d, x, sx, begin, end, w, sw)
    ref = (sums(x, begin, end, w)[0].float() * factors(sx, begin, end, sw, cout)).to(torch.bfloat16)
    assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.nan_to_num(), ref.nan_to_num())
    assert int(y.isnan().any(1).sum()) <= 34 and bool(y[40].isnan().all())


@pytest.mark.parametrize("scale_width", [1, 4])
def test_quantise_products_and_back(moe, scale_width):
    # as a served block uses them, on rows in expert order
    counts, h, f = [3, 0, 70, 200], 256, 144
    rows, e = sum(counts), len(counts)
    begin, end = ranges(counts, DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    draw = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=DEV) * scale).bfloat16()  # noqa: E731
    x, w1, w2 = draw(rows, h), draw(e, 2 * f, h, scale=h ** -0.5), draw(e, h, f, scale=f ** -0.5)
    q1, s1 = moe.moe_quantize_rows(moe.MoeQuantDesc(e * 2 * f, h), w1)
    q2, s2 = moe.moe_quantize_rows(moe.MoeQuantDesc(e * h, f), w2)
    q, s = moe.moe_quantize_rows(moe.MoeQuantDesc(rows, h, scale_stride=scale_width), x)
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, h, f, x_scale_stride=scale_width), q, s, begin, end, q1, s1)
    qa, sa = moe.moe_quantize_rows(moe.MoeQuantDesc(rows, f), act)
    y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, f, h), qa, sa, begin, end, q2, s2)
    def scaled(q, s, w, sw):  # sums of whole numbers, which are exact in 64 bits (a sum of scaled ones is not: where it is zero, say)
        return sums(q, begin, end, w)[0] * factors(s.double(), begin, end, sw.double(), w.shape[1])

    v = scaled(q, s[:, 0], q1.view(e, 2 * f, h), s1.view(e, 2 * f))
    act_ref = swiglu(v[:, :f], v[:, f:])
    assert bool(((act.double() - act_ref).abs() <= (HALF_BF16 + 2.0 ** -17) * act_ref.abs() + 1e-6 * float(act_ref.abs().max())).all())
    ref = scaled(qa, sa[:, 0], q2.view(e, h, f), s2.view(e, h))
    assert bool(((y.double() - ref).abs() <= (HALF_BF16 + 2.0 ** -20) * ref.abs()).all())
    # and against the block in bf16's own values: a code is half a step (1 / 254 of its row's largest, some 3.5 deviations)
    # off at most, uniformly: 3.5 / 254 / sqrt(3) = 0.8% of each operand in the 2-norm, four of them and the activation
    v = sums(x, begin, end, w1)[0]
    whole = sums(swiglu(v[:, :f], v[:, f:]), begin, end, w2.double())[0]
    assert float((y.double() - whole).norm() / whole.norm()) < 0.04


def test_same_bits_every_time(moe):
    rows, e, cin, cout = 1000, 7, 512, 520
    begin, end = ranges([rows // e] * e, DEV)
    x, w = codes(1, rows, cin).abs(), codes(2, e, cout, cin).abs()
    sx, sw = scales(3, rows), scales(4, e, cout)
    d = moe.MoeExpertI8Desc(e, rows, cin, cout)
    first = moe.moe_expert_product_i8(d, x, sx, begin, end, w, sw, torch.zeros(rows, cout, dtype=torch.bfloat16, device=DEV))
    for _ in range(20):
        again = moe.moe_expert_product_i8(d, x, sx, begin, end, w, sw, torch.zeros_like(first))
        assert torch.equal(first, again)
