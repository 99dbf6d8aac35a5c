"""The gated 8-bit product at the edges: gates of every size, its weights and
rows past 32 bits (a tensor map and offsets of its own), ranges of every kind,
scales that are not numbers in gate or in up, every width of tiles; by tiles and,
for a few rows, by the kernel that streams the weights."""
import pytest
import torch

from layer_reference import ranges
from test_gpu_experts_i8 import DEV, codes, factors, scales, sums
from test_gpu_i8_edges import near_swiglu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def gate_up(x, sx, begin, end, w, sw):
    """fp32 [rows, 2F] as the kernels have it, of sums that stay within 2^24."""
    ref, mag = sums(x, begin, end, w)
    assert float(mag.max()) <= 2 ** 24
    return ref.float() * factors(sx, begin, end, sw, w.shape[1])


@pytest.mark.parametrize("counts", [[3, 0, 4, 1, 4], [96, 0, 33, 200]], ids=["few", "tiles"])
@pytest.mark.parametrize("cin,f", [(64, 264), (144, 128)])
def test_gates_of_every_size(moe, counts, cin, f):
    # rows from gates of some 0.01 to some 100 (sums of 64 products of codes deviate by 43000)
    e, rows = len(counts), sum(counts)
    begin, end = ranges(counts, DEV)
    x, w = codes(1, rows, cin), codes(2, e, 2 * f, cin)
    sx = torch.exp2(torch.linspace(-14, -1, rows, device=DEV))
    sw = torch.exp(0.2 * torch.randn(e, 2 * f, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)) * 2.0 ** -8
    v = gate_up(x, sx, begin, end, w, sw)
    g = v[:, :f]
    assert all(bool((s * g > most).any()) for s in (1, -1) for most in (10, 88, 150)) and bool((g.abs() < 0.01).any())
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, cin, f), x, sx, begin, end, w, sw)
    # (below -88 the sigmoid is under 2^-126 and act under 1e-30, which near_swiglu leaves for that)
    assert float((v[:, :f].abs().max() * v[:, f:].abs().max())) < 1e7
    assert near_swiglu(act, v)


@pytest.mark.parametrize("rows", [11, 300])
def test_ranges_of_every_kind(moe, rows):
    # out of order, empty, backwards, from before the first row, past the last, far past it; and rows of none
    f = 136
    x, sx = codes(5, rows, 144), scales(6, rows) * 2.0 ** -2
    begin = torch.tensor([5, 3, 4, 9, -7, rows, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    end = torch.tensor([7, 3, 2, 2 ** 31 - 1, 2, rows + 5, 2 ** 31 - 1, -1], dtype=torch.int32, device=DEV)
    w, sw = codes(7, 8, 2 * f, 144), scales(8, 8, 2 * f)
    act = torch.full((rows, f), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(8, rows, 144, f), x, sx, begin, end, w, sw, act)
    b, t = begin.clamp(min=0, max=rows), end.clamp(min=0, max=rows)
    v = gate_up(x, sx, b, t, w, sw)
    inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for lo, hi in zip(b.tolist(), t.tolist()):
        inside[lo:hi] = True
    assert inside.tolist()[:11] == [True, True, False, False, False, True, True, False, False, True, True]
    assert near_swiglu(act[inside], v[inside]) and bool((act[~inside] == 9.0).all())


@pytest.mark.parametrize("counts", [[2, 0, 3], [33, 0, 137]], ids=["few", "tiles"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scales_that_are_not_numbers(moe, counts, bad):
    # of a gate in the first expert and an up in the last, and of a row: they and no others are lost
    rows, cin, f = sum(counts), 64, 136
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin), codes(2, 3, 2 * f, cin), scales(3, rows), scales(4, 3, 2 * f)
    clean = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(3, rows, cin, f), x, sx, begin, end, w, sw)
    assert near_swiglu(clean, gate_up(x, sx, begin, end, w, sw))
    sw[0, 9], sw[2, f + 20], sx[rows - 1] = bad, bad, bad
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(3, rows, cin, f), x, sx, begin, end, w, sw)
    lost = torch.zeros(rows, f, dtype=torch.bool, device=DEV)
    lost[:counts[0], 9] = lost[counts[0]:, 20] = lost[rows - 1] = True
    assert torch.equal(act[~lost], clean[~lost])
    if bad != bad:
        assert bool(act[lost].isnan().all())
    else:  # (an infinite gate times zero, or a zero sum times infinity, is NaN; where it goes to minus infinity too)
        assert not bool(act[lost].isfinite().any())


@pytest.mark.parametrize("width", [32, 64, 96, 128, 160, 192])
def test_every_width_of_tiles(moe, width):
    # the widest tile sets how many stages there are; many steps go around all of them
    counts, cin, f = [width, 1, width - 31], 1000 * 16, 136
    rows = sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, rows, cin, most=32), codes(2, 3, 2 * f, cin, most=32), scales(3, rows) * 2.0 ** 4, scales(4, 3, 2 * f)
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(3, rows, cin, f), x, sx, begin, end, w, sw)
    assert near_swiglu(act, gate_up(x, sx, begin, end, w, sw))


@pytest.mark.parametrize("rows", [5, 77])
def test_weights_past_32_bits(moe, rows):
    e, f, cin = 41, 4096, 16384  # 5.5 GB
    w = torch.zeros(e, 2 * f, cin, dtype=torch.int8, device=DEV)
    w[-1], w[0] = codes(2, 2 * f, cin, most=30), codes(3, 2 * f, cin, most=30)
    sw = scales(4, e, 2 * f)
    begin = torch.zeros(e, dtype=torch.int32, device=DEV)
    end = torch.zeros(e, dtype=torch.int32, device=DEV)
    end[0], begin[-1], end[-1] = 2, 2, rows
    x, sx = codes(1, rows, cin, most=30), scales(5, rows) * 2.0 ** 4
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, cin, f), x, sx, begin, end, w, sw)
    assert near_swiglu(act[:2], gate_up(x[:2], sx[:2], begin[:1], end[:1], w[:1], sw[:1]))
    assert near_swiglu(act[2:], gate_up(x[2:], sx[2:], begin[:1], end[-1:] - 2, w[-1:], sw[-1:]))


def test_rows_past_32_bits(moe):
    # rows 65536 bytes apart, results of 65536 channels: 2.6 and 5.2 GB, and rows behind 2^31 bytes of each
    rows, cin, f = 40000, 64, 65536
    buffer = torch.zeros(rows, 65536, dtype=torch.int8, device=DEV)
    x = buffer[:, 48 * 16:48 * 16 + cin]
    at = [0, 16383, 16384, 32767, 32768, 39999]
    x[at] = codes(1, 6, cin)
    sx = scales(2, rows)
    begin = torch.tensor([0, 16383, 32767, 39999], dtype=torch.int32, device=DEV)
    end = torch.tensor([1, 16385, 32769, 40000], dtype=torch.int32, device=DEV)
    w, sw = codes(3, 4, 2 * f, cin), scales(4, 4, 2 * f)
    act = torch.zeros(rows, f, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(4, rows, cin, f, x_stride=65536), x, sx, begin, end, w, sw, act)
    b, t = ranges([1, 2, 2, 1], DEV)
    assert near_swiglu(act[at], gate_up(x[at].contiguous(), sx[at], b, t, w, sw))
    assert int((act != 0).any(1).sum()) == 6


def test_few_rows_past_32_bits(moe):
    # four rows 2^31 bytes apart
    cin, f, stride = 528, 136, 1 << 31
    buffer = torch.zeros(3 * stride + 1024, dtype=torch.int8, device=DEV)
    x = buffer.as_strided((4, cin), (stride, 1))
    x.copy_(codes(1, 4, cin))
    sx, w, sw = scales(2, 4), codes(3, 2, 2 * f, cin), scales(4, 2, 2 * f)
    begin, end = ranges([1, 3], DEV)
    act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(2, 4, cin, f, x_stride=stride), x, sx, begin, end, w, sw)
    assert near_swiglu(act, gate_up(x.contiguous(), sx, begin, end, w, sw))
