"""Sums past 2^24: exact from the kernel of a few rows, fp32 sums from tiles, for
the same rows in buffers of different size. The limits are those of
test_gpu_experts_i8: each step of 16 products rounds or truncates the running sum
once."""
import pytest
import torch

from layer_reference import HALF_BF16, ranges
from test_gpu_experts_i8 import DEV, codes, factors, scales, sums

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cin", [7168, 65536])
@pytest.mark.parametrize("counts", [[1, 3], [0, 16, 0, 0, 0, 0], [2, 0, 6]], ids=str)
def test_rows_of_small_and_large_buffers(cin, counts):
    from combine_moe_layout_03_gb300 import moe
    e, rows, n = len(counts), sum(counts), 136
    assert rows <= 16 and rows <= 2 * e + 4
    begin, end = ranges(counts, DEV)
    x, w, sx, sw = codes(1, 100, cin).abs(), codes(2, e, n, cin).abs(), scales(3, 100), scales(4, e, n)
    few = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, rows, cin, n), x[:rows], sx[:rows], begin, end, w, sw)
    many = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(e, 100, cin, n), x, sx, begin, end, w, sw)[:rows]
    ref, mag = sums(x[:rows], begin, end, w)
    assert float(ref.min()) > 2 ** 24
    f = factors(sx[:rows], begin, end, sw, n)
    assert torch.equal(few, (ref.float() * f).to(torch.bfloat16))
    lim = (cin / 16 + 4) * 2.0 ** -23 * mag * f.double() * 1.01
    ref = ref * f.double()
    assert bool(((many.double() - ref).abs() <= lim + (HALF_BF16 + 3 * 2.0 ** -24) * ref).all())
    assert bool(((many.double() - few.double()).abs() <= lim + 2 * (HALF_BF16 + 3 * 2.0 ** -24) * ref).all())
