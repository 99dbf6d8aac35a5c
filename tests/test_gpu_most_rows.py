"""The experts' products with as many rows as they take, 2^31 - 129, nearly all of
one expert (80 GB): each of them is in a tile and where it belongs. And as many rows
to 8 bits (110 GB)."""
import pytest
import torch

from test_gpu_experts import normal, whole
from test_gpu_experts_i8 import DEV, codes, scales
from test_gpu_i8_edges import near_swiglu, product_of

pytestmark = pytest.mark.gpu
ROWS = 2 ** 31 - 129
FIRST = 5  # rows of the first expert


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def places():
    """Rows that are not zero: the ends, tiles' ends near them, and some of all."""
    g = torch.Generator().manual_seed(1)
    at = {0, 4, 5, 6, FIRST + 191, FIRST + 192, FIRST + 255, FIRST + 256, 2 ** 30, 2136356790, ROWS - 300, ROWS - 2, ROWS - 1}
    at |= set(torch.randint(0, ROWS, (400,), generator=g).tolist())
    return torch.tensor(sorted(at), device=DEV)


def ends(at):
    """Ranges of all rows, and of those at `at` alone."""
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    few = int((at < FIRST).sum())
    return t(0, FIRST), t(FIRST, ROWS), t(0, few), t(few, len(at))


def rows_that_are_not_zero(y):
    """Of rows of 16 bytes."""
    piece, v = 1 << 26, y.view(torch.int64)
    return sum(int((v[i:i + piece, 0] | v[i:i + piece, 1]).count_nonzero()) for i in range(0, len(v), piece))


@pytest.mark.parametrize("glu", [False, True])
def test_8_bit_products(moe, glu):
    at = places()
    begin, end, b, t = ends(at)
    x, sx = torch.zeros(ROWS, 16, dtype=torch.int8, device=DEV), torch.ones(ROWS, device=DEV)
    x[at], sx[at] = codes(1, len(at), 16), scales(2, len(at))
    halves = 2 if glu else 1
    w, sw = codes(3, 2, halves * 8, 16), scales(4, 2, halves * 8)
    y = torch.full((ROWS, 8), 9.0, dtype=torch.bfloat16, device=DEV)
    call = moe.moe_expert_swiglu_i8 if glu else moe.moe_expert_product_i8
    call(moe.MoeExpertI8Desc(2, ROWS, 16, 8), x, sx, begin, end, w, sw, y)
    if glu:
        v = torch.cat([(x[at[i:j]].float() @ w[e].float().t()) * (sx[at[i:j], None] * sw[e])
                       for e, (i, j) in enumerate(zip(b.tolist(), t.tolist()))])  # sums of 16 are exact in 32 bits
        assert near_swiglu(y[at], v)
    else:
        assert torch.equal(y[at], product_of(x[at], sx[at], b, t, w, sw))
    assert rows_that_are_not_zero(y) == rows_that_are_not_zero(y[at])


@pytest.mark.parametrize("name", ["moe_expert_product", "moe_expert_swiglu", "moe_expert_product_backward_input"])
def test_bf16_products(moe, name):
    at = places()
    begin, end, b, t = ends(at)
    x = torch.zeros(ROWS, 8, dtype=torch.bfloat16, device=DEV)
    x[at] = whole(1, len(at), 8)
    w = whole(3, 2, 16 if "swiglu" in name else 8, 8)
    y = torch.full((ROWS, 8), 9.0, dtype=torch.bfloat16, device=DEV)
    getattr(moe, name)(moe.MoeExpertDesc(2, ROWS, 8, 8), x, begin, end, w, y)
    v = torch.cat([x[at[i:j]].double() @ (w[e] if "input" in name else w[e].t()).double()  # sums of whole numbers
                   for e, (i, j) in enumerate(zip(b.tolist(), t.tolist()))])
    assert near_swiglu(y[at], v) if "swiglu" in name else torch.equal(y[at], v.to(torch.bfloat16))
    assert rows_that_are_not_zero(y) == rows_that_are_not_zero(y[at])


def test_rows_to_8_bits(moe):
    n = 2 ** 31 - 1
    at = torch.cat([places(), torch.arange(n - 130, n, device=DEV)]).unique()
    x = torch.zeros(n, 16, dtype=torch.bfloat16, device=DEV)
    x[at] = normal(1, len(at), 16)
    q = torch.full((n, 16), 9, dtype=torch.int8, device=DEV)
    s = torch.full((n, 1), 9.0, device=DEV)
    moe.moe_quantize_rows(moe.MoeQuantDesc(n, 16), x, q, s)
    few = moe.moe_quantize_rows(moe.MoeQuantDesc(len(at), 16), x[at])
    assert torch.equal(q[at], few[0]) and torch.equal(s[at], few[1])
    assert rows_that_are_not_zero(q) == len(at)
    # a row of zeros has the scale of the floor: that of the first row that is zero stands for all
    zero = moe.moe_quantize_rows(moe.MoeQuantDesc(1, 16), torch.zeros(1, 16, dtype=torch.bfloat16, device=DEV))[1]
    piece = 1 << 26
    assert sum(int((s[i:i + piece] == zero).count_nonzero()) for i in range(0, n, piece)) == n - len(at)
