"""Rows to 8-bit integers: codes and scales bit for bit those of the rule, whose
quotients and products are IEEE fp32 (numpy's)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    return m


def rule(x):
    """(codes int8, scales fp32) of x [rows, width] by the header's formula."""
    x = x.detach().float().cpu().numpy()
    with np.errstate(all="ignore"):
        most = np.abs(x).max(1).astype(np.float32)
        fine = np.isfinite(x).all(1)
        a = np.maximum(np.where(fine, most, np.float32(1)), np.float32(1e-30)).astype(np.float32)
        m = (x * (np.float32(127) / a)[:, None]).astype(np.float32)
        q = np.where(fine[:, None], np.rint(m.astype(np.float64)), 0.0).astype(np.int8)
        s = np.where(fine, a / np.float32(127), np.float32(NAN)).astype(np.float32)
    return q, s


def draw(seed, rows, width, f32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device=DEV) * torch.exp(4 * torch.randn(rows, 1, generator=g, device=DEV))
    return x if f32 else x.bfloat16()


def check(moe, x, **kw):
    rows, width = x.shape
    f32 = x.dtype == torch.float32
    d = moe.MoeQuantDesc(rows, width, moe.MOE_ROWS_F32 if f32 else moe.MOE_ROWS_BF16, x.stride(0) if rows > 1 else 0, **kw)
    q = torch.full((rows, width), 77, dtype=torch.int8, device=DEV)
    s = torch.full((rows, d.scale_stride), 7.0, device=DEV)
    moe.moe_quantize_rows(d, x, q, s)
    rq, rs = rule(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s[:, 0].cpu().numpy(), rs, equal_nan=True)
    assert not s[:, 1:].any()


# widths around every choice of threads a row, and the largest
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("width", [16, 32, 48, 256, 272, 1008, 1024, 1040, 2048, 2064, 4080, 4096, 4112, 7168, 8192, 8208, 16384, 16400, 32784, 65536])
def test_widths(moe, width, f32):
    for rows in (1, 3, 9) if width > 4096 else (1, 2, 7, 8, 9, 33, 257):
        check(moe, draw(rows, rows, width, f32), scale_stride=4 if rows % 2 else 1)


@pytest.mark.parametrize("f32", [False, True])
def test_many_rows(moe, f32):
    check(moe, draw(5, 20011, 528, f32))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("width,pad", [(64, 8), (2048, 40), (7168, 1024)])
def test_strided_rows(moe, width, pad, f32):
    check(moe, draw(3, 41, width + pad, f32)[:, pad:])


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("width", [16, 496, 2048, 7168, 65536])
def test_rows_of_every_kind(moe, width, f32):
    x = draw(9, 16, width, f32)
    big = torch.finfo(x.dtype).max
    x[0] = 0
    x[1] = -0.0
    x[2, 0], x[2, 1:] = INF, 1.0
    x[3, width - 1] = -INF
    x[4, width // 2] = NAN
    x[5] = NAN
    x[6] = big
    x[7] = -big
    x[8], x[8, 3] = 0, -torch.finfo(x.dtype).tiny  # far below the floor of the largest magnitude
    x[9] = 1e-30
    x[10] = 1e-38
    x[11], x[11, 5] = 1.0, big                     # all the others round to zero
    x[12] = (torch.arange(width, device=DEV) % 255 - 127).to(x.dtype)                   # the codes themselves
    x[13] = ((torch.arange(width, device=DEV) % 255 - 127).float() * 0.5).to(x.dtype)   # halves, when 127 is the largest
    x[13, 0] = 127
    x[14, 1] = -NAN
    check(moe, x)
    check(moe, x, scale_stride=4)


def test_halves_go_to_the_even_number(moe):
    x = torch.zeros(1, 256, device=DEV)
    x[0, :254] = torch.arange(-127, 127, device=DEV) + 0.5
    x[0, 255] = 127.0  # 127 / a is one
    q, _ = moe.moe_quantize_rows(moe.MoeQuantDesc(1, 256, moe.MOE_ROWS_F32), x)
    ref = np.rint(x.double().cpu().numpy())
    assert np.array_equal(q.cpu().numpy().astype(np.float64), ref) and ref[0, 126] == 0 and ref[0, 127] == 0 and ref[0, 128] == 2


@pytest.mark.parametrize("used", [-3, 0, 1, 8, 13, 100])
@pytest.mark.parametrize("width", [64, 2048, 7168])
def test_rows_behind_the_last_stay(moe, used, width):
    rows = 21
    x = draw(2, rows, width, False)
    q = torch.full((rows, width), 55, dtype=torch.int8, device=DEV)
    s = torch.full((rows, 1), 5.0, device=DEV)
    moe.moe_quantize_rows(moe.MoeQuantDesc(rows, width), x, q, s, torch.tensor([used], dtype=torch.int32, device=DEV))
    n = min(max(used, 0), rows)
    rq, rs = rule(x)
    assert np.array_equal(q[:n].cpu().numpy(), rq[:n]) and np.array_equal(s[:n, 0].cpu().numpy(), rs[:n])
    assert bool((q[n:] == 55).all()) and bool((s[n:] == 5.0).all())


def test_rows_past_32_bits(moe):
    # 2.4e9 elements: offsets pass 31 bits in elements and 32 in bytes
    n, width = 36000, 65536
    x = torch.zeros(n, width, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1131, 32767, 32768, n - 1], device=DEV)
    x[at] = draw(4, 5, width, False)
    q, s = moe.moe_quantize_rows(moe.MoeQuantDesc(n, width), x)
    rq, rs = rule(x[at])
    assert np.array_equal(q[at].cpu().numpy(), rq) and np.array_equal(s[at, 0].cpu().numpy(), rs)
    assert int((q != 0).any(1).sum()) == 5
