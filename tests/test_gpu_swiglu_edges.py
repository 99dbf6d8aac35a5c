"""What infinity and NaN do to a checkpoint's group of 128, and to the gradients
that are taken from it."""
import pytest
import torch

from layer_reference import kept
from test_gpu_swiglu import DEV, normal

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("f", [264, 384])
def test_infinity_takes_its_group_and_nan_only_itself(f):
    from combine_moe_layout_03_gb300 import moe
    gu, da = normal(1, 6, 2 * f), normal(2, 6, f)
    hit = torch.zeros(6, 2 * f, dtype=torch.bool, device=DEV)
    for r, c, v in ((0, 5, INF), (1, 130, NAN), (2, f + 7, -INF), (3, f + 257, NAN), (4, 0, NAN), (4, 9, INF)):
        gu[r, c] = v
        hit[r, c] = True
    gu[5, :128] = NAN  # a group of nothing else
    hit[5, :128] = True
    d = moe.MoeGluDesc(6, f)
    n = d.groups
    ckpt, scales = moe.swiglu_checkpoint(d, DEV)
    act = moe.moe_swiglu(d, gu, None, ckpt, scales)
    dgu = moe.moe_swiglu_backward(d, ckpt, scales, da)
    group = torch.arange(f, device=DEV) // 128
    lost = torch.zeros(6, 2 * f, dtype=torch.bool, device=DEV)  # groups with an infinity
    for h in range(2):
        v = gu[:, h * f:(h + 1) * f].float()
        codes, sc = kept(torch.nan_to_num(v, nan=0.0, posinf=INF, neginf=-INF))
        assert torch.equal(scales[:, h * n:(h + 1) * n], sc)
        mine = ckpt[:, h * f:(h + 1) * f].view(torch.float8_e4m3fn).float()
        on = hit[:, h * f:(h + 1) * f]
        assert bool(torch.isnan(mine[on]).all()) and torch.equal(mine[~on], codes.float()[~on])
        lost[:, h * f:(h + 1) * f] = torch.isinf(sc)[:, group]
    # what a place's two kept values leave finite stays finite
    gone = (hit | lost)[:, :f] | (hit | lost)[:, f:]
    assert bool(torch.isfinite(dgu[:, :f][~gone]).all()) and bool(torch.isfinite(dgu[:, f:][~gone]).all())
    assert bool(torch.isnan(dgu[:, :f][gone]).all())
    touched = hit[:, :f] | hit[:, f:]
    assert bool(torch.isfinite(act[~touched]).all()) and not bool(torch.isfinite(act[touched]).any())
