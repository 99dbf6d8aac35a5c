"""Calls on a stream other than the current one: their outputs are not memory
that the current stream still has work queued for."""
import pytest
import torch

from layer_reference import product, ranges, route
from test_gpu_experts import DEV, normal, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_03_gb300 import moe as m
    yield m
    assert m.moe_device_status() == m.MOE_OK


def behind_pending_work(call, like):
    """call() while the current stream is still to write to blocks of the outputs' sizes that it has given back."""
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some tens of milliseconds
    for t in like:
        for _ in range(2):
            torch.empty_like(t).view(torch.uint8).fill_(0x7b)
    out = call()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream(moe, raw):
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    counts, cin, f = [40, 0, 77], 256, 128
    rows = sum(counts)
    begin, end = ranges(counts, DEV)
    x, w, dy = whole(1, rows, cin), whole(2, 3, 2 * f, cin), whole(3, rows, 2 * f)
    d, gd = moe.MoeExpertDesc(3, rows, cin, 2 * f), moe.MoeGluDesc(rows, f)
    gu, da = normal(4, rows, 2 * f), normal(5, rows, f)
    ckpt, scales = moe.swiglu_checkpoint(gd, DEV)
    moe.moe_swiglu(gd, gu, None, ckpt, scales)
    logits = torch.randn(300, 32, device=DEV)
    rd = moe.MoeRouteDesc(300, 32, 4)
    idx, weights = moe.moe_route(rd, logits)
    assert (idx.cpu().numpy() == route(logits, None, 4, "softmax", 1, 1, "max", True, 1.0)[0]).all()
    assert torch.equal(moe.moe_expert_product(d, x, begin, end, w), product(x, begin, end, w)[0].to(torch.bfloat16))
    calls = [lambda **k: moe.moe_route(rd, logits, **k), lambda **k: moe.moe_route_backward(rd, logits, idx, weights, **k),
             lambda **k: moe.moe_swiglu(gd, gu, **k), lambda **k: moe.moe_swiglu_backward(gd, ckpt, scales, da, **k),
             lambda **k: moe.moe_expert_product(d, x, begin, end, w, **k),
             lambda **k: moe.moe_expert_swiglu(moe.MoeExpertDesc(3, rows, cin, f), x, begin, end, w, **k),
             lambda **k: moe.moe_expert_product_backward_input(d, dy, begin, end, w, **k),
             lambda **k: moe.moe_expert_product_backward_weight(d, dy, x, begin, end, **k)]
    for call in calls:
        want = call()
        want = want if isinstance(want, tuple) else (want,)
        got = behind_pending_work(lambda: call(stream=stream), want)
        got = got if isinstance(got, tuple) else (got,)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_default_stream_by_its_handle(moe):
    logits = torch.randn(30, 16, device=DEV)
    d = moe.MoeRouteDesc(30, 16, 2)
    torch.cuda.synchronize()
    a, b = moe.moe_route(d, logits), moe.moe_route(d, logits, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
