"""Plain 64-bit forms of the router, the gated activation and the experts'
products, for the tests (torch, on whatever device the inputs are)."""
import numpy as np
import torch

NEG = float("-inf")
HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative
UNIT = 2.0 ** -24      # half a step of fp32, relative


def scores(x, score):
    """x float64 [N, E], -inf where an expert is taken out."""
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    top = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(x > NEG, np.exp(x - top), 0.0)
    den = p.sum(1, keepdims=True)
    return np.divide(p, den, out=np.zeros_like(p), where=den > 0)


def clean(logits):
    x = logits.detach().double().cpu().numpy()
    return np.where(x > NEG, np.minimum(x, np.finfo(np.float32).max), NEG)  # NaN compares false


def route(logits, bias, k, score, groups, topk_groups, group_score, renorm, scale):
    """(ids [N, k], weights float64 [N, k]) row by row."""
    x = clean(logits)
    n, e = x.shape
    with np.errstate(over="ignore"):
        s = scores(x, score)
    b = None if bias is None else bias.double().cpu().numpy()
    ids, w = np.full((n, k), -1, np.int64), np.zeros((n, k))
    for t in range(n):
        key = x[t] if b is None else s[t] + b
        key = np.where((x[t] > NEG) & (key > NEG), key, NEG)
        left = set(range(e))
        if groups > 1:
            per, count = e // groups, []
            for g in range(groups):
                mine = [i for i in range(g * per, (g + 1) * per) if key[i] > NEG]
                v = sorted((key[i] if b is not None or group_score == "max" else s[t][i] for i in mine), reverse=True)
                count.append(NEG if not v else v[0] if group_score == "max" or len(v) < 2 else v[0] + v[1])
            first = sorted(range(groups), key=lambda g: (-count[g], g))[:topk_groups]
            left = {i for g in first for i in range(g * per, (g + 1) * per)}
        order = sorted((i for i in left if key[i] > NEG), key=lambda i: (-key[i], i))[:k]
        ids[t, :len(order)] = order
        v = s[t][order]
        if renorm and len(order):  # relative to the largest, as small scores keep their ratios
            logs = x[t][order] if score == "softmax" else -np.logaddexp(0.0, -x[t][order])
            v = np.exp(logs - logs.max())
            v = v / v.sum()
        w[t, :len(order)] = scale * v
    return ids, w


def route_weights(x, ids, score, renorm, scale):
    """Weights of given ids as a differentiable function of x (torch float64 [N, E])."""
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, -1)
    got = ids >= 0
    v = torch.where(got, p.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=p.dtype))
    if renorm:
        v = v / v.sum(1, keepdim=True).clamp(min=1e-300)
    return scale * v


def kept(v):
    """(codes' values, scales) of e4m3 per 128 channels by the format's fp32 rule, v fp32 [rows, F]."""
    rows, f = v.shape
    p = torch.nn.functional.pad(v, (0, -f % 128)).view(rows, -(-f // 128), 128)
    a = p.abs().amax(-1).clamp(min=1e-4)
    most = torch.full_like(a, 448.0)  # a tensor: a quotient by a number is not an IEEE division on the GPU
    codes = (p * (most / a)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(rows, -(-f // 128) * 128)[:, :f], a / most


def kept_values(codes, scales, f):
    """float64 values of checkpoint codes uint8 [rows, f] of one half and its scales."""
    return codes.view(torch.float8_e4m3fn).float().double() * scales.double().repeat_interleave(128, 1)[:, :f]


def near(got, ref, lim):
    """got (bf16) is within lim of ref, or is ref's own rounding (as where that overflows)."""
    return bool((((got.double() - ref).abs() <= lim) | (got == ref.to(got.dtype))).all())


def swiglu(g, u):
    return g * torch.sigmoid(g) * u


def ranges(counts, device, start=0):
    off = torch.tensor([start] + list(counts)).cumsum(0)
    return off[:-1].to(device, torch.int32), off[1:].to(device, torch.int32)


def product(x, begin, end, w):
    """float64 y [rows, N] and the sums of magnitudes, both zero outside the ranges."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e, (b, t) in enumerate(zip(begin.tolist(), end.tolist())):
        if t > b:
            a, m = x[b:t].double(), w[e].double()
            y[b:t], mag[b:t] = a @ m.t(), a.abs() @ m.abs().t()
    return y, mag
