"""What is measured of the experts held in 8-bit integers: the rounding of rows to
8 bits with a scale each, the experts' products with a scale for each token and
channel, and the gated first product.

Four kinds of case:

* quant    rows of bf16 or fp32 -> int8 and one fp32 scale a row
* product  y[s] = W[e] x[s] for the rows s of every expert e, both in int8
* glu      the first product with silu(gate) * up in its epilogue
* block    rows of bf16 through all of it: quantise, first product and
           activation, quantise, second product

Sizes follow the framework's workloads: hidden 7168, top-8 of 256 experts on 8
ranks, so 32 experts a rank; 2048 is a generic expert width.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence, before its dispatch: latency is all that counts
        dict(name="quant_token", kind="quant", rows=1, width=7168, f32=False, record=True),
        # the activation of a decode batch of odd size, before the second product
        dict(name="quant_decode", kind="quant", rows=203, width=2048, f32=False, record=False),
        # the activation of a prefill batch: 4096 tokens of top-8
        dict(name="quant_prefill", kind="quant", rows=32768, width=2048, f32=False, record=False),
        # weights, once, from their 32-bit masters: 8 experts' first product, a scale for each channel
        dict(name="quant_weights", kind="quant", rows=32768, width=7168, f32=True, record=False),
        # one token's second product: eight experts, one row each
        dict(name="product_token", kind="product", rows=8, e=32, cin=2048, cout=7168, spread="one", record=False),
        # a small layer of odd sizes
        dict(name="product_odd", kind="product", rows=77, e=5, cin=1008, cout=1000, spread="zipf", record=False),
        # prefill, second product with some experts far busier than others and some idle
        dict(name="product_prefill_skewed", kind="product", rows=12345, e=32, cin=2048, cout=7168, spread="zipf", record=False),
        # one token's first product and activation, out of its dispatched records
        dict(name="glu_token", kind="glu", rows=8, e=32, cin=7168, f=2048, spread="one", record=True),
        # a decode batch's first product: every expert has a few rows, the weights are the work
        dict(name="glu_decode", kind="glu", rows=256, e=32, cin=7168, f=2048, spread="even", record=True),
        # prefill's first product, out of dispatched records
        dict(name="glu_prefill", kind="glu", rows=16384, e=32, cin=7168, f=2048, spread="even", record=True),
        # the whole block for a decode batch with some experts idle
        dict(name="block_decode", kind="block", rows=251, e=32, cin=7168, f=2048, spread="zipf"),
        # the whole block for a prefill batch
        dict(name="block_prefill", kind="block", rows=12345, e=32, cin=7168, f=2048, spread="even"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quant", "product", "glu", "block"])
    if kind == "quant":
        f32 = rng.random() < 0.5
        return dict(kind=kind, rows=_log(rng, 1, 16384 if f32 else 32768), width=16 * _log(rng, 4, 448), f32=f32,
                    record=rng.random() < 0.5)
    common = dict(rows=_log(rng, 1, 8000), e=_log(rng, 1, 32), spread=rng.choice(["one", "even", "zipf"]), cin=16 * _log(rng, 8, 300))
    if kind == "product":
        return dict(kind=kind, cout=8 * _log(rng, 16, 600), record=rng.random() < 0.5, **common)
    f = 16 * _log(rng, 8, 128)
    if kind == "glu":
        return dict(kind=kind, f=f, record=rng.random() < 0.5, **common)
    return dict(kind=kind, f=f, **common)


def _counts(case):
    """Rows of each expert (host): a fixed, case-determined partition of the rows, the same for every seed."""
    rows, e = case["rows"], case["e"]
    if case["spread"] == "one":  # the experts at the end get the rows, as evenly as may be, at most eight of them
        busy = min(e, 8)
        share = [0.0] * (e - busy) + [1.0] * busy
    elif case["spread"] == "even":
        share = [1.0 + 0.2 * math.sin(3.0 * i) for i in range(e)]
    else:  # zipf over a fixed shuffle; one in eight has none
        share = [1.0 / ((i * 5) % e + 1) ** 0.5 if e < 8 or i % 8 != 3 else 0.0 for i in range(e)]
    total, acc, ends = sum(share), 0.0, []
    for s in share:
        acc += s
        ends.append(int(round(rows * acc / total)))
    ends[-1] = rows
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


# --------------------------------------------------------------------------- inputs

def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    """Normal draws in pieces; int8: rounded, so that a row's largest are near 127 at a scale of 36."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        v = torch.randn(n, generator=g, device=DEV) * scale
        flat[i:i + n] = v.round_().clamp_(-127, 127) if dtype == torch.int8 else v
    return out


def _weights(g, s, name, e, n, k):
    s["w" + name] = _normal(g, e, n, k, scale=36.0, dtype=torch.int8)
    s["sw" + name] = torch.exp(_normal(g, e, n, scale=0.2, dtype=torch.float32)) * (k ** -0.5 / 36.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    rows = case["rows"]
    f32 = dict(dtype=torch.float32, device=DEV)
    if case["kind"] == "quant":
        width = case["width"]
        t = torch.float32 if case["f32"] else torch.bfloat16
        # rows of different size, with a few outlying channels as activations have them
        s["x"] = _normal(g, rows, width, dtype=t)
        s["x"] *= torch.exp(_normal(g, rows, 1, dtype=torch.float32)).to(t)
        s["x"][:, ::97] *= 6.0
        s["q"] = torch.empty(rows, width, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(rows, 4 if case["record"] else 1, **f32)
        return s
    counts = _counts(case)
    e, cin = case["e"], case["cin"]
    off = torch.tensor([0] + counts).cumsum(0)
    s["begin"], s["end"] = off[:-1].to(DEV, torch.int32), off[1:].to(DEV, torch.int32)
    # the plain form's plan: the experts that have rows, and each row's place in a padded batch
    busy = [i for i, c in enumerate(counts) if c]
    s["most"] = max(counts)
    s["busy"] = torch.tensor(busy, device=DEV)
    which = torch.repeat_interleave(torch.arange(len(busy)), torch.tensor([counts[i] for i in busy]))
    s["place"] = (which * s["most"] + torch.arange(rows) - off[:-1][torch.tensor(busy)][which]).to(DEV)
    if case["kind"] == "block":
        f = case["f"]
        _weights(g, s, "1", e, 2 * f, cin)
        _weights(g, s, "2", e, cin, f)
        s["x"] = _normal(g, rows, cin)
        s["q"], s["q_act"] = (torch.empty(rows, n, dtype=torch.int8, device=DEV) for n in (cin, f))
        s["scales"], s["scales_act"] = (torch.empty(rows, 1, **f32) for _ in range(2))
        s["act"] = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)
        s["y"] = torch.empty(rows, cin, dtype=torch.bfloat16, device=DEV)
        return s
    cout = 2 * case["f"] if case["kind"] == "glu" else case["cout"]
    _weights(g, s, "", e, cout, cin)
    x = _normal(g, rows, cin, scale=36.0, dtype=torch.int8)
    scales = torch.exp(_normal(g, rows, scale=0.3, dtype=torch.float32)) / 36.0
    if case["record"]:  # payload and scale of dispatched records: header, ids and weights before, 16 bytes with the scale behind
        rec = torch.zeros(rows, 80 + cin + 16, dtype=torch.int8, device=DEV)
        rec[:, 80:80 + cin] = x
        s["x"] = rec[:, 80:80 + cin]
        s["scales"] = rec.view(torch.float32)[:, (80 + cin) // 4]
        s["scales"].copy_(scales)
    else:
        s["x"], s["scales"] = x, scales
    s["y"] = torch.empty(rows, case["f"] if case["kind"] == "glu" else cout, dtype=torch.bfloat16, device=DEV)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _PLAIN[state["kind"]])(state)


def _own(s):
    """The calls a user's program makes: argument blocks are marshalled at a buffer set's first pass and kept beside the buffers."""
    if "calls" not in s:
        s["calls"] = _calls(s)
    for call in s["calls"]:
        call()
    return {"q": s["q"], "scales": s["scales"]} if s["kind"] == "quant" else {"y": s["y"]}


def _calls(s):
    from combine_moe_layout_03_gb300 import moe

    kind, rows = s["kind"], s["rows"]
    if kind == "quant":
        d = moe.MoeQuantDesc(rows, s["width"], moe.MOE_ROWS_F32 if s["f32"] else moe.MOE_ROWS_BF16, scale_stride=s["scales"].shape[1])
        return [moe.prepare_quantize_rows(d, s["x"], s["q"], s["scales"])]
    e, cin = s["e"], s["cin"]
    if kind == "block":
        f = s["f"]
        return [moe.prepare_quantize_rows(moe.MoeQuantDesc(rows, cin), s["x"], s["q"], s["scales"]),
                moe.prepare_expert_swiglu_i8(moe.MoeExpertI8Desc(e, rows, cin, f), s["q"], s["scales"], s["begin"], s["end"],
                                             s["w1"], s["sw1"], s["act"]),
                moe.prepare_quantize_rows(moe.MoeQuantDesc(rows, f), s["act"], s["q_act"], s["scales_act"]),
                moe.prepare_expert_product_i8(moe.MoeExpertI8Desc(e, rows, f, cin), s["q_act"], s["scales_act"], s["begin"], s["end"],
                                              s["w2"], s["sw2"], s["y"])]
    d = moe.MoeExpertI8Desc(e, rows, cin, s["y"].shape[1], x_stride=s["x"].stride(0), x_scale_stride=s["scales"].stride(0))
    prepare_call = moe.prepare_expert_swiglu_i8 if kind == "glu" else moe.prepare_expert_product_i8
    return [prepare_call(d, s["x"], s["scales"], s["begin"], s["end"], s["w"], s["sw"], s["y"])]


# --------------------------------------------------------------------------- plain forms, in 32 bits

def _plain_rows(x, wide=1):
    """int8 rows and their scales [rows, wide], zero behind the first. The quotients are those of the format's rule, rounded once each."""
    x = x.float()
    most = x.abs().amax(1, keepdim=True)
    fine = most < float("inf")  # false for NaN too
    a = torch.where(fine, most, torch.ones_like(most)).clamp(min=1e-30)
    top = torch.full_like(a, 127.0)  # a tensor: quotients by a number are not rounded once on every device
    q = torch.where(fine, torch.round(x * (top / a)), torch.zeros_like(x)).to(torch.int8)
    scales = torch.where(fine, a / top, torch.full_like(a, float("nan")))
    return q, torch.nn.functional.pad(scales, (0, wide - 1))


def _plain_quant(s):
    q, scales = _plain_rows(s["x"], s["scales"].shape[1])
    return {"q": q, "scales": scales}


def _plain_sums(s, x, scales, w, sw):
    """The experts' products of int8 rows, batched by expert and padded to the busiest one."""
    b = torch.zeros(len(s["busy"]) * s["most"], x.shape[1], device=x.device).index_copy(0, s["place"], x.float())
    y = torch.bmm(b.view(len(s["busy"]), s["most"], -1), w[s["busy"]].float().transpose(1, 2)) * sw[s["busy"]][:, None, :]
    return y.view(-1, y.shape[-1])[s["place"]] * scales.view(-1, 1)


def _plain_glu_of(v):
    gate, up = v.chunk(2, 1)
    return (gate / (1.0 + torch.exp(-gate)) * up).bfloat16()


def _plain_product(s):
    return {"y": _plain_sums(s, s["x"], s["scales"], s["w"], s["sw"]).bfloat16()}


def _plain_glu(s):
    return {"y": _plain_glu_of(_plain_sums(s, s["x"], s["scales"], s["w"], s["sw"]))}


def _plain_block(s):
    act = _plain_glu_of(_plain_sums(s, *_plain_rows(s["x"]), s["w1"], s["sw1"]))
    return {"y": _plain_sums(s, *_plain_rows(act), s["w2"], s["sw2"]).bfloat16()}


_PLAIN = {"quant": _plain_quant, "product": _plain_product, "glu": _plain_glu, "block": _plain_block}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    rows = case["rows"]
    if case["kind"] == "quant":
        n = rows * case["width"]
        return {"bytes": n * (5 if case["f32"] else 3) + rows * (16 if case["record"] else 4), "flops": 4 * n}
    cin = case["cin"]
    busy = sum(c > 0 for c in _counts(case))
    if case["kind"] == "product":
        cout = case["cout"]
        return {"bytes": rows * (cin + 4 + 2 * cout) + busy * cout * (cin + 4), "flops": 2 * rows * cin * cout}
    f = case["f"]
    if case["kind"] == "glu":
        return {"bytes": rows * (cin + 4 + 2 * f) + busy * 2 * f * (cin + 4), "flops": 4 * rows * cin * f}
    return {"bytes": rows * 4 * cin + busy * (2 * f * (cin + 4) + cin * (f + 4)), "flops": 6 * rows * cin * f}


# --------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quant":
        q, scales = _exact_rows(s["x"])
        out = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        out[:, 0] = scales
        return {"q": q.to(torch.int8), "scales": out}
    if kind == "block":
        act = _exact_glu(_exact_sums(s, *_exact_rows(s["x"]), s["w1"], s["sw1"])).to(torch.bfloat16)
        return {"y": _exact_sums(s, *_exact_rows(act), s["w2"], s["sw2"])}
    y = _exact_sums(s, s["x"], s["scales"], s["w"], s["sw"])
    return {"y": _exact_glu(y) if kind == "glu" else y}


def _exact_rows(x):
    """Codes by the format's rule (the quotient and the product in 32 bits, halves to the even number), scales in 64 bits."""
    q = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    scales = torch.empty(x.shape[0], dtype=torch.float64, device=DEV)
    for lo in range(0, x.shape[0], 4096):
        part = x[lo:lo + 4096].float()
        a = part.abs().max(1).values.clamp(min=1e-30)
        m = (part * torch.div(torch.full_like(a, 127.0), a)[:, None]).double()
        low = torch.floor(m)
        over = m - low
        up = (over > 0.5) | ((over == 0.5) & (torch.remainder(low, 2.0) == 1.0))
        q[lo:lo + 4096] = low + up
        scales[lo:lo + 4096] = a.double() / 127.0
    return q, scales


def _exact_sums(s, x, scales, w, sw):
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=DEV)
    lo = 0
    for e, c in enumerate(_counts(s)):
        if c:
            y[lo:lo + c] = (x[lo:lo + c].double() @ w[e].double().t()) * scales[lo:lo + c].double()[:, None] * sw[e].double()
        lo += c
    return y


def _exact_glu(v):
    f = v.shape[1] // 2
    return v[:, :f] * torch.special.expit(v[:, :f]) * v[:, f:]
