"""What is measured of the operators around MoE dispatch and combine: the router, the
experts' products and the gated activation with its 8-bit checkpoint.

Six kinds of case:

* route        logits -> the chosen experts' ids and weights
* route_train  the same, and the gradient of the logits from that of the weights
* swiglu       gate|up rows -> activation + e4m3 checkpoint, then the backward pass
               from the checkpoint alone (activation again, gradient of gate|up)
* product      y[s] = W[e] x[s] for the rows s of every expert e
* glu          the first product with the activation in its epilogue; with
               "train", also its checkpoint and the activation's backward from it
* backward     a product's input gradient and weight gradient

Routing follows the framework's workloads: 256 experts in 8 groups, top-8, hidden
7168 and 8 ranks, so 32 experts a rank; 2048 is a generic expert width.
"""
import math

import torch

own = False

DEV = "cuda"
NEG = float("-inf")
BIG = torch.finfo(torch.float32).max


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: latency is all that counts
        dict(name="route_token", kind="route", n=1, e=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             group_score="top2", renorm=True, scale=2.5, bf16=False, masked=0.0),
        # a decode batch of odd size; bf16 logits; a router whose outputs are padded to a stride, some experts taken out
        dict(name="route_decode", kind="route", n=203, e=160, k=6, score="softmax", bias=False, groups=1, topk_groups=1,
             group_score="max", renorm=False, scale=1.0, bf16=True, masked=0.3),
        # training, prefill-sized batch of the framework's skewed workload: groups, balance bias, forward and backward
        dict(name="route_train_groups", kind="route_train", n=16384, e=256, k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renorm=True, scale=2.5, bf16=False, masked=0.0),
        # training with a plain softmax router in bf16; every logit gets a gradient
        dict(name="route_train_softmax", kind="route_train", n=4096, e=256, k=8, score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renorm=False, scale=1.0, bf16=True, masked=0.0),
        # a small batch of rows whose width is no multiple of the checkpoint's group
        dict(name="swiglu_small", kind="swiglu", rows=77, f=1000),
        # a prefill batch's rows: 4096 tokens of top-8
        dict(name="swiglu_prefill", kind="swiglu", rows=32768, f=2048),
        # one token's second product: eight experts, one row each
        dict(name="down_token", kind="product", rows=8, e=32, cin=2048, cout=7168, spread="one", record=False),
        # a decode batch's first product and activation: every expert has a few rows, the weights are the work
        dict(name="glu_decode", kind="glu", rows=256, e=32, cin=7168, f=2048, spread="even", record=False, train=False),
        # prefill, second product with some experts far busier than others and some idle
        dict(name="down_prefill_skewed", kind="product", rows=12345, e=32, cin=2048, cout=7168, spread="zipf", record=False),
        # training, first product out of dispatched records, with the checkpoint and the activation's backward
        dict(name="glu_train", kind="glu", rows=16384, e=32, cin=7168, f=2048, spread="even", record=True, train=True),
        # a small layer's backward, ragged and with idle experts, weight gradient in bf16
        dict(name="backward_small", kind="backward", rows=251, e=16, cin=1024, cout=1016, spread="zipf", f32=False),
        # training, the backward pass of the first product: both gradients, the weight gradient in 32 bits
        dict(name="backward_train", kind="backward", rows=16384, e=32, cin=7168, cout=4096, spread="even", f32=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm; whole multiples of 1024 are left to the listed cases."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + (v % 1024 == 0)


def draw(rng):
    kind = rng.choice(["route", "route_train", "swiglu", "product", "glu", "backward"])
    if kind in ("route", "route_train"):
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * _log(rng, 4, 256 // groups if groups > 1 else 512)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(12, topk_groups * (e // groups)))
        return dict(kind=kind, n=_log(rng, 1, 8192), e=e, k=k, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, group_score=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.0, 0.3]))
    if kind == "swiglu":
        return dict(kind=kind, rows=_log(rng, 1, 16384), f=8 * _log(rng, 8, 256))
    common = dict(rows=_log(rng, 1, 6000), e=_log(rng, 1, 32), spread=rng.choice(["one", "even", "zipf"]))
    cin, cout = 8 * _log(rng, 16, 383), 8 * _log(rng, 16, 383)
    if kind == "product":
        return dict(kind=kind, cin=cin, cout=cout, record=rng.random() < 0.5, **common)
    if kind == "glu":
        return dict(kind=kind, cin=cin, f=8 * _log(rng, 16, 256), record=rng.random() < 0.5, train=rng.random() < 0.5, **common)
    return dict(kind=kind, cin=cin, cout=cout, f32=rng.random() < 0.5, **common)


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
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV) * scale
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["kind"] in ("route", "route_train"):
        n, e, k = case["n"], case["e"], case["k"]
        t = torch.bfloat16 if case["bf16"] else torch.float32
        logits = _normal(g, n, e, scale=1.5, dtype=t)
        if case["masked"]:  # experts taken out for a token, and for the last token every one of them
            gone = torch.rand(n, e, generator=g, device=DEV) < case["masked"]
            gone[-1] = n > 1
            logits.masked_fill_(gone, NEG)
        s["logits"] = logits
        s["bias"] = _normal(g, e, scale=0.05, dtype=torch.float32) if case["bias"] else None
        s["topk_idx"] = torch.empty(n, k, dtype=torch.int32, device=DEV)
        s["topk_weights"] = torch.empty(n, k, dtype=torch.float32, device=DEV)
        if case["kind"] == "route_train":
            s["grad_weights"] = _normal(g, n, k, dtype=torch.float32)
            s["grad_logits"] = torch.empty_like(logits)
        return s
    if case["kind"] == "swiglu":
        rows, f = case["rows"], case["f"]
        s["gate_up"] = _normal(g, rows, 2 * f)
        s["grad_act"] = _normal(g, rows, f)
        _glu_buffers(s, rows, f)
        return s
    counts = _counts(case)
    rows, e = case["rows"], case["e"]
    off = torch.tensor([0] + counts).cumsum(0)
    s["begin"], s["end"] = off[:-1].to(DEV, torch.int32), off[1:].to(DEV, torch.int32)
    # the plain form's plan: the experts that have rows, and each row's place in a padded batch
    busy = [i for i, c in enumerate(counts) if c]
    s["most"] = max(counts)
    s["busy"] = torch.tensor(busy, device=DEV)
    which = torch.repeat_interleave(torch.arange(len(busy)), torch.tensor([counts[i] for i in busy]))
    s["place"] = (which * s["most"] + torch.arange(rows) - off[:-1][torch.tensor(busy)][which]).to(DEV)
    cin = case["cin"]
    cout = 2 * case["f"] if case["kind"] == "glu" else case["cout"]
    s["w"] = _normal(g, e, cout, cin, scale=cin ** -0.5)
    if case.get("record"):  # the payload of dispatched records: 80 bytes of header, ids and weights before each row
        rec = torch.zeros(rows, cin + 40, dtype=torch.bfloat16, device=DEV)
        rec[:, 40:] = _normal(g, rows, cin)
        s["x"] = rec[:, 40:]
    else:
        s["x"] = _normal(g, rows, cin)
    if case["kind"] == "product":
        s["y"] = torch.empty(rows, cout, dtype=torch.bfloat16, device=DEV)
    elif case["kind"] == "glu":
        _glu_buffers(s, rows, case["f"], case["train"])
        if case["train"]:
            s["grad_act"] = _normal(g, rows, case["f"])
    else:
        s["grad_y"] = _normal(g, rows, cout)
        s["grad_x"] = torch.empty(rows, cin, dtype=torch.bfloat16, device=DEV)
        s["grad_w"] = torch.empty(e, cout, cin, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
    return s


def _glu_buffers(s, rows, f, train=True):
    s["act"] = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)
    s["ckpt"] = s["ckpt_scales"] = None
    if train:
        s["ckpt"] = torch.empty(rows, 2 * f, dtype=torch.uint8, device=DEV)
        s["ckpt_scales"] = torch.empty(rows, 2 * -(-f // 128), dtype=torch.float32, device=DEV)
        s["grad_gate_up"] = torch.empty(rows, 2 * f, dtype=torch.bfloat16, device=DEV)
        s["act_again"] = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)


# --------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _PLAIN[state["kind"]])(state)


def _own(s):
    """The calls a user's program makes: argument blocks are marshalled at a buffer set's first pass and kept beside the buffers."""
    if "calls" not in s:
        s["calls"] = _calls(s)
    for call in s["calls"]:
        call()
    return _outputs(s)


def _outputs(s):
    kind = s["kind"]
    if kind == "route":
        return {"idx": s["topk_idx"], "weights": s["topk_weights"]}
    if kind == "route_train":
        return {"idx": s["topk_idx"], "weights": s["topk_weights"], "grad_logits": s["grad_logits"]}
    if kind == "product":
        return {"y": s["y"]}
    if kind == "backward":
        return {"grad_x": s["grad_x"], "grad_w": s["grad_w"]}
    if kind == "glu" and not s["train"]:
        return {"act": s["act"]}
    return {"act": s["act"], "grad_gate_up": s["grad_gate_up"], "act_again": s["act_again"]}


def _calls(s):
    from combine_moe_layout_03_gb300 import moe

    kind = s["kind"]
    if kind in ("route", "route_train"):
        d = moe.MoeRouteDesc(
            num_tokens=s["n"], num_experts=s["e"], topk=s["k"],
            score=moe.MOE_SCORE_SIGMOID if s["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
            num_groups=s["groups"], topk_groups=s["topk_groups"],
            group_score=moe.MOE_GROUP_TOP2_SUM if s["group_score"] == "top2" else moe.MOE_GROUP_MAX,
            renormalize=s["renorm"], scale=s["scale"],
            logits_kind=moe.MOE_LOGITS_BF16 if s["bf16"] else moe.MOE_LOGITS_F32)
        calls = [moe.prepare_route(d, s["logits"], s["bias"], s["topk_idx"], s["topk_weights"])]
        if kind == "route_train":
            calls.append(moe.prepare_route_backward(d, s["logits"], s["topk_idx"], s["grad_weights"], s["grad_logits"]))
        return calls
    if kind == "swiglu":
        d = moe.MoeGluDesc(rows=s["rows"], width=s["f"])
        return [moe.prepare_swiglu(d, s["gate_up"], s["act"], s["ckpt"], s["ckpt_scales"]),
                moe.prepare_swiglu_backward(d, s["ckpt"], s["ckpt_scales"], s["grad_act"], s["grad_gate_up"], s["act_again"])]
    x, w = s["x"], s["w"]
    d = moe.MoeExpertDesc(num_experts=s["e"], rows=s["rows"], in_features=s["cin"],
                          out_features=s["f"] if kind == "glu" else s["cout"], x_stride=x.stride(0))
    if kind == "product":
        return [moe.prepare_expert_product(d, x, s["begin"], s["end"], w, s["y"])]
    if kind == "glu":
        calls = [moe.prepare_expert_swiglu(d, x, s["begin"], s["end"], w, s["act"], s["ckpt"], s["ckpt_scales"])]
        if s["train"]:
            calls.append(moe.prepare_swiglu_backward(moe.MoeGluDesc(rows=s["rows"], width=s["f"]), s["ckpt"], s["ckpt_scales"],
                                                     s["grad_act"], s["grad_gate_up"], s["act_again"]))
        return calls
    return [moe.prepare_expert_product_backward_input(d, s["grad_y"], s["begin"], s["end"], w, s["grad_x"]),
            moe.prepare_expert_product_backward_weight(d, s["grad_y"], x, s["begin"], s["end"], s["grad_w"],
                                                       moe.MOE_GRAD_F32 if s["f32"] else moe.MOE_GRAD_BF16)]


# --------------------------------------------------------------------------- plain forms (32 bits; 64 where experts are ordered)

def _plain_scores(s, x):
    """Scores of the logits x; -inf and NaN count as absent."""
    x = torch.where(x > NEG, x, torch.full_like(x, NEG)).clamp(max=BIG)
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(-1, keepdim=True).values
    p = torch.exp(x - torch.where(top > NEG, top, torch.zeros_like(top)))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_choose(s):
    x = s["logits"].double()
    n, e = x.shape
    score = _plain_scores(s, x)
    key = x.clamp(max=BIG) if s["bias"] is None else score + s["bias"].double()
    ok = (x > NEG) & (key > NEG)
    key = torch.where(ok, key, torch.full_like(key, NEG))
    if s["groups"] > 1:
        by = (n, s["groups"], e // s["groups"])
        if s["group_score"] == "max":
            rank = key.view(by).max(-1).values
        else:
            v = torch.where(ok, score, torch.full_like(score, NEG)) if s["bias"] is None else key
            two = v.view(by).sort(dim=-1, descending=True).values[..., :2]
            rank = torch.where(two[..., :1] > NEG, torch.where(two > NEG, two, torch.zeros_like(two)), two).sum(-1)
        first = rank.sort(dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        take = torch.zeros(by[:2], dtype=torch.bool, device=x.device).scatter(1, first, True)
        key = torch.where(take[..., None].expand(by).reshape(n, e), key, torch.full_like(key, NEG))
    v, idx = key.sort(dim=-1, descending=True, stable=True)
    v, idx = v[:, :s["k"]], idx[:, :s["k"]]
    return torch.where(v > NEG, idx, torch.full_like(idx, -1)).to(torch.int32)


def _plain_weights(s, idx):
    score = _plain_scores(s, s["logits"].float())
    w = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0).long()), torch.zeros((), device=idx.device))
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return w * s["scale"]


def _plain_route(s):
    idx = _plain_choose(s)
    return {"idx": idx, "weights": _plain_weights(s, idx)}


def _plain_route_train(s):
    idx = _plain_choose(s)
    w = _plain_weights(s, idx)
    g = torch.where(idx >= 0, s["grad_weights"], torch.zeros((), device=idx.device))
    at = idx.clamp(min=0).long()
    x = s["logits"].float()
    score = _plain_scores(s, x)
    zero = torch.zeros_like(score)
    spread = lambda v: zero.scatter_add(1, at, torch.where(idx >= 0, v, torch.zeros_like(v)))  # noqa: E731
    if s["score"] == "sigmoid":
        fall = 1.0 / (1.0 + torch.exp(x.clamp(min=-BIG, max=BIG).gather(1, at)))
        if s["renorm"]:
            d = spread(w * fall * (g - (g * w).sum(-1, keepdim=True) / s["scale"]))
        else:
            d = spread(w * fall * g)
    elif s["renorm"]:
        d = spread(w * (g - (g * w).sum(-1, keepdim=True) / s["scale"]))
    else:
        d = score * (spread(g * s["scale"]) - (g * w).sum(-1, keepdim=True))
    return {"idx": idx, "weights": w, "grad_logits": d.to(s["logits"].dtype)}


def _plain_kept(v):
    """What e4m3 codes with a 32-bit scale per 128 channels keep of v [rows, f] (f padded to whole groups)."""
    rows, f = v.shape
    p = torch.nn.functional.pad(v, (0, -f % 128)).view(rows, -1, 128)
    a = p.abs().amax(-1, keepdim=True).clamp(min=1e-4)
    most = torch.full_like(a, 448.0)  # a tensor: quotients by a number are not rounded once on every device
    q = (p * (most / a)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * (a / most)).view(rows, -1)[:, :f]


def _plain_glu(gate, up, grad=None):
    out = {"act": (gate / (1.0 + torch.exp(-gate)) * up).bfloat16()}
    if grad is not None:
        gate, up = _plain_kept(gate), _plain_kept(up)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        grad = grad.float()
        out["grad_gate_up"] = torch.cat([grad * up * sig * (1.0 + gate * (1.0 - sig)), grad * gate * sig], -1).bfloat16()
        out["act_again"] = (gate * sig * up).bfloat16()
    return out


def _plain_swiglu(s):
    v = s["gate_up"].float()
    return _plain_glu(v[:, :s["f"]], v[:, s["f"]:], s["grad_act"])


def _batched(s, x):
    """Rows by expert, padded to the busiest one: [experts with rows, most, width] in 32 bits."""
    out = torch.zeros(len(s["busy"]) * s["most"], x.shape[1], device=x.device)
    return out.index_copy(0, s["place"], x.float()).view(len(s["busy"]), s["most"], -1)


def _rows(s, b):
    return b.reshape(-1, b.shape[-1])[s["place"]]


def _plain_rows(s):
    w = s["w"][s["busy"]].float()
    return _rows(s, torch.bmm(_batched(s, s["x"]), w.transpose(1, 2)))


def _plain_product(s):
    return {"y": _plain_rows(s).bfloat16()}


def _plain_expert_glu(s):
    v = _plain_rows(s)
    return _plain_glu(v[:, :s["f"]], v[:, s["f"]:], s["grad_act"] if s["train"] else None)


def _plain_backward(s):
    dy = _batched(s, s["grad_y"])
    dx = _rows(s, torch.bmm(dy, s["w"][s["busy"]].float())).bfloat16()
    dw = torch.zeros(s["w"].shape, dtype=torch.float32 if s["f32"] else torch.bfloat16, device=dx.device)
    dw[s["busy"]] = torch.bmm(dy.transpose(1, 2), _batched(s, s["x"])).to(dw.dtype)
    return {"grad_x": dx, "grad_w": dw}


_PLAIN = {"route": _plain_route, "route_train": _plain_route_train, "swiglu": _plain_swiglu, "product": _plain_product,
          "glu": _plain_expert_glu, "backward": _plain_backward}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind in ("route", "route_train"):
        n, e, k = case["n"], case["e"], case["k"]
        t = 2 if case["bf16"] else 4
        b = n * e * t + n * k * 8 + (4 * e if case["bias"] else 0)
        f = 10 * n * e
        if kind == "route_train":  # the gradient's rows are written, and the weights' gradient read
            b += n * e * t + n * k * 4
            f += 6 * n * e
        return {"bytes": b, "flops": f}
    glu = lambda rows, f, gate_up: rows * ((4 * f if gate_up else 0) + 2 * f + 2 * f + 4 * f + 2 * f + 8 * -(-f // 128) + 2 * f)  # noqa: E731
    if kind == "swiglu":
        rows, f = case["rows"], case["f"]
        return {"bytes": glu(rows, f, True), "flops": 40 * rows * f}
    rows, cin = case["rows"], case["cin"]
    busy = sum(c > 0 for c in _counts(case))
    if kind == "product":
        cout = case["cout"]
        return {"bytes": 2 * (rows * (cin + cout) + busy * cin * cout), "flops": 2 * rows * cin * cout}
    if kind == "glu":
        f = case["f"]
        b = 2 * (rows * cin + busy * cin * 2 * f) + (glu(rows, f, False) if case["train"] else 2 * rows * f)
        return {"bytes": b, "flops": 4 * rows * cin * f}
    cout = case["cout"]
    b = 2 * (rows * (2 * cin + cout) + busy * cin * cout) + (4 if case["f32"] else 2) * case["e"] * cin * cout
    return {"bytes": b, "flops": 4 * rows * cin * cout}


# --------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("route", "route_train"):
        return _exact_route(s)
    if kind == "swiglu":
        v = s["gate_up"].double()
        return _exact_glu(s, v[:, :s["f"]], v[:, s["f"]:], s["grad_act"])
    counts = _counts(case)
    begin = [sum(counts[:i]) for i in range(len(counts))]
    spans = [(e, b, b + c) for e, (b, c) in enumerate(zip(begin, counts)) if c]
    if kind == "backward":
        dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV)
        for e, lo, hi in spans:
            dy = s["grad_y"][lo:hi].double()
            dx[lo:hi] = dy @ s["w"][e].double()
            dw[e] = dy.t() @ s["x"][lo:hi].double()
        return {"grad_x": dx, "grad_w": dw}
    y = torch.zeros(s["x"].shape[0], s["w"].shape[1], dtype=torch.float64, device=DEV)
    for e, lo, hi in spans:
        y[lo:hi] = s["x"][lo:hi].double() @ s["w"][e].double().t()
    if kind == "product":
        return {"y": y}
    return _exact_glu(s, y[:, :s["f"]], y[:, s["f"]:], s["grad_act"] if s["train"] else None)


def _exact_kept(v):
    """e4m3 by its definition: the nearest multiple of 2^(exponent - 3), ties to even, exponent >= -6, largest 448."""
    out = torch.empty_like(v)
    for lo in range(0, v.shape[1], 128):
        part = v[:, lo:lo + 128]
        a = part.abs().amax(1, keepdim=True).float().clamp(min=1e-4)
        most = torch.full_like(a, 448.0)
        m = (part.float() * (most / a)).double()  # the format's rule: both quotients and the product in 32 bits
        step = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, lo:lo + 128] = torch.round(m / step).mul(step).clamp(-448.0, 448.0) * (a / most).double()
    return out


def _exact_glu(s, gate, up, grad):
    out = {"act": gate * torch.special.expit(gate) * up}
    if grad is None:
        return out
    gate, up, grad = _exact_kept(gate), _exact_kept(up), grad.double()
    sig = torch.special.expit(gate)
    d_gate = grad * up * (sig + gate * sig * torch.special.expit(-gate))
    out["grad_gate_up"] = torch.cat([d_gate, grad * gate * sig], 1)
    out["act_again"] = gate * sig * up
    return out


def _exact_route(s):
    x = s["logits"].double()
    n, e = x.shape
    here = torch.arange(n, device=DEV)
    dead = torch.isnan(x) | (x == NEG)
    x = x.clamp(max=BIG).masked_fill(dead, NEG)
    if s["score"] == "sigmoid":
        score = torch.special.expit(x)
    else:
        score = torch.softmax(x, -1).nan_to_num(0.0)
    key = (score + s["bias"].double() if s["bias"] is not None else x).masked_fill(dead, NEG)
    if s["groups"] > 1:
        size = e // s["groups"]
        rank = torch.full((n, s["groups"]), NEG, dtype=torch.float64, device=DEV)
        for q in range(s["groups"]):
            part = key[:, q * size:(q + 1) * size]
            if s["group_score"] == "max":
                rank[:, q] = part.amax(1)
            else:
                part = (part if s["bias"] is not None else score[:, q * size:(q + 1) * size].masked_fill(dead[:, q * size:(q + 1) * size], NEG)).clone()
                best = part.amax(1)
                part[here, part.argmax(1)] = NEG
                second = part.amax(1)
                rank[:, q] = best + second.masked_fill(second == NEG, 0.0)
        keep = torch.zeros(n, s["groups"], dtype=torch.bool, device=DEV)
        for _ in range(s["topk_groups"]):
            first = (rank == rank.amax(1, keepdim=True)).int().argmax(1)
            keep[here, first] = True
            rank[here, first] = NEG
            rank = rank.masked_fill(keep, NEG)
        key = key.masked_fill(~keep.repeat_interleave(size, 1), NEG)
    idx = torch.full((n, s["k"]), -1, dtype=torch.int64, device=DEV)
    for j in range(s["k"]):
        best = key.amax(1)
        first = (key == best[:, None]).int().argmax(1)
        idx[:, j] = torch.where(best > NEG, first, torch.full_like(first, -1))
        key[here, first] = NEG
    got = idx >= 0
    at = idx.clamp(min=0)
    chosen = score.gather(1, at) * got
    total = chosen.sum(1, keepdim=True).clamp(min=1e-300)
    w = s["scale"] * (chosen / total if s["renorm"] else chosen)
    out = {"idx": idx.to(torch.int32), "weights": w}
    if s["kind"] == "route_train":
        g = s["grad_weights"].double() * got
        # derivative of the loss by each score, then through the score
        if s["renorm"]:
            by = s["scale"] * (g - (g * chosen).sum(1, keepdim=True) / total) / total * got
        else:
            by = s["scale"] * g
        d = torch.zeros_like(score).scatter_add_(1, at, by)
        if s["score"] == "sigmoid":
            out["grad_logits"] = d * score * torch.special.expit(-x)
        else:
            out["grad_logits"] = score * (d - (d * score).sum(1, keepdim=True))
    return out
