"""One MoE layer out of the library's calls: router, layout and dispatch, the
experts, combine; and for training the backward pass of all of it.

    layer = MoeLayer(hidden=7168, width=2048, num_experts=256, topk=8, ...)
    out, kept = layer.forward(x, logits, w1, w2, bias)      # kept: None without train=True
    grads = layer.backward(kept, grad_out, w1, w2)
    experts = layer.quantize(w1, w2)                        # serving with 8-bit weights
    out = layer.forward_i8(x, logits, experts, bias)

The router's logits are the caller's (a plain product of x with the router's
weights). w1 is bf16 [E, 2F, H] (gate rows, then up rows), w2 bf16 [E, H, F].
Tokens travel as BF16 records, which the first product reads where dispatch put
them. Between the passes a training step keeps the records, the 8-bit checkpoint
of gate and up and the experts' outputs; neither gate and up nor the activation
is kept in bf16. No call waits for the device, so a step can be captured in a
CUDA graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import moe


@dataclass
class MoeLayer:
    hidden: int
    width: int
    num_experts: int
    topk: int
    num_ranks: int = 1
    score: int = moe.MOE_SCORE_SOFTMAX
    num_groups: int = 1
    topk_groups: int = 1
    group_score: int = moe.MOE_GROUP_TOP2_SUM
    renormalize: bool = True
    scale: float = 1.0

    def _descs(self, n: int, logits):
        route = moe.MoeRouteDesc(
            n, self.num_experts, self.topk, self.score, self.num_groups, self.topk_groups, self.group_score,
            self.renormalize, self.scale,
            moe.MOE_LOGITS_BF16 if logits.dtype == torch.bfloat16 else moe.MOE_LOGITS_F32,
            logits.stride(0) if n > 1 else 0)
        pairs = moe.MoeDesc(n, self.topk, self.num_experts, self.num_ranks, self.hidden)
        return route, pairs

    def _want_tokens(self, what: str, t, n: int):
        """Dispatch and combine see pointers only: rows have to lie one behind the other."""
        if t.dim() != 2 or t.shape[0] != n or t.shape[1] != self.hidden:
            raise moe.MoeError(moe.MOE_ERR_SHAPE, f"{what}: [{n}, {self.hidden}] is wanted, not {list(t.shape)}")
        moe._want(what, t, torch.bfloat16, n * self.hidden)

    def _want_weights(self, what: str, w, n: int, k: int):
        if tuple(w.shape) != (self.num_experts, n, k):
            raise moe.MoeError(moe.MOE_ERR_SHAPE, f"{what}: [{self.num_experts}, {n}, {k}] is wanted, not {list(w.shape)}")

    def forward(self, x, logits, w1, w2, bias=None, train: bool = False):
        """x bf16 [N, H] (dense), logits fp32 or bf16 [N, E] -> (out bf16 [N, H], what backward needs or None)."""
        n, h, f = x.shape[0], self.hidden, self.width
        self._want_tokens("x", x, n)
        route, d = self._descs(n, logits)
        idx, weights = moe.moe_route(route, logits, bias)
        lay, rec = moe.moe_layout_dispatch(d, idx, weights, x, None)
        begin, end = moe.expert_row_ranges(lay)
        first = moe.moe_record_layout(d)["off_payload"] // 2
        rows = rec.view(torch.bfloat16)[:, first:first + h]  # the records' payload, in slot order
        rd = moe.MoeExpertDesc(self.num_experts, n * self.topk, h, f, x_stride=rows.stride(0))
        ckpt = moe.swiglu_checkpoint(moe.MoeGluDesc(n * self.topk, f), x.device) if train else (None, None)
        act = moe.moe_expert_swiglu(rd, rows, begin, end, w1, None, *ckpt)
        y = moe.moe_expert_product(moe.MoeExpertDesc(self.num_experts, n * self.topk, f, h), act, begin, end, w2)
        out = moe.moe_combine(d, moe.MOE_COMBINE_TOPK, y, idx, weights, lay["slot_of"])
        if not train:
            return out, None
        return out, dict(route=route, d=d, logits=logits, idx=idx, weights=weights, lay=lay, rows=rows, ckpt=ckpt, y=y)

    def quantize(self, w1, w2) -> tuple:
        """The experts in 8 bits for forward_i8: (w1 int8, its scales [E, 2F], w2 int8, its scales [E, H]), from bf16
        or fp32 weights."""
        out = []
        for what, w, n, k in (("w1", w1, 2 * self.width, self.hidden), ("w2", w2, self.hidden, self.width)):
            self._want_weights(what, w, n, k)
            kind = moe.MOE_ROWS_F32 if w.dtype == torch.float32 else moe.MOE_ROWS_BF16
            q, scales = moe.moe_quantize_rows(moe.MoeQuantDesc(self.num_experts * n, k, kind), w)
            out += [q.view(w.shape), scales.view(self.num_experts, n)]
        return tuple(out)

    def forward_i8(self, x, logits, experts: tuple, bias=None):
        """forward with the experts of quantize, for serving: tokens are rounded to 8 bits once and travel so, the
        activation is rounded again before the second product. x bf16 [N, H] (dense), H and F multiples of 16."""
        n, h, f = x.shape[0], self.hidden, self.width
        self._want_tokens("x", x, n)
        w1, s1, w2, s2 = experts
        for what, w, rows, k in (("w1", w1, 2 * f, h), ("w2", w2, h, f)):
            self._want_weights(what, w, rows, k)
        route, plain = self._descs(n, logits)
        d = moe.MoeDesc(n, self.topk, self.num_experts, self.num_ranks, h, moe.MOE_PAYLOAD_RAW, moe.MOE_PAYLOAD_RAW, h, 16)
        idx, weights = moe.moe_route(route, logits, bias)
        q, scales = moe.moe_quantize_rows(moe.MoeQuantDesc(n, h, scale_stride=4), x)
        lay, rec = moe.moe_layout_dispatch(d, idx, weights, q, scales)
        begin, end = moe.expert_row_ranges(lay)
        at = moe.moe_record_layout(d)
        rows = rec.view(torch.int8)[:, at["off_payload"]:at["off_payload"] + h]
        row_scales = rec.view(torch.float32)[:, at["off_scales"] // 4]
        p = n * self.topk
        act = moe.moe_expert_swiglu_i8(moe.MoeExpertI8Desc(self.num_experts, p, h, f, rows.stride(0), row_scales.stride(0)),
                                       rows, row_scales, begin, end, w1, s1)
        used = lay["expert_offset"][-1:]  # rows that hold a pair
        q, scales = moe.moe_quantize_rows(moe.MoeQuantDesc(p, f), act, num_rows=used)
        y = moe.moe_expert_product_i8(moe.MoeExpertI8Desc(self.num_experts, p, f, h), q, scales, begin, end, w2, s2)
        return moe.moe_combine(plain, moe.MOE_COMBINE_TOPK, y, idx, weights, lay["slot_of"])

    def backward(self, kept: dict, grad_out, w1, w2, grad_kind: int = moe.MOE_GRAD_F32, grad_w1=None, grad_w2=None) -> dict:
        """Gradients of x (bf16), logits (their type), w1 and w2 (grad_kind; written or, with MOE_GRAD_F32_ADD, added
        to grad_w1 and grad_w2). grad_out is bf16 [N, H], dense."""
        d, lay, rows = kept["d"], kept["lay"], kept["rows"]
        self._want_tokens("grad_out", grad_out, d.num_tokens)
        h, f, p = self.hidden, self.width, d.num_tokens * self.topk
        begin, end = moe.expert_row_ranges(lay)
        used = lay["expert_offset"][-1:]  # rows that hold a pair
        # (rows that no pair names are read by nothing below)
        grad_y = torch.empty((p, h), dtype=torch.bfloat16, device=grad_out.device)
        _, grad_weights = moe.moe_combine_backward(d, grad_out, kept["weights"], lay["slot_of"], kept["y"], p, grad_y)
        second = moe.MoeExpertDesc(self.num_experts, p, f, h)
        grad_act = moe.moe_expert_product_backward_input(second, grad_y, begin, end, w2)
        act = torch.empty_like(grad_act)
        grad_gate_up = moe.moe_swiglu_backward(moe.MoeGluDesc(p, f), *kept["ckpt"], grad_act, act=act, num_rows=used)
        grad_w2 = moe.moe_expert_product_backward_weight(second, grad_y, act, begin, end, grad_w2, grad_kind)
        first = moe.MoeExpertDesc(self.num_experts, p, h, 2 * f, x_stride=rows.stride(0))
        grad_rows = moe.moe_expert_product_backward_input(first, grad_gate_up, begin, end, w1)
        grad_w1 = moe.moe_expert_product_backward_weight(first, grad_gate_up, rows, begin, end, grad_w1, grad_kind)
        return dict(x=moe.moe_dispatch_backward(d, grad_rows, lay["slot_of"]),
                    logits=moe.moe_route_backward(kept["route"], kept["logits"], kept["idx"], grad_weights),
                    w1=grad_w1, w2=grad_w2)
