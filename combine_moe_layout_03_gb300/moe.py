"""Thin Python binding of libmoe.so (include/moe.h) through ctypes.

Argument marshalling only: every step of layout, dispatch and combine runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. There is no fallback: if libmoe.so is missing, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_ALIGNMENT = -2
MOE_ERR_SHAPE = -3
MOE_ERR_CAPACITY = -4
MOE_ERR_CUDA = -5
MOE_ERR_DEVICE_IDS = -6
MOE_ERR_TOO_LARGE = -7
MOE_ERR_TIMEOUT = -8
MOE_NOALLOC_SCRATCH_BYTES = 2 << 20

MOE_PAYLOAD_BF16 = 0
MOE_PAYLOAD_FP8_E4M3_B128 = 1
MOE_PAYLOAD_NVFP4_B16 = 2
MOE_PAYLOAD_RAW = 3
MOE_PAYLOAD_FP8_E4M3_UE8M0 = 4

MOE_COMBINE_TOPK = 0
MOE_COMBINE_RANKS = 1
MOE_COMBINE_TOPK_RANKS = 2

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_GROUP_MAX = 0
MOE_GROUP_TOP2_SUM = 1
MOE_LOGITS_F32 = 0
MOE_LOGITS_BF16 = 1

MOE_GRAD_BF16 = 0
MOE_GRAD_F32 = 1
MOE_GRAD_F32_ADD = 2

MOE_ROWS_BF16 = 0
MOE_ROWS_F32 = 1

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"` "
        "(there is no CPU fallback)")
_lib = ctypes.CDLL(LIB_PATH)

_i32, _i64, _sz, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class _Desc(ctypes.Structure):
    _fields_ = [("num_tokens", _i32), ("topk", _i32), ("num_experts", _i32), ("num_ranks", _i32),
                ("hidden", _i32), ("in_kind", _i32), ("out_kind", _i32),
                ("raw_payload_bytes", _i32), ("raw_scale_bytes", _i32)]


class _Layout(ctypes.Structure):
    _fields_ = [("record_bytes", _i32), ("off_ids", _i32), ("off_weights", _i32),
                ("off_payload", _i32), ("off_scales", _i32), ("payload_bytes", _i32),
                ("scale_bytes", _i32)]


_D = ctypes.POINTER(_Desc)
_lib.moe_strerror.restype = ctypes.c_char_p
_lib.moe_strerror.argtypes = [ctypes.c_int]
_lib.moe_record_layout.restype = ctypes.c_int
_lib.moe_record_layout.argtypes = [_D, ctypes.POINTER(_Layout)]
_lib.moe_workspace_size.restype = _sz
_lib.moe_workspace_size.argtypes = [_D]
_lib.moe_layout.restype = ctypes.c_int
_lib.moe_layout.argtypes = [_D] + [_vp] * 9 + [_sz, _vp]
_lib.moe_layout_noalloc.restype = ctypes.c_int
_lib.moe_layout_noalloc.argtypes = [_D] + [_vp] * 10
_lib.moe_layout_status.restype = ctypes.c_int
_lib.moe_layout_status.argtypes = [_vp, ctypes.POINTER(_i32), _vp]
_lib.moe_dispatch.restype = ctypes.c_int
_lib.moe_dispatch.argtypes = [_D] + [_vp] * 6 + [_sz, _vp]
_lib.moe_layout_dispatch.restype = ctypes.c_int
_lib.moe_layout_dispatch.argtypes = [_D] + [_vp] * 12 + [_sz, _vp, _sz, _vp]
_lib.moe_combine.restype = ctypes.c_int
_lib.moe_combine.argtypes = [_D, ctypes.c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
_lib.moe_combine_norm.restype = ctypes.c_int
_lib.moe_combine_norm.argtypes = [_D, ctypes.c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                  ctypes.c_float, _vp, _vp, _vp]


class _SlotDesc(ctypes.Structure):
    _fields_ = [("num_tensors", _i32), ("num_ranks", _i32), ("bytes", _i64 * 4)]


_SD = ctypes.POINTER(_SlotDesc)
_lib.moe_slot_layout.restype = ctypes.c_int
_lib.moe_slot_layout.argtypes = [_SD, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
_lib.moe_pack_slots.restype = ctypes.c_int
_lib.moe_pack_slots.argtypes = [_SD, ctypes.POINTER(_vp), _vp, _vp]
_lib.moe_unpack_slots.restype = ctypes.c_int
_lib.moe_unpack_slots.argtypes = [_SD, _vp, ctypes.POINTER(_vp), _vp]
_lib.moe_rank_layout.restype = ctypes.c_int
_lib.moe_rank_layout.argtypes = [_D, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.moe_layout_ll_dispatch.restype = ctypes.c_int
_lib.moe_layout_ll_dispatch.argtypes = [_D] + [_vp] * 10 + [_i32] + [_vp] * 5 + [_sz, _vp, _sz, _vp, _sz, _vp]
_lib.moe_layout_ll.restype = ctypes.c_int
_lib.moe_layout_ll.argtypes = [_D] + [_vp] * 8 + [_i32] + [_vp] * 5 + [_sz, _vp]
_lib.moe_layout_ranks.restype = ctypes.c_int
_lib.moe_layout_ranks.argtypes = [_D] + [_vp] * 8 + [_i32] + [_vp] * 5 + [_sz, _vp]
_lib.moe_dispatch_ranks.restype = ctypes.c_int
_lib.moe_dispatch_ranks.argtypes = [_D] + [_vp] * 6 + [_sz, _vp]
_lib.moe_combine_gather_ranks.restype = ctypes.c_int
_lib.moe_combine_gather_ranks.argtypes = [_D, _vp, _i64, _vp, _vp, _vp]
_lib.moe_ll_layout.restype = ctypes.c_int
_lib.moe_ll_layout.argtypes = [_D, _i32] + [_vp] * 8 + [_vp]
_lib.moe_dispatch_ll.restype = ctypes.c_int
_lib.moe_dispatch_ll.argtypes = [_D, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp]
_lib.moe_combine_backward.restype = ctypes.c_int
_lib.moe_combine_backward.argtypes = [_D, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]
_lib.moe_dispatch_backward.restype = ctypes.c_int
_lib.moe_dispatch_backward.argtypes = [_D, _vp, _i64, _vp, _vp, _vp]
_lib.moe_combine_gather_ranks_backward.restype = ctypes.c_int
_lib.moe_combine_gather_ranks_backward.argtypes = [_D, _vp, _vp, _vp, _i64, _vp]
_lib.moe_mask_topk_ids.restype = ctypes.c_int
_lib.moe_mask_topk_ids.argtypes = [_vp, _i32, _i32, _vp, _vp]
_lib.moe_device_status.restype = ctypes.c_int
_lib.moe_device_status.argtypes = [_vp, ctypes.c_int]
_lib.moe_set_wait_limit_ns.restype = ctypes.c_int
_lib.moe_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.moe_pack_record.restype = ctypes.c_int
_lib.moe_pack_record.argtypes = [_D, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.moe_unpack_record.restype = ctypes.c_int
_lib.moe_unpack_record.argtypes = [_D, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]


class _RouteDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("num_tokens", "num_experts", "topk", "num_groups", "topk_groups", "score",
                                          "group_score", "renormalize", "logits_kind", "logits_stride")]
    _fields_ += [("scale", ctypes.c_float)]


class _GluDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("width", _i32)]


class _ExpertDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("x_stride", _i64), ("num_experts", _i32), ("in_features", _i32),
                ("out_features", _i32)]


class _QuantDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("x_stride", _i64), ("width", _i32), ("x_kind", _i32), ("scale_stride", _i32)]


class _ExpertI8Desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("x_stride", _i64), ("x_scale_stride", _i64), ("num_experts", _i32),
                ("in_features", _i32), ("out_features", _i32)]


for _name, _desc, _args in (
        ("moe_route", _RouteDesc, [_vp] * 5), ("moe_route_backward", _RouteDesc, [_vp] * 5),
        ("moe_swiglu", _GluDesc, [_vp] * 6), ("moe_swiglu_backward", _GluDesc, [_vp] * 7),
        ("moe_expert_product", _ExpertDesc, [_vp] * 6), ("moe_expert_swiglu", _ExpertDesc, [_vp] * 8),
        ("moe_expert_product_backward_input", _ExpertDesc, [_vp] * 6),
        ("moe_expert_product_backward_weight", _ExpertDesc, [_vp] * 5 + [ctypes.c_int, _vp]),
        ("moe_quantize_rows", _QuantDesc, [_vp] * 5),
        ("moe_expert_product_i8", _ExpertI8Desc, [_vp] * 8), ("moe_expert_swiglu_i8", _ExpertI8Desc, [_vp] * 8)):
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = [ctypes.POINTER(_desc)] + _args


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {moe_strerror(code)} ({code})")
        self.code = code


@dataclass
class MoeDesc:
    """Shape and format of one call (moe_desc_t)."""
    num_tokens: int
    topk: int
    num_experts: int
    num_ranks: int
    hidden: int
    in_kind: int = MOE_PAYLOAD_BF16
    out_kind: int = MOE_PAYLOAD_BF16
    raw_payload_bytes: int = 0
    raw_scale_bytes: int = 0

    def c(self) -> _Desc:
        return _Desc(self.num_tokens, self.topk, self.num_experts, self.num_ranks, self.hidden,
                     self.in_kind, self.out_kind, self.raw_payload_bytes, self.raw_scale_bytes)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr() if t.numel() else None
    return t


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def moe_strerror(code: int) -> str:
    return _lib.moe_strerror(int(code)).decode()


def moe_record_layout(desc: MoeDesc) -> dict:
    lay = _Layout()
    _check(_lib.moe_record_layout(ctypes.byref(desc.c()), ctypes.byref(lay)), "moe_record_layout")
    return {name: getattr(lay, name) for name, _ in _Layout._fields_}


def moe_workspace_size(desc: MoeDesc) -> int:
    return int(_lib.moe_workspace_size(ctypes.byref(desc.c())))


def layout_outputs(desc: MoeDesc, device) -> dict:
    """Allocates the output tensors of moe_layout (torch device memory)."""
    n, k, e, r = desc.num_tokens, desc.topk, desc.num_experts, desc.num_ranks
    i32 = dict(dtype=torch.int32, device=device)
    return dict(
        tokens_per_expert=torch.empty(e, **i32),
        tokens_per_rank=torch.empty(r, **i32),
        is_token_in_rank=torch.empty((n, r), dtype=torch.uint8, device=device),
        expert_offset=torch.empty(e + 1, **i32),
        rank_offset=torch.empty(r + 1, **i32),
        slot_of=torch.empty((n, k), **i32),
        src_of_slot=torch.empty(n * k, **i32),
    )


def moe_layout(desc: MoeDesc, topk_idx: torch.Tensor, out: dict | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Routing layout (see include/moe.h). Returns the dict of output tensors
    (plus 'workspace')."""
    if out is None:
        out = layout_outputs(desc, topk_idx.device)
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_size(desc), 256), dtype=torch.uint8,
                                device=topk_idx.device)
    rc = _lib.moe_layout(ctypes.byref(desc.c()), _ptr(topk_idx), _ptr(out["tokens_per_expert"]),
                         _ptr(out["tokens_per_rank"]), _ptr(out["is_token_in_rank"]),
                         _ptr(out["expert_offset"]), _ptr(out["rank_offset"]),
                         _ptr(out["slot_of"]), _ptr(out.get("src_of_slot")), _ptr(workspace),
                         workspace.numel(), _stream(stream))
    _check(rc, "moe_layout")
    out["workspace"] = workspace
    return out


def moe_layout_noalloc(desc: MoeDesc, topk_idx: torch.Tensor, out: dict | None = None,
                       status: torch.Tensor | None = None, stream=None) -> dict:
    """Routing layout without a workspace, for callers that cannot provide
    device scratch: the library uses its own fixed 2 MiB device array instead
    (see include/moe.h for the size limit and the rule that calls overlapping
    on the GPU race). `status` (int32 [1] on the device) receives this call's
    status word."""
    if out is None:
        out = layout_outputs(desc, topk_idx.device)
    rc = _lib.moe_layout_noalloc(ctypes.byref(desc.c()), _ptr(topk_idx),
                                 _ptr(out["tokens_per_expert"]), _ptr(out["tokens_per_rank"]),
                                 _ptr(out["is_token_in_rank"]), _ptr(out["expert_offset"]),
                                 _ptr(out["rank_offset"]), _ptr(out["slot_of"]),
                                 _ptr(out.get("src_of_slot")), _ptr(status), _stream(stream))
    _check(rc, "moe_layout_noalloc")
    return out


def moe_device_status(clear: bool = True) -> int:
    """Status of the kernels with bounded waits on this device since the last
    clearing call: MOE_OK or MOE_ERR_TIMEOUT (synchronises the device)."""
    v = _i32(0)
    _check(_lib.moe_device_status(ctypes.byref(v), 1 if clear else 0), "moe_device_status")
    return v.value


def moe_set_wait_limit_ns(ns: int) -> None:
    """Budget of the bounded waits for later launches (0 = the default one
    second; a test hook, see include/moe.h)."""
    _check(_lib.moe_set_wait_limit_ns(int(ns)), "moe_set_wait_limit_ns")


def moe_layout_status(workspace: torch.Tensor, stream=None) -> int:
    """Status word of the last moe_layout on this workspace (synchronises)."""
    v = _i32(0)
    _check(_lib.moe_layout_status(_ptr(workspace), ctypes.byref(v), _stream(stream)),
           "moe_layout_status")
    return v.value


def moe_dispatch(desc: MoeDesc, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                 hidden: torch.Tensor, scales: torch.Tensor | None, slot_of: torch.Tensor,
                 records: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Permute and pack: writes one record per routed pair into `records`
    (uint8 [N*k, record_bytes] when allocated here)."""
    lay = moe_record_layout(desc)
    if records is None:
        records = torch.empty((desc.num_tokens * desc.topk, lay["record_bytes"]),
                              dtype=torch.uint8, device=topk_idx.device)
    nbytes = records.numel() * records.element_size()
    rc = _lib.moe_dispatch(ctypes.byref(desc.c()), _ptr(topk_idx), _ptr(topk_weights),
                           _ptr(hidden), _ptr(scales), _ptr(slot_of), _ptr(records), nbytes,
                           _stream(stream))
    _check(rc, "moe_dispatch")
    return records


def moe_combine(desc: MoeDesc, mode: int, expert_out: torch.Tensor,
                topk_idx: torch.Tensor | None, topk_weights: torch.Tensor | None,
                slot_of: torch.Tensor | None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Combine (see include/moe.h): returns bf16 [N, H]."""
    if out is None:
        out = torch.empty((desc.num_tokens, desc.hidden), dtype=torch.bfloat16,
                          device=expert_out.device)
    rows = expert_out.numel() // max(desc.hidden, 1)
    rc = _lib.moe_combine(ctypes.byref(desc.c()), int(mode), _ptr(expert_out), rows,
                          _ptr(topk_idx), _ptr(topk_weights), _ptr(slot_of), _ptr(out),
                          _stream(stream))
    _check(rc, "moe_combine")
    return out


def moe_combine_norm(desc: MoeDesc, mode: int, expert_out: torch.Tensor,
                     topk_idx: torch.Tensor | None, topk_weights: torch.Tensor | None,
                     slot_of: torch.Tensor | None, residual_in: torch.Tensor,
                     gamma: torch.Tensor, eps: float, normed_out: torch.Tensor | None = None,
                     residual_out: torch.Tensor | None = None, stream=None):
    """Combine fused with residual add and RMSNorm (see include/moe.h).
    Returns (normed_out, residual_out), both bf16 [N, H]."""
    shape = (desc.num_tokens, desc.hidden)
    if normed_out is None:
        normed_out = torch.empty(shape, dtype=torch.bfloat16, device=expert_out.device)
    if residual_out is None:
        residual_out = torch.empty(shape, dtype=torch.bfloat16, device=expert_out.device)
    rows = expert_out.numel() // max(desc.hidden, 1)
    rc = _lib.moe_combine_norm(ctypes.byref(desc.c()), int(mode), _ptr(expert_out), rows,
                               _ptr(topk_idx), _ptr(topk_weights), _ptr(slot_of),
                               _ptr(residual_in), _ptr(gamma), float(eps), _ptr(normed_out),
                               _ptr(residual_out), _stream(stream))
    _check(rc, "moe_combine_norm")
    return normed_out, residual_out


def moe_rank_layout(desc: MoeDesc, lay: dict, expert_alignment: int = 1, out: dict | None = None,
                    stream=None) -> dict:
    """Per-rank receive layout from moe_layout's outputs (see include/moe.h)."""
    n, r, e = desc.num_tokens, desc.num_ranks, desc.num_experts
    dev = lay["tokens_per_rank"].device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = dict(send_head=torch.empty((n, r), **i32), recv_src_idx=torch.empty(n * r, **i32),
                   recv_offset=torch.empty(r + 1, **i32),
                   recv_tokens_per_expert=torch.empty(e, **i32))
    rc = _lib.moe_rank_layout(ctypes.byref(desc.c()), _ptr(lay["is_token_in_rank"]),
                              _ptr(lay["tokens_per_rank"]), _ptr(lay["tokens_per_expert"]),
                              int(expert_alignment), _ptr(out["send_head"]),
                              _ptr(out.get("recv_src_idx")), _ptr(out["recv_offset"]),
                              _ptr(out["recv_tokens_per_expert"]), _stream(stream))
    _check(rc, "moe_rank_layout")
    return out


def rank_layout_outputs(desc: MoeDesc, device) -> dict:
    """Fresh receive-layout output tensors of one call (int32, on device)."""
    n, r, e = desc.num_tokens, desc.num_ranks, desc.num_experts
    i32 = dict(dtype=torch.int32, device=device)
    return dict(send_head=torch.empty((n, r), **i32), recv_src_idx=torch.empty(n * r, **i32),
                recv_offset=torch.empty(r + 1, **i32), recv_tokens_per_expert=torch.empty(e, **i32))


def moe_layout_ranks(desc: MoeDesc, topk_idx: torch.Tensor, expert_alignment: int = 1,
                     out: dict | None = None, rank_out: dict | None = None, workspace=None,
                     stream=None) -> tuple[dict, dict]:
    """moe_layout and moe_rank_layout in one call (see include/moe.h).
    Returns (layout outputs with the workspace, receive-layout outputs)."""
    if out is None:
        out = layout_outputs(desc, topk_idx.device)
    if rank_out is None:
        rank_out = rank_layout_outputs(desc, topk_idx.device)
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_size(desc), 256), dtype=torch.uint8, device=topk_idx.device)
    prepare_layout_ranks(desc, topk_idx, expert_alignment, out, rank_out, workspace, stream)()
    out["workspace"] = workspace
    return out, rank_out


def prepare_layout_ranks(desc: MoeDesc, topk_idx, expert_alignment: int, out: dict, rank_out: dict,
                         workspace, stream=None) -> Prepared:
    d = desc.c()
    args = (ctypes.byref(d),
            *_vps(topk_idx, out["tokens_per_expert"], out["tokens_per_rank"], out["is_token_in_rank"],
                  out["expert_offset"], out["rank_offset"], out["slot_of"], out.get("src_of_slot")),
            ctypes.c_int32(expert_alignment),
            *_vps(rank_out["send_head"], rank_out.get("recv_src_idx"), rank_out["recv_offset"],
                  rank_out["recv_tokens_per_expert"], workspace),
            ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_layout_ranks", args, (d, topk_idx, out, rank_out, workspace))


def moe_dispatch_ranks(desc: MoeDesc, topk_idx, topk_weights, hidden, scales, send_head,
                       records=None, stream=None) -> torch.Tensor:
    """One record per (token, rank) at send_head; records uint8 [N*R, record_bytes]
    when allocated here."""
    lay = moe_record_layout(desc)
    if records is None:
        records = torch.empty((desc.num_tokens * desc.num_ranks, lay["record_bytes"]),
                              dtype=torch.uint8, device=topk_idx.device)
    rc = _lib.moe_dispatch_ranks(ctypes.byref(desc.c()), _ptr(topk_idx), _ptr(topk_weights),
                                 _ptr(hidden), _ptr(scales), _ptr(send_head), _ptr(records),
                                 records.numel() * records.element_size(), _stream(stream))
    _check(rc, "moe_dispatch_ranks")
    return records


def moe_combine_gather_ranks(desc: MoeDesc, recv_out: torch.Tensor, send_head: torch.Tensor,
                             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = bf16(sum over ranks of recv_out[send_head[t, r]]), bf16 [N, H]."""
    if out is None:
        out = torch.empty((desc.num_tokens, desc.hidden), dtype=torch.bfloat16,
                          device=recv_out.device)
    rows = recv_out.numel() // max(desc.hidden, 1)
    rc = _lib.moe_combine_gather_ranks(ctypes.byref(desc.c()), _ptr(recv_out), rows,
                                       _ptr(send_head), _ptr(out), _stream(stream))
    _check(rc, "moe_combine_gather_ranks")
    return out


def moe_combine_backward(desc: MoeDesc, grad_out, topk_weights, slot_of, expert_out=None,
                         rows: int | None = None, grad_expert_out=None, grad_weights=None,
                         stream=None):
    """Backward of the top-k weighted combine (see include/moe.h). Returns
    (grad_expert_out bf16 [rows, H], grad_weights fp32 [N, k] or None)."""
    h = desc.hidden
    if rows is None:
        rows = expert_out.numel() // h if expert_out is not None else grad_expert_out.numel() // h
    dev = grad_out.device
    if grad_expert_out is None:
        grad_expert_out = torch.zeros((rows, h), dtype=torch.bfloat16, device=dev)
    if expert_out is not None and grad_weights is None:
        grad_weights = torch.empty((desc.num_tokens, desc.topk), dtype=torch.float32, device=dev)
    rc = _lib.moe_combine_backward(ctypes.byref(desc.c()), _ptr(grad_out), _ptr(topk_weights),
                                   _ptr(slot_of), _ptr(expert_out), int(rows), _ptr(grad_expert_out),
                                   _ptr(grad_weights) if expert_out is not None else None,
                                   _stream(stream))
    _check(rc, "moe_combine_backward")
    return grad_expert_out, grad_weights if expert_out is not None else None


def moe_dispatch_backward(desc: MoeDesc, grad_in, slot_of, grad_hidden=None, stream=None):
    """Backward of dispatch: grad_hidden[t] = bf16(sum_j grad_in[slot_of[t, j]])."""
    if grad_hidden is None:
        grad_hidden = torch.empty((desc.num_tokens, desc.hidden), dtype=torch.bfloat16,
                                  device=grad_in.device)
    rows = grad_in.numel() // max(desc.hidden, 1)
    rc = _lib.moe_dispatch_backward(ctypes.byref(desc.c()), _ptr(grad_in), rows, _ptr(slot_of),
                                    _ptr(grad_hidden), _stream(stream))
    _check(rc, "moe_dispatch_backward")
    return grad_hidden


def moe_combine_gather_ranks_backward(desc: MoeDesc, grad_out, send_head, grad_recv, stream=None):
    """grad_recv[send_head[t, r]] = grad_out[t] for every rank row the token read."""
    rows = grad_recv.numel() // max(desc.hidden, 1)
    rc = _lib.moe_combine_gather_ranks_backward(ctypes.byref(desc.c()), _ptr(grad_out),
                                                _ptr(send_head), _ptr(grad_recv), rows,
                                                _stream(stream))
    _check(rc, "moe_combine_gather_ranks_backward")
    return grad_recv


def moe_ll_layout(desc: MoeDesc, max_tokens_per_rank: int, topk_idx, lay: dict,
                  out: dict | None = None, stream=None) -> dict:
    """Fixed-capacity, expert-major receive layout (see include/moe.h)."""
    n, k, e, r = desc.num_tokens, desc.topk, desc.num_experts, desc.num_ranks
    cap = r * max_tokens_per_rank
    dev = topk_idx.device
    if out is None:
        out = dict(ll_slot_of=torch.empty((n, k), dtype=torch.int32, device=dev),
                   src_info=torch.empty((e, cap), dtype=torch.int32, device=dev),
                   layout_range=torch.empty((e, r), dtype=torch.int64, device=dev),
                   recv_count=torch.empty(e, dtype=torch.int32, device=dev))
    rc = _lib.moe_ll_layout(ctypes.byref(desc.c()), int(max_tokens_per_rank), _ptr(topk_idx),
                            _ptr(lay["slot_of"]), _ptr(lay["expert_offset"]),
                            _ptr(lay["src_of_slot"]), _ptr(out["ll_slot_of"]),
                            _ptr(out["src_info"]), _ptr(out["layout_range"]),
                            _ptr(out["recv_count"]), _stream(stream))
    _check(rc, "moe_ll_layout")
    out["capacity"] = cap
    return out


def ll_layout_outputs(desc: MoeDesc, max_tokens_per_rank: int, device) -> dict:
    """Fresh fixed-capacity layout output tensors of one call (on device)."""
    n, k, e, r = desc.num_tokens, desc.topk, desc.num_experts, desc.num_ranks
    cap = r * max_tokens_per_rank
    return dict(ll_slot_of=torch.empty((n, k), dtype=torch.int32, device=device),
                src_info=torch.empty((e, cap), dtype=torch.int32, device=device),
                layout_range=torch.empty((e, r), dtype=torch.int64, device=device),
                recv_count=torch.empty(e, dtype=torch.int32, device=device), capacity=cap)


def moe_layout_ll(desc: MoeDesc, max_tokens_per_rank: int, topk_idx: torch.Tensor, out: dict | None = None,
                  ll_out: dict | None = None, workspace=None, stream=None) -> tuple[dict, dict]:
    """moe_layout and moe_ll_layout in one call (see include/moe.h).
    Returns (layout outputs with the workspace, fixed-capacity outputs)."""
    if out is None:
        out = layout_outputs(desc, topk_idx.device)
    if ll_out is None:
        ll_out = ll_layout_outputs(desc, max_tokens_per_rank, topk_idx.device)
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_size(desc), 256), dtype=torch.uint8, device=topk_idx.device)
    prepare_layout_ll(desc, max_tokens_per_rank, topk_idx, out, ll_out, workspace, stream)()
    out["workspace"] = workspace
    return out, ll_out


def prepare_layout_ll(desc: MoeDesc, max_tokens_per_rank: int, topk_idx, out: dict, ll_out: dict, workspace,
                      stream=None) -> Prepared:
    d = desc.c()
    args = (ctypes.byref(d),
            *_vps(topk_idx, out["tokens_per_expert"], out["tokens_per_rank"], out["is_token_in_rank"],
                  out["expert_offset"], out["rank_offset"], out["slot_of"], out.get("src_of_slot")),
            ctypes.c_int32(max_tokens_per_rank),
            *_vps(ll_out["ll_slot_of"], ll_out["src_info"], ll_out["layout_range"], ll_out["recv_count"],
                  workspace),
            ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_layout_ll", args, (d, topk_idx, out, ll_out, workspace))


def moe_dispatch_ll(desc: MoeDesc, hidden, scales, ll_slot_of, capacity: int,
                    x_out=None, scales_out=None, stream=None):
    """Payload and scales into [E * capacity, ...] buffers; returns (x_out, scales_out)."""
    lay = moe_record_layout(desc)
    rows = desc.num_experts * capacity
    dev = hidden.device
    if x_out is None:
        x_out = torch.empty((rows, lay["payload_bytes"]), dtype=torch.uint8, device=dev)
    if scales_out is None and lay["scale_bytes"]:
        scale_row = (lay["scale_bytes"] + 15) // 16 * 16
        scales_out = torch.empty((rows, scale_row), dtype=torch.uint8, device=dev)
    sb = scales_out.numel() * scales_out.element_size() if scales_out is not None else 0
    rc = _lib.moe_dispatch_ll(ctypes.byref(desc.c()), _ptr(hidden), _ptr(scales), _ptr(ll_slot_of),
                              _ptr(x_out), x_out.numel() * x_out.element_size(), _ptr(scales_out),
                              sb, _stream(stream))
    _check(rc, "moe_dispatch_ll")
    return x_out, scales_out


def _slot_desc(num_ranks: int, sizes) -> _SlotDesc:
    d = _SlotDesc()
    d.num_tensors = len(sizes)
    d.num_ranks = num_ranks
    for i, b in enumerate(sizes):
        d.bytes[i] = int(b)
    return d


def moe_slot_layout(num_ranks: int, bytes_per_rank) -> tuple[list[int], int]:
    """Offsets of the tensors in a rank slot and the slot size (host only)."""
    d = _slot_desc(num_ranks, bytes_per_rank)
    off = (_i64 * 4)()
    sb = _i64(0)
    _check(_lib.moe_slot_layout(ctypes.byref(d), off, ctypes.byref(sb)), "moe_slot_layout")
    return [off[i] for i in range(len(bytes_per_rank))], sb.value


def moe_pack_slots(tensors: list, num_ranks: int, slots: torch.Tensor | None = None, stream=None):
    """Packs tensors (each rank-major, numel divisible by num_ranks) into
    slots uint8 [R, slot_bytes]."""
    sizes = [t.numel() * t.element_size() // num_ranks for t in tensors]
    _, sb = moe_slot_layout(num_ranks, sizes)
    if slots is None:
        slots = torch.empty((num_ranks, sb), dtype=torch.uint8, device=tensors[0].device)
    d = _slot_desc(num_ranks, sizes)
    arr = (_vp * 4)(*[_ptr(t) for t in tensors])
    _check(_lib.moe_pack_slots(ctypes.byref(d), arr, _ptr(slots), _stream(stream)), "moe_pack_slots")
    return slots


def moe_unpack_slots(slots: torch.Tensor, outputs: list, num_ranks: int, stream=None):
    """Fills outputs (rank-major) from slots [R, slot_bytes]."""
    sizes = [t.numel() * t.element_size() // num_ranks for t in outputs]
    d = _slot_desc(num_ranks, sizes)
    arr = (_vp * 4)(*[_ptr(t) for t in outputs])
    _check(_lib.moe_unpack_slots(ctypes.byref(d), _ptr(slots), arr, _stream(stream)),
           "moe_unpack_slots")
    return outputs


def moe_mask_topk_ids(topk_idx: torch.Tensor, num_actual_tokens: torch.Tensor, stream=None):
    """Sets ids of tokens at or past the device scalar num_actual_tokens to -1."""
    n, k = topk_idx.shape
    _check(_lib.moe_mask_topk_ids(_ptr(topk_idx), n, k, _ptr(num_actual_tokens), _stream(stream)),
           "moe_mask_topk_ids")
    return topk_idx


def moe_pack_record(desc: MoeDesc, src_token: int, slot_j: int, expert: int, ids_row, w_row,
                    payload_row, scales_row):
    """Host-only: builds one record (numpy uint8) from host numpy rows."""
    import numpy as np
    lay = moe_record_layout(desc)
    rec = np.zeros(lay["record_bytes"], dtype=np.uint8)
    arrs = [np.ascontiguousarray(a) if a is not None else None
            for a in (ids_row, w_row, payload_row, scales_row)]
    p = [a.ctypes.data if a is not None else None for a in arrs]
    _check(_lib.moe_pack_record(ctypes.byref(desc.c()), src_token, slot_j, expert, p[0], p[1],
                                p[2], p[3], rec.ctypes.data), "moe_pack_record")
    return rec


def moe_unpack_record(desc: MoeDesc, record):
    """Host-only: splits one record (numpy uint8) into its fields."""
    import numpy as np
    lay = moe_record_layout(desc)
    rec = np.ascontiguousarray(record, dtype=np.uint8)
    t, j, e = _i32(), _i32(), _i32()
    ids = np.zeros(desc.topk, np.int32)
    w = np.zeros(desc.topk, np.float32)
    pay = np.zeros(lay["payload_bytes"], np.uint8)
    sc = np.zeros(lay["scale_bytes"], np.uint8)
    _check(_lib.moe_unpack_record(ctypes.byref(desc.c()), rec.ctypes.data, ctypes.byref(t),
                                  ctypes.byref(j), ctypes.byref(e), ids.ctypes.data,
                                  w.ctypes.data, pay.ctypes.data,
                                  sc.ctypes.data if sc.size else None),
           "moe_unpack_record")
    return dict(src_token=t.value, slot_j=j.value, expert=e.value, ids=ids, weights=w,
                payload=pay, scales=sc)


class Prepared:
    """One libmoe call with its arguments marshalled once, for repeated
    launches on the same buffers and stream (argument marshalling only; each
    call of the object enqueues the library's kernels again)."""

    def __init__(self, name: str, args: tuple, keep: tuple):
        # a function object of its own, without argument types: the arguments
        # are ctypes values already, and converting them again takes 0.2 us a call
        self._fn = _lib[name]
        self._name = name
        self._args = args
        self._keep = keep  # ctypes structs and tensors the arguments point into

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != MOE_OK:
            raise MoeError(rc, self._name)


def _vps(*ts):
    return tuple(ctypes.c_void_p(_ptr(t)) for t in ts)


def prepare_layout(desc: MoeDesc, topk_idx, out: dict, workspace, stream=None) -> Prepared:
    d = desc.c()
    ptrs = _vps(topk_idx, out["tokens_per_expert"], out["tokens_per_rank"],
                out["is_token_in_rank"], out["expert_offset"], out["rank_offset"], out["slot_of"],
                out.get("src_of_slot"), workspace)
    args = (ctypes.byref(d), *ptrs, ctypes.c_size_t(workspace.numel()),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_layout", args, (d, topk_idx, out, workspace))


def moe_layout_dispatch(desc: MoeDesc, topk_idx, topk_weights, hidden, scales, out: dict | None = None,
                        workspace=None, records=None, stream=None):
    """moe_layout then moe_dispatch in one call (see include/moe.h); the
    dispatch overlaps the layout. Returns (layout outputs dict, records)."""
    dev = topk_idx.device
    if out is None:
        out = layout_outputs(desc, dev)
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_size(desc), 256), dtype=torch.uint8, device=dev)
    if records is None:
        rb = moe_record_layout(desc)["record_bytes"]
        records = torch.empty((max(desc.num_tokens * desc.topk, 1), rb), dtype=torch.uint8, device=dev)
    prepare_layout_dispatch(desc, topk_idx, topk_weights, hidden, scales, out, workspace, records,
                            stream)()
    out["workspace"] = workspace
    return out, records


def prepare_layout_dispatch(desc: MoeDesc, topk_idx, topk_weights, hidden, scales, out: dict,
                            workspace, records, stream=None) -> Prepared:
    d = desc.c()
    ptrs = _vps(topk_idx, topk_weights, hidden, scales, out["tokens_per_expert"],
                out["tokens_per_rank"], out["is_token_in_rank"], out["expert_offset"],
                out["rank_offset"], out["slot_of"], out.get("src_of_slot"), workspace)
    args = (ctypes.byref(d), *ptrs, ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(_ptr(records)),
            ctypes.c_size_t(records.numel() * records.element_size()), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_layout_dispatch", args, (d, topk_idx, topk_weights, hidden, scales, out,
                                                  workspace, records))


def prepare_dispatch(desc: MoeDesc, topk_idx, topk_weights, hidden, scales, slot_of, records,
                     stream=None) -> Prepared:
    d = desc.c()
    ptrs = _vps(topk_idx, topk_weights, hidden, scales, slot_of, records)
    args = (ctypes.byref(d), *ptrs, ctypes.c_size_t(records.numel() * records.element_size()),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_dispatch", args, (d, topk_idx, topk_weights, hidden, scales, slot_of,
                                           records))


def prepare_ll_layout(desc: MoeDesc, max_tokens_per_rank: int, topk_idx, lay: dict, out: dict,
                      stream=None) -> Prepared:
    d = desc.c()
    ptrs = _vps(topk_idx, lay["slot_of"], lay["expert_offset"], lay["src_of_slot"],
                out["ll_slot_of"], out["src_info"], out["layout_range"], out["recv_count"])
    args = (ctypes.byref(d), ctypes.c_int32(max_tokens_per_rank), *ptrs,
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_ll_layout", args, (d, topk_idx, lay, out))


def prepare_dispatch_ll(desc: MoeDesc, hidden, scales, ll_slot_of, x_out, scales_out,
                        stream=None) -> Prepared:
    d = desc.c()
    sb = scales_out.numel() * scales_out.element_size() if scales_out is not None else 0
    args = (ctypes.byref(d), *_vps(hidden, scales, ll_slot_of, x_out),
            ctypes.c_size_t(x_out.numel() * x_out.element_size()), ctypes.c_void_p(_ptr(scales_out)),
            ctypes.c_size_t(sb), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_dispatch_ll", args, (d, hidden, scales, ll_slot_of, x_out, scales_out))


def prepare_rank_layout(desc: MoeDesc, lay: dict, expert_alignment: int, out: dict,
                        stream=None) -> Prepared:
    d = desc.c()
    args = (ctypes.byref(d), *_vps(lay["is_token_in_rank"], lay["tokens_per_rank"],
                                   lay["tokens_per_expert"]),
            ctypes.c_int32(expert_alignment),
            *_vps(out["send_head"], out.get("recv_src_idx"), out["recv_offset"],
                  out["recv_tokens_per_expert"]),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_rank_layout", args, (d, lay, out))


def prepare_dispatch_ranks(desc: MoeDesc, topk_idx, topk_weights, hidden, scales, send_head,
                           records, stream=None) -> Prepared:
    d = desc.c()
    args = (ctypes.byref(d), *_vps(topk_idx, topk_weights, hidden, scales, send_head, records),
            ctypes.c_size_t(records.numel() * records.element_size()),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_dispatch_ranks", args, (d, topk_idx, topk_weights, hidden, scales,
                                                 send_head, records))


def prepare_layout_ll_dispatch(desc: MoeDesc, max_tokens_per_rank: int, topk_idx, hidden, scales, out: dict,
                               ll_out: dict, workspace, x_out, scales_out, stream=None) -> Prepared:
    """moe_layout_ll and moe_dispatch_ll in one call (see include/moe.h)."""
    d = desc.c()
    sb = scales_out.numel() * scales_out.element_size() if scales_out is not None else 0
    args = (ctypes.byref(d),
            *_vps(topk_idx, hidden, scales, out["tokens_per_expert"], out["tokens_per_rank"],
                  out["is_token_in_rank"], out["expert_offset"], out["rank_offset"], out["slot_of"],
                  out.get("src_of_slot")),
            ctypes.c_int32(max_tokens_per_rank),
            *_vps(ll_out["ll_slot_of"], ll_out["src_info"], ll_out["layout_range"], ll_out["recv_count"],
                  workspace),
            ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(_ptr(x_out)),
            ctypes.c_size_t(x_out.numel() * x_out.element_size()), ctypes.c_void_p(_ptr(scales_out)),
            ctypes.c_size_t(sb), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_layout_ll_dispatch", args, (d, topk_idx, hidden, scales, out, ll_out, workspace,
                                                     x_out, scales_out))


def prepare_combine_gather_ranks(desc: MoeDesc, recv_out, send_head, out, stream=None) -> Prepared:
    d = desc.c()
    rows = recv_out.numel() // max(desc.hidden, 1)
    args = (ctypes.byref(d), ctypes.c_void_p(_ptr(recv_out)), ctypes.c_int64(rows),
            *_vps(send_head, out), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_combine_gather_ranks", args, (d, recv_out, send_head, out))


def prepare_combine(desc: MoeDesc, mode: int, expert_out, topk_idx, topk_weights, slot_of, out,
                    stream=None) -> Prepared:
    d = desc.c()
    rows = expert_out.numel() // max(desc.hidden, 1)
    ptrs = _vps(topk_idx, topk_weights, slot_of, out)
    args = (ctypes.byref(d), ctypes.c_int(mode), ctypes.c_void_p(_ptr(expert_out)),
            ctypes.c_int64(rows), *ptrs, ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_combine", args, (d, expert_out, topk_idx, topk_weights, slot_of, out))


def prepare_combine_backward(desc: MoeDesc, grad_out, topk_weights, slot_of, expert_out, rows: int,
                             grad_expert_out, grad_weights, stream=None) -> Prepared:
    d = desc.c()
    args = (ctypes.byref(d), *_vps(grad_out, topk_weights, slot_of, expert_out),
            ctypes.c_int64(rows), *_vps(grad_expert_out, grad_weights),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_combine_backward", args, (d, grad_out, topk_weights, slot_of, expert_out,
                                                   grad_expert_out, grad_weights))


def prepare_dispatch_backward(desc: MoeDesc, grad_in, slot_of, grad_hidden, stream=None) -> Prepared:
    d = desc.c()
    rows = grad_in.numel() // max(desc.hidden, 1)
    args = (ctypes.byref(d), ctypes.c_void_p(_ptr(grad_in)), ctypes.c_int64(rows),
            *_vps(slot_of, grad_hidden), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_dispatch_backward", args, (d, grad_in, slot_of, grad_hidden))


def prepare_combine_norm(desc: MoeDesc, mode: int, expert_out, topk_idx, topk_weights, slot_of,
                         residual_in, gamma, eps: float, normed_out, residual_out,
                         stream=None) -> Prepared:
    d = desc.c()
    rows = expert_out.numel() // max(desc.hidden, 1)
    args = (ctypes.byref(d), ctypes.c_int(mode), ctypes.c_void_p(_ptr(expert_out)),
            ctypes.c_int64(rows), *_vps(topk_idx, topk_weights, slot_of, residual_in, gamma),
            ctypes.c_float(eps), *_vps(normed_out, residual_out), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_combine_norm", args, (d, expert_out, topk_idx, topk_weights, slot_of,
                                               residual_in, gamma, normed_out, residual_out))


# ---- router, gated activation and experts' products ---------------------------
# The descriptors hold sizes and kinds; what a call reads and writes is checked
# against them here (type, device, density and room), since the library sees
# pointers only.

@dataclass
class MoeRouteDesc:
    """Shape and rule of one router call (moe_route_desc_t)."""
    num_tokens: int
    num_experts: int
    topk: int
    score: int = MOE_SCORE_SOFTMAX
    num_groups: int = 1
    topk_groups: int = 1
    group_score: int = MOE_GROUP_TOP2_SUM
    renormalize: bool = True
    scale: float = 1.0
    logits_kind: int = MOE_LOGITS_F32
    logits_stride: int = 0

    def c(self) -> _RouteDesc:
        return _RouteDesc(self.num_tokens, self.num_experts, self.topk, self.num_groups, self.topk_groups, self.score,
                          self.group_score, int(self.renormalize), self.logits_kind, self.logits_stride, self.scale)

    @property
    def logits_dtype(self):
        return torch.bfloat16 if self.logits_kind == MOE_LOGITS_BF16 else torch.float32


@dataclass
class MoeGluDesc:
    """Rows and width F of one gated activation (moe_glu_desc_t)."""
    rows: int
    width: int

    def c(self) -> _GluDesc:
        return _GluDesc(self.rows, self.width)

    @property
    def groups(self) -> int:
        return -(-self.width // 128)


@dataclass
class MoeExpertDesc:
    """Shape of one call of the experts' products (moe_expert_desc_t)."""
    num_experts: int
    rows: int
    in_features: int
    out_features: int
    x_stride: int = 0

    def c(self) -> _ExpertDesc:
        return _ExpertDesc(self.rows, self.x_stride, self.num_experts, self.in_features, self.out_features)


@dataclass
class MoeQuantDesc:
    """Shape and format of one moe_quantize_rows call (moe_quant_desc_t)."""
    rows: int
    width: int
    x_kind: int = MOE_ROWS_BF16
    x_stride: int = 0
    scale_stride: int = 1

    def c(self) -> _QuantDesc:
        return _QuantDesc(self.rows, self.x_stride, self.width, self.x_kind, self.scale_stride)

    @property
    def x_dtype(self):
        return torch.float32 if self.x_kind == MOE_ROWS_F32 else torch.bfloat16


@dataclass
class MoeExpertI8Desc:
    """Shape of one call of the experts' 8-bit products (moe_expert_i8_desc_t)."""
    num_experts: int
    rows: int
    in_features: int
    out_features: int
    x_stride: int = 0
    x_scale_stride: int = 0

    def c(self) -> _ExpertI8Desc:
        return _ExpertI8Desc(self.rows, self.x_stride, self.x_scale_stride, self.num_experts, self.in_features,
                             self.out_features)


def _fresh(shape, dtype, device, stream):
    """An output of a call on `stream`, out of that stream's memory: a block of the current stream's may still be
    written by what is queued there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _want(what: str, t, dtype, numel: int, optional: bool = False):
    """t is a dense CUDA tensor of dtype with at least numel elements."""
    if t is None:
        if optional or numel <= 0:
            return
        raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: missing")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: a dense CUDA tensor of {dtype} is wanted")
    if t.numel() < numel:
        raise MoeError(MOE_ERR_CAPACITY, f"{what}: {t.numel()} elements, {numel} needed")


def _want_rows(what: str, t, dtype, rows: int, width: int, stride: int):
    """t is a CUDA tensor of dtype that holds `rows` rows of `width` elements, `stride` apart; dimensions before the
    last count as rows if they lie evenly."""
    if t is None:
        if rows <= 0:
            return
        raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: missing")
    if t.dtype != dtype or not t.is_cuda:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: a CUDA tensor of {dtype} is wanted")
    if rows <= 0:
        return
    if t.numel() == 0:
        raise MoeError(MOE_ERR_CAPACITY, f"{what}: empty, {rows} rows of {width} needed")
    dims = [(n, d) for n, d in zip(t.shape, t.stride()) if n > 1]
    block = 1  # a dense run of elements, as many dimensions from the last as make a row
    while dims and block < width and dims[-1][1] == block:
        block *= dims.pop()[0]
    have, apart = block, stride
    for n, d in reversed(dims):
        if d != apart or block < width:
            raise MoeError(MOE_ERR_INVALID_ARG,
                           f"{what}: dense rows of {width}, {stride} apart, are wanted, not {list(t.shape)} with strides {list(t.stride())}")
        have += (n - 1) * d
        apart *= n
    if have < (rows - 1) * stride + width:
        raise MoeError(MOE_ERR_CAPACITY, f"{what}: {have} elements, {(rows - 1) * stride + width} needed")


def _want_logits(desc: MoeRouteDesc, logits):
    _want_rows("logits", logits, desc.logits_dtype, desc.num_tokens, desc.num_experts,
               desc.logits_stride or desc.num_experts)


def prepare_route(desc: MoeRouteDesc, logits, bias, topk_idx, topk_weights, stream=None) -> Prepared:
    n, k = desc.num_tokens, desc.topk
    _want_logits(desc, logits)
    _want("bias", bias, torch.float32, desc.num_experts, optional=True)
    _want("topk_idx", topk_idx, torch.int32, n * k)
    _want("topk_weights", topk_weights, torch.float32, n * k)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(logits, bias, topk_idx, topk_weights), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_route", args, (d, logits, bias, topk_idx, topk_weights))


def moe_route(desc: MoeRouteDesc, logits, bias=None, topk_idx=None, topk_weights=None, stream=None):
    """The experts of each token and their weights (see include/moe.h).
    Returns (topk_idx int32 [N, k], topk_weights fp32 [N, k])."""
    shape = (desc.num_tokens, desc.topk)
    if topk_idx is None:
        topk_idx = _fresh(shape, torch.int32, logits.device, stream)
    if topk_weights is None:
        topk_weights = _fresh(shape, torch.float32, logits.device, stream)
    prepare_route(desc, logits, bias, topk_idx, topk_weights, stream)()
    return topk_idx, topk_weights


def prepare_route_backward(desc: MoeRouteDesc, logits, topk_idx, grad_weights, grad_logits, stream=None) -> Prepared:
    n, k = desc.num_tokens, desc.topk
    _want_logits(desc, logits)
    _want("topk_idx", topk_idx, torch.int32, n * k)
    _want("grad_weights", grad_weights, torch.float32, n * k)
    _want("grad_logits", grad_logits, desc.logits_dtype, n * desc.num_experts)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(logits, topk_idx, grad_weights, grad_logits), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_route_backward", args, (d, logits, topk_idx, grad_weights, grad_logits))


def moe_route_backward(desc: MoeRouteDesc, logits, topk_idx, grad_weights, grad_logits=None, stream=None):
    """Gradient of the logits, [N, E] of their type (see include/moe.h)."""
    if grad_logits is None:
        grad_logits = _fresh((desc.num_tokens, desc.num_experts), desc.logits_dtype, logits.device, stream)
    prepare_route_backward(desc, logits, topk_idx, grad_weights, grad_logits, stream)()
    return grad_logits


def swiglu_checkpoint(desc: MoeGluDesc, device):
    """Fresh checkpoint buffers: (codes uint8 [rows, 2F], scales fp32 [rows, 2 * ceil(F/128)])."""
    return (torch.empty((desc.rows, 2 * desc.width), dtype=torch.uint8, device=device),
            torch.empty((desc.rows, 2 * desc.groups), dtype=torch.float32, device=device))


def _want_checkpoint(desc: MoeGluDesc, ckpt, ckpt_scales, optional: bool):
    _want("ckpt", ckpt, torch.uint8, desc.rows * 2 * desc.width, optional)
    _want("ckpt_scales", ckpt_scales, torch.float32, desc.rows * 2 * desc.groups, optional)


def prepare_swiglu(desc: MoeGluDesc, gate_up, act, ckpt=None, ckpt_scales=None, num_rows=None, stream=None) -> Prepared:
    _want("num_rows", num_rows, torch.int32, 1, optional=True)
    _want("gate_up", gate_up, torch.bfloat16, desc.rows * 2 * desc.width)
    _want("act", act, torch.bfloat16, desc.rows * desc.width, optional=True)
    _want_checkpoint(desc, ckpt, ckpt_scales, optional=True)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(num_rows, gate_up, act, ckpt, ckpt_scales), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_swiglu", args, (d, num_rows, gate_up, act, ckpt, ckpt_scales))


def moe_swiglu(desc: MoeGluDesc, gate_up, act=None, ckpt=None, ckpt_scales=None, num_rows=None, stream=None):
    """act = silu(gate) * up, and the checkpoint if buffers for it are given. Returns act bf16 [rows, F]."""
    if act is None:
        act = _fresh((desc.rows, desc.width), torch.bfloat16, gate_up.device, stream)
    prepare_swiglu(desc, gate_up, act, ckpt, ckpt_scales, num_rows, stream)()
    return act


def prepare_swiglu_backward(desc: MoeGluDesc, ckpt, ckpt_scales, grad_act, grad_gate_up, act=None, num_rows=None,
                            stream=None) -> Prepared:
    _want("num_rows", num_rows, torch.int32, 1, optional=True)
    _want_checkpoint(desc, ckpt, ckpt_scales, optional=False)
    _want("grad_act", grad_act, torch.bfloat16, desc.rows * desc.width)
    _want("grad_gate_up", grad_gate_up, torch.bfloat16, desc.rows * 2 * desc.width)
    _want("act", act, torch.bfloat16, desc.rows * desc.width, optional=True)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(num_rows, ckpt, ckpt_scales, grad_act, grad_gate_up, act),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_swiglu_backward", args, (d, num_rows, ckpt, ckpt_scales, grad_act, grad_gate_up, act))


def moe_swiglu_backward(desc: MoeGluDesc, ckpt, ckpt_scales, grad_act, grad_gate_up=None, act=None, num_rows=None,
                        stream=None):
    """Gradient of gate|up from the checkpoint; act (if given) receives the activation again.
    Returns grad_gate_up bf16 [rows, 2F]."""
    if grad_gate_up is None:
        grad_gate_up = _fresh((desc.rows, 2 * desc.width), torch.bfloat16, grad_act.device, stream)
    prepare_swiglu_backward(desc, ckpt, ckpt_scales, grad_act, grad_gate_up, act, num_rows, stream)()
    return grad_gate_up


def expert_row_ranges(lay: dict):
    """(row_begin, row_end) of rows in slot order, from moe_layout's outputs (views, no copy)."""
    off = lay["expert_offset"]
    return off[:-1], off[1:]


def _want_experts(desc: MoeExpertDesc, row_begin, row_end):
    _want("row_begin", row_begin, torch.int32, desc.num_experts)
    _want("row_end", row_end, torch.int32, desc.num_experts)


def prepare_expert_product(desc: MoeExpertDesc, x, row_begin, row_end, w, y, stream=None) -> Prepared:
    e, r, k, n = desc.num_experts, desc.rows, desc.in_features, desc.out_features
    _want_experts(desc, row_begin, row_end)
    _want_rows("x", x, torch.bfloat16, r, k, desc.x_stride or k)
    _want("w", w, torch.bfloat16, e * n * k)
    _want("y", y, torch.bfloat16, r * n)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(x, row_begin, row_end, w, y), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_expert_product", args, (d, x, row_begin, row_end, w, y))


def moe_expert_product(desc: MoeExpertDesc, x, row_begin, row_end, w, y=None, stream=None):
    """y[s] = w[e] x[s] for the rows of every expert (see include/moe.h). Returns y bf16 [rows, N]."""
    if y is None:
        y = _fresh((desc.rows, desc.out_features), torch.bfloat16, w.device, stream)
    prepare_expert_product(desc, x, row_begin, row_end, w, y, stream)()
    return y


def prepare_expert_swiglu(desc: MoeExpertDesc, x, row_begin, row_end, w, act, ckpt=None, ckpt_scales=None,
                          stream=None) -> Prepared:
    e, r, k, f = desc.num_experts, desc.rows, desc.in_features, desc.out_features
    _want_experts(desc, row_begin, row_end)
    _want_rows("x", x, torch.bfloat16, r, k, desc.x_stride or k)
    _want("w", w, torch.bfloat16, e * 2 * f * k)
    _want("act", act, torch.bfloat16, r * f)
    _want_checkpoint(MoeGluDesc(r, f), ckpt, ckpt_scales, optional=True)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(x, row_begin, row_end, w, act, ckpt, ckpt_scales), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_expert_swiglu", args, (d, x, row_begin, row_end, w, act, ckpt, ckpt_scales))


def moe_expert_swiglu(desc: MoeExpertDesc, x, row_begin, row_end, w, act=None, ckpt=None, ckpt_scales=None, stream=None):
    """silu(gate) * up with gate|up = w[e] x[s], w [E, 2F, K], desc.out_features = F; and the checkpoint if buffers
    for it are given (swiglu_checkpoint). Returns act bf16 [rows, F]."""
    if act is None:
        act = _fresh((desc.rows, desc.out_features), torch.bfloat16, w.device, stream)
    prepare_expert_swiglu(desc, x, row_begin, row_end, w, act, ckpt, ckpt_scales, stream)()
    return act


def prepare_expert_product_backward_input(desc: MoeExpertDesc, grad_y, row_begin, row_end, w, grad_x,
                                          stream=None) -> Prepared:
    e, r, k, n = desc.num_experts, desc.rows, desc.in_features, desc.out_features
    _want_experts(desc, row_begin, row_end)
    _want("grad_y", grad_y, torch.bfloat16, r * n)
    _want("w", w, torch.bfloat16, e * n * k)
    _want("grad_x", grad_x, torch.bfloat16, r * k)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(grad_y, row_begin, row_end, w, grad_x), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_expert_product_backward_input", args, (d, grad_y, row_begin, row_end, w, grad_x))


def moe_expert_product_backward_input(desc: MoeExpertDesc, grad_y, row_begin, row_end, w, grad_x=None, stream=None):
    """grad_x[s] = w[e]^T grad_y[s]. Returns grad_x bf16 [rows, K]."""
    if grad_x is None:
        grad_x = _fresh((desc.rows, desc.in_features), torch.bfloat16, w.device, stream)
    prepare_expert_product_backward_input(desc, grad_y, row_begin, row_end, w, grad_x, stream)()
    return grad_x


def prepare_expert_product_backward_weight(desc: MoeExpertDesc, grad_y, x, row_begin, row_end, grad_w,
                                           grad_kind: int = MOE_GRAD_BF16, stream=None) -> Prepared:
    e, r, k, n = desc.num_experts, desc.rows, desc.in_features, desc.out_features
    _want_experts(desc, row_begin, row_end)
    _want("grad_y", grad_y, torch.bfloat16, r * n)
    _want_rows("x", x, torch.bfloat16, r, k, desc.x_stride or k)
    _want("grad_w", grad_w, torch.bfloat16 if grad_kind == MOE_GRAD_BF16 else torch.float32, e * n * k)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(grad_y, x, row_begin, row_end, grad_w), ctypes.c_int(grad_kind),
            ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_expert_product_backward_weight", args, (d, grad_y, x, row_begin, row_end, grad_w))


def moe_expert_product_backward_weight(desc: MoeExpertDesc, grad_y, x, row_begin, row_end, grad_w=None,
                                       grad_kind: int = MOE_GRAD_BF16, stream=None):
    """grad_w[e] = sum of grad_y[s]^T x[s] over e's rows, written as bf16 or fp32 or added to an fp32 grad_w (written
    where none is given). Returns grad_w [E, N, K]."""
    if grad_w is None:
        # every element is written, those of experts without rows too
        if grad_kind == MOE_GRAD_F32_ADD:
            grad_kind = MOE_GRAD_F32
        grad_w = _fresh((desc.num_experts, desc.out_features, desc.in_features),
                        torch.bfloat16 if grad_kind == MOE_GRAD_BF16 else torch.float32, row_begin.device, stream)
    prepare_expert_product_backward_weight(desc, grad_y, x, row_begin, row_end, grad_w, grad_kind, stream)()
    return grad_w


def prepare_quantize_rows(desc: MoeQuantDesc, x, q, scales, num_rows=None, stream=None) -> Prepared:
    r, n = desc.rows, desc.width
    _want("num_rows", num_rows, torch.int32, 1, optional=True)
    _want_rows("x", x, desc.x_dtype, r, n, desc.x_stride or n)
    _want("q", q, torch.int8, r * n)
    _want("scales", scales, torch.float32, r * (desc.scale_stride or 1))
    d = desc.c()
    args = (ctypes.byref(d), *_vps(num_rows, x, q, scales), ctypes.c_void_p(_stream(stream)))
    return Prepared("moe_quantize_rows", args, (d, num_rows, x, q, scales))


def moe_quantize_rows(desc: MoeQuantDesc, x, q=None, scales=None, num_rows=None, stream=None):
    """Rows to 8-bit integers with a scale each (see include/moe.h).
    Returns (q int8 [rows, width], scales fp32 [rows, scale_stride])."""
    if q is None:
        q = _fresh((desc.rows, desc.width), torch.int8, x.device, stream)
    if scales is None:
        scales = _fresh((desc.rows, desc.scale_stride or 1), torch.float32, x.device, stream)
    prepare_quantize_rows(desc, x, q, scales, num_rows, stream)()
    return q, scales


def _prepare_expert_i8(name: str, desc: MoeExpertI8Desc, halves: int, x, x_scales, row_begin, row_end, w, w_scales, out,
                       stream) -> Prepared:
    e, r, k, n = desc.num_experts, desc.rows, desc.in_features, desc.out_features
    if x_scales is not None and x_scales.dim() == 2 and x_scales.shape[1]:  # as moe_quantize_rows returns them: the first of each row
        x_scales = x_scales[:, 0]
    _want("row_begin", row_begin, torch.int32, e)
    _want("row_end", row_end, torch.int32, e)
    _want_rows("x", x, torch.int8, r, k, desc.x_stride or k)
    _want_rows("x_scales", x_scales, torch.float32, r, 1, desc.x_scale_stride or 1)
    _want("w", w, torch.int8, e * halves * n * k)
    _want("w_scales", w_scales, torch.float32, e * halves * n)
    _want("act" if halves == 2 else "y", out, torch.bfloat16, r * n)
    d = desc.c()
    args = (ctypes.byref(d), *_vps(x, x_scales, row_begin, row_end, w, w_scales, out), ctypes.c_void_p(_stream(stream)))
    return Prepared(name, args, (d, x, x_scales, row_begin, row_end, w, w_scales, out))


def prepare_expert_product_i8(desc: MoeExpertI8Desc, x, x_scales, row_begin, row_end, w, w_scales, y,
                              stream=None) -> Prepared:
    return _prepare_expert_i8("moe_expert_product_i8", desc, 1, x, x_scales, row_begin, row_end, w, w_scales, y, stream)


def moe_expert_product_i8(desc: MoeExpertI8Desc, x, x_scales, row_begin, row_end, w, w_scales, y=None, stream=None):
    """y[s] = w[e] x[s] for int8 rows and weights, with their scales (see include/moe.h). Returns y bf16 [rows, N]."""
    if y is None:
        y = _fresh((desc.rows, desc.out_features), torch.bfloat16, w.device, stream)
    prepare_expert_product_i8(desc, x, x_scales, row_begin, row_end, w, w_scales, y, stream)()
    return y


def prepare_expert_swiglu_i8(desc: MoeExpertI8Desc, x, x_scales, row_begin, row_end, w, w_scales, act,
                             stream=None) -> Prepared:
    return _prepare_expert_i8("moe_expert_swiglu_i8", desc, 2, x, x_scales, row_begin, row_end, w, w_scales, act, stream)


def moe_expert_swiglu_i8(desc: MoeExpertI8Desc, x, x_scales, row_begin, row_end, w, w_scales, act=None, stream=None):
    """silu(gate) * up with gate|up = w[e] x[s] as in moe_expert_product_i8, w int8 [E, 2F, K], desc.out_features = F.
    Returns act bf16 [rows, F]."""
    if act is None:
        act = _fresh((desc.rows, desc.out_features), torch.bfloat16, w.device, stream)
    prepare_expert_swiglu_i8(desc, x, x_scales, row_begin, row_end, w, w_scales, act, stream)()
    return act


def exported_symbols() -> list[str]:
    return ["moe_strerror", "moe_record_layout", "moe_workspace_size", "moe_layout",
            "moe_layout_status", "moe_dispatch", "moe_combine", "moe_pack_record",
            "moe_unpack_record", "moe_layout_noalloc", "moe_combine_norm", "moe_slot_layout",
            "moe_pack_slots", "moe_unpack_slots", "moe_mask_topk_ids", "moe_rank_layout",
            "moe_dispatch_ranks", "moe_combine_gather_ranks", "moe_ll_layout",
            "moe_dispatch_ll", "moe_combine_backward", "moe_dispatch_backward",
            "moe_combine_gather_ranks_backward", "moe_layout_dispatch", "moe_device_status",
            "moe_layout_ranks", "moe_layout_ll", "moe_layout_ll_dispatch", "moe_set_wait_limit_ns",
            "moe_route", "moe_route_backward", "moe_swiglu", "moe_swiglu_backward", "moe_expert_product",
            "moe_expert_swiglu", "moe_expert_product_backward_input", "moe_expert_product_backward_weight",
            "moe_quantize_rows", "moe_expert_product_i8", "moe_expert_swiglu_i8"]
