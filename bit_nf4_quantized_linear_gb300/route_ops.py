"""Torch-facing wrappers of the router of ``include/nf4.h``: the experts of each token, their weights, the
tables that sort the tokens by expert, and the gradient of the logits.

As in ``ops``: PyTorch supplies device memory and the current stream, every step of the
computation runs in the library's kernels, and there is no CPU path.
"""
from __future__ import annotations

import struct
from typing import NamedTuple, Optional

import torch

from . import _lib
from .block_ops import _DTYPES, _dtype, _fn, _on, _one_device, _raw_stream, _workspace

_ROUTE = struct.Struct("@P2q2P8if4x")  # nf4_route
_SCORES = {"softmax": _lib.SCORE_SOFTMAX, "sigmoid": _lib.SCORE_SIGMOID}


class Routes(NamedTuple):
    """Where tokens go.  R = tokens * k rows; those from offsets[E] on are no pair's (tokens that are not live)."""
    experts: torch.Tensor                 # int32 [tokens, k], ascending; -1 for a token that is not live
    weights: torch.Tensor                 # fp32 [tokens, k]
    offsets: Optional[torch.Tensor]       # int32 [E + 1]: rows offsets[e] .. offsets[e + 1] - 1 belong to expert e
    row_token: Optional[torch.Tensor]     # int32 [R]: the token of each row, -1 for none
    token_rows: Optional[torch.Tensor]    # int32 [tokens, k]: the row of each route, -1 for none
    row_weight: Optional[torch.Tensor]    # fp32 [R]: the weight of each row


def _explain_route(name, logits, k, score, bias, groups, top_groups, group_top, live):
    _one_device(name, logits, bias, live)
    _dtype(name, logits)
    if logits.dim() != 2 or logits.shape[1] < 1 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"{name}: logits must be [tokens, experts] with unit column stride")
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError(f"{name}: score must be 'softmax' or 'sigmoid', got {score!r}")
    if groups < 1 or E % groups or not 1 <= top_groups <= groups or group_top not in (1, 2):
        raise ValueError(f"{name}: {E} experts do not form {groups} groups of which {top_groups} are kept by their best {group_top}")
    if not 1 <= k <= top_groups * (E // groups):
        raise ValueError(f"{name}: {k} experts of the {top_groups * (E // groups)} that are kept")
    if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (E,) or not bias.is_contiguous()):
        raise ValueError(f"{name}: bias must be a contiguous fp32 [{E}] tensor")
    raise ValueError(f"{name}: live must be a contiguous bool or uint8 [{T}] tensor")


def _route(name, logits, k, score, bias, groups, top_groups, group_top, renormalise, scale, live):
    """The packed nf4_route of checked arguments, and the tensor that the logits' pointer lies in."""
    dt, shape, stride, at = logits.dtype, logits.shape, logits.stride(), logits.get_device()
    T, E = shape if len(shape) == 2 else (0, 0)
    ok = (dt in _DTYPES and at >= 0 and E > 0 and (stride[1] == 1 or E == 1) and score in _SCORES and groups > 0 and E % groups == 0
          and 1 <= top_groups <= groups and (group_top == 1 or group_top == 2) and 1 <= k <= top_groups * (E // groups))
    bp = lp = 0
    if bias is not None:
        bp = bias.data_ptr()
        ok = ok and bias.dtype is torch.float32 and bias.shape == (E,) and bias.is_contiguous() and bias.get_device() == at
    if live is not None:
        lp = live.data_ptr()
        ok = (ok and (live.dtype is torch.bool or live.dtype is torch.uint8) and live.shape == (T,) and live.is_contiguous()
              and live.get_device() == at)
    if not ok:
        _explain_route(name, logits, k, score, bias, groups, top_groups, group_top, live)
    ld = stride[0] if T > 1 else E
    if ld < E:  # rows that share storage
        logits, ld = logits.contiguous(), E
    d = _ROUTE.pack(logits.data_ptr(), ld, T, bp, lp, E, k, _DTYPES[dt], _SCORES[score], groups, top_groups, group_top, bool(renormalise),
                    scale)
    return d, logits


def route_experts(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
                  top_groups: Optional[int] = None, group_top: int = 1, renormalise: bool = False, scale: float = 1.0,
                  live: Optional[torch.Tensor] = None, tables: bool = True) -> Routes:
    """nf4_route_fwd: the k experts of each token of logits [tokens, E] (fp32, bf16 or fp16) and their weights, by
    `score` "softmax" or "sigmoid" s: the k largest s + bias (`bias` fp32 [E] moves the choice alone), equal ones by the
    lower index (s + bias is -inf where the logit is: a hidden expert, like one whose bias is -inf), of the `top_groups` (None: all) best of `groups` runs of experts, each worth its largest (`group_top` 1) or the sum
    of its two largest (2).  The weight is scale * s, with `renormalise` over the sum of the chosen.  Tokens of
    live[t] == 0 get no experts.  With `tables`, the rows of the (token, expert) pairs sorted by expert and then by token:
    `offsets` and `row_weight` are what grouped_fwd takes, `token_rows` what moe_combine takes."""
    name = "route_experts"
    d, held = _route(name, logits, k, score, bias, groups, groups if top_groups is None else top_groups, group_top, renormalise, scale, live)
    (T, E), dev, i32, f32 = logits.shape, logits.device, torch.int32, torch.float32
    experts = torch.empty((T, k), dtype=i32, device=dev)
    weights = torch.empty((T, k), dtype=f32, device=dev)
    offsets = row_token = token_rows = row_weight = ws = None
    need = 0
    with _on(dev):
        if tables:
            offsets = torch.empty(E + 1, dtype=i32, device=dev)
            row_token = torch.empty(T * k, dtype=i32, device=dev)
            token_rows = torch.empty((T, k), dtype=i32, device=dev)
            row_weight = torch.empty(T * k, dtype=f32, device=dev)
            need = _workspace(_lib.OP_ROUTE, T, E, dev)
            if need:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
            rc = _fn("nf4_route_fwd")(d, experts.data_ptr(), weights.data_ptr(), offsets.data_ptr(), row_token.data_ptr(),
                                      token_rows.data_ptr(), row_weight.data_ptr(), ws.data_ptr() if need else None, need,
                                      _raw_stream(dev))
        else:
            rc = _fn("nf4_route_fwd")(d, experts.data_ptr(), weights.data_ptr(), None, None, None, None, None, 0, _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_route_fwd")
    return Routes(experts, weights, offsets, row_token, token_rows, row_weight)


def route_experts_bwd(logits: torch.Tensor, routes: Routes, *, grad_weights: Optional[torch.Tensor] = None,
                      grad_row_weight: Optional[torch.Tensor] = None, score: str = "softmax", renormalise: bool = False,
                      scale: float = 1.0) -> torch.Tensor:
    """nf4_route_bwd: the gradient of the logits of route_experts, in their dtype, from those of `weights` (fp32 [tokens, k])
    and of `row_weight` (fp32 [R], as grouped_swiglu_bwd returns it), either None.  `routes` is the forward's; score,
    renormalise and scale as there.  The choice of the experts has no gradient."""
    name = "route_experts_bwd"
    experts, token_rows, at = routes.experts, routes.token_rows, logits.get_device()
    for t in (experts, token_rows, grad_weights, grad_row_weight):
        if t is not None and t.get_device() != at:
            _one_device(name, logits, experts, token_rows, grad_weights, grad_row_weight)
    if experts.dtype is not torch.int32 or experts.dim() != 2 or experts.shape[:1] != logits.shape[:1] or not experts.is_contiguous():
        raise ValueError(f"{name}: routes.experts must be the contiguous int32 [tokens, k] of the forward")
    T, k = experts.shape
    d, held = _route(name, logits, k, score, None, 1, 1, 1, renormalise, scale, None)
    if grad_weights is not None and (grad_weights.dtype is not torch.float32 or grad_weights.shape != (T, k)):
        raise ValueError(f"{name}: grad_weights must be fp32 [{T}, {k}]")
    if grad_row_weight is not None:
        if grad_row_weight.dtype is not torch.float32 or grad_row_weight.shape != (T * k,):
            raise ValueError(f"{name}: grad_row_weight must be fp32 [{T * k}]")
        if token_rows is None or token_rows.dtype is not torch.int32 or token_rows.shape != (T, k) or not token_rows.is_contiguous():
            raise ValueError(f"{name}: grad_row_weight needs the forward's token_rows")
    gw, gr = (None if g is None else g.contiguous() for g in (grad_weights, grad_row_weight))
    out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    with _on(logits.device):
        rc = _fn("nf4_route_bwd")(d, experts.data_ptr(), None if token_rows is None else token_rows.data_ptr(),
                                  None if gw is None else gw.data_ptr(), None if gr is None else gr.data_ptr(), out.data_ptr(),
                                  logits.shape[1], _raw_stream(logits.device))
    if rc:
        _lib.check(rc, "nf4_route_bwd")
    return out
