"""Torch-facing wrappers of the training-block entry points of ``include/nf4.h``: causal
attention over packed sequences, the gated residual norm, and the AdamW step.

As in ``ops``: PyTorch supplies device memory and the current stream, every step of
the computation runs in the library's kernels, and there is no CPU path.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib, codebooks
from .ops import _device_codebook, _need_cuda, _ptr, _stream, workspace_size

_DTYPES = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16, torch.float16: _lib.DTYPE_F16}


def _one_device(name: str, *ts):
    _need_cuda(name, *ts)
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise ValueError(f"{name}: tensors on different devices {sorted(map(str, devs))}")


def _dtype(name: str, t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: expected fp32, bf16 or fp16, got {t.dtype}")
    return _DTYPES[t.dtype]


# ------------------------------------------------------------------- attention --

def _heads(name: str, what: str, t: torch.Tensor, like: torch.Tensor, shape: tuple) -> torch.Tensor:
    """t as a [T, heads, D] operand with unit stride within a head; `shape` may hold None for a free size."""
    if t.dim() != 3 or any(n is not None and n != s for n, s in zip(shape, t.shape)):
        raise ValueError(f"{name}: {what} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != like.dtype:
        raise ValueError(f"{name}: {what} must have q's dtype")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: {what} must have unit stride within a head")
    return t


def _attention(name, q, k, v, cu_seqlens, scale, more=()):
    _one_device(name, q, k, v, cu_seqlens, *more)
    dt = _dtype(name, q)
    _heads(name, "q", q, q, (None, None, None))
    T, Hq, D = q.shape
    _heads(name, "k", k, q, (T, None, D))
    _heads(name, "v", v, q, tuple(k.shape))
    Hk = k.shape[1]
    if Hk == 0 or Hq == 0 or Hq % Hk != 0:
        raise ValueError(f"{name}: {Hq} query heads do not divide into groups over {Hk} key heads")
    nseq = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 2:
            raise ValueError(f"{name}: cu_seqlens must be a contiguous int32 [sequences + 1] tensor")
        nseq = cu_seqlens.numel() - 1
    return _lib.nf4_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), q.stride(1), k.stride(0), k.stride(1),
                              v.stride(0), v.stride(1), _ptr(cu_seqlens), nseq, T, Hq, Hk, D, dt,
                              D ** -0.5 if scale is None else float(scale))


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None):
    """nf4_attention_fwd: causal attention of packed sequences, q [T, Hq, D] over k, v [T, Hk, D]
    (any token and head strides).  `cu_seqlens` int32 [sequences + 1] holds the row offsets (None:
    one sequence); rows outside them give zeros.  Returns (o [T, Hq, D], lse fp32 [Hq, T])."""
    d = _attention("attention_fwd", q, k, v, cu_seqlens, scale, (out,))
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else _heads(
        "attention_fwd", "out", out, q, tuple(q.shape))
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    _lib.check(_lib.lib().nf4_attention_fwd(ctypes.byref(d), o.data_ptr(), o.stride(0), o.stride(1), lse.data_ptr(),
                                            _stream()), "nf4_attention_fwd")
    return o, lse


def attention_bwd(go: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                  lse: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None):
    """nf4_attention_bwd: the gradients (gq, gk, gv) of attention_fwd from its o, lse and go = dL/do."""
    name = "attention_bwd"
    d = _attention(name, q, k, v, cu_seqlens, scale, (go, o, lse))
    _heads(name, "go", go, q, tuple(q.shape))
    _heads(name, "o", o, q, tuple(q.shape))
    T, Hq, _ = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (Hq, T) or not lse.is_contiguous():
        raise ValueError(f"{name}: lse must be the contiguous fp32 [Hq, T] of the forward")
    gq, gk, gv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    need = workspace_size(_lib.OP_ATTENTION_BWD, T, Hq, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _lib.check(_lib.lib().nf4_attention_bwd(
        ctypes.byref(d), o.data_ptr(), o.stride(0), o.stride(1), lse.data_ptr(), go.data_ptr(), go.stride(0), go.stride(1),
        gq.data_ptr(), gq.stride(0), gq.stride(1), gk.data_ptr(), gk.stride(0), gk.stride(1),
        gv.data_ptr(), gv.stride(0), gv.stride(1), ws.data_ptr(), need, _stream()), name)
    return gq, gk, gv


# --------------------------------------------------------- gated residual norm --

def _rows(name: str, what: str, t: Optional[torch.Tensor], like: torch.Tensor):
    if t is None:
        return
    if t.shape != like.shape or t.dtype != like.dtype or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: {what} must be a {like.dtype} {tuple(like.shape)} tensor with unit column stride")


def _pitch(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else max(t.stride(0), t.shape[1])


def _norm(name, y, residual, w_post, gate, scale, w_pre, eps, more=()):
    _one_device(name, y, residual, w_post, gate, w_pre, *more)
    dt = _dtype(name, y)
    if y.dim() != 2 or y.shape[1] < 1:
        raise ValueError(f"{name}: y must be [tokens, width]")
    _rows(name, "y", y, y)
    _rows(name, "residual", residual, y)
    T, H = y.shape
    for what, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (H,) or not w.is_contiguous()):
            raise ValueError(f"{name}: {what} must be a contiguous fp32 [{H}] tensor")
    kind = _lib.GATE_NONE
    if gate is not None and gate.dim() == 1:
        kind = _lib.GATE_CHANNEL
        if gate.dtype != torch.float32 or tuple(gate.shape) != (H,) or not gate.is_contiguous():
            raise ValueError(f"{name}: a channel gate must be a contiguous fp32 [{H}] tensor")
    elif gate is not None:
        kind = _lib.GATE_TOKEN
        _rows(name, "a token gate", gate, y)
    return _lib.nf4_norm_residual(y.data_ptr(), _pitch(y), _ptr(residual), _pitch(residual), _ptr(gate),
                                  _pitch(gate) if kind == _lib.GATE_TOKEN else 0, _ptr(w_post), _ptr(w_pre), T, H, kind,
                                  dt, float(scale), float(eps))


def norm_residual_fwd(y: torch.Tensor, residual: Optional[torch.Tensor] = None, *, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, w_pre: Optional[torch.Tensor] = None,
                      eps: float = 1e-6):
    """nf4_norm_residual_fwd: z = residual + scale * gate * norm(y; w_post) and h = norm(z; w_pre), the
    norms being x / sqrt(mean(x^2) + eps) * w.  y, residual [T, H]; w_post, w_pre fp32 [H] (w_post None:
    y itself; w_pre None: no h); gate fp32 [H], or [T, H] in y's dtype, or None.  Returns (z, h, stats);
    z is y itself where nothing changes it, and stats (fp32 [2, T]) is what the backward needs."""
    name = "norm_residual_fwd"
    d = _norm(name, y, residual, w_post, gate, scale, w_pre, eps)
    same = residual is None and w_post is None and gate is None and float(scale) == 1.0
    T, H = y.shape
    z = y if same else torch.empty((T, H), dtype=y.dtype, device=y.device)
    h = None if w_pre is None else torch.empty((T, H), dtype=y.dtype, device=y.device)
    stats = torch.empty((2, T), dtype=torch.float32, device=y.device)
    _lib.check(_lib.lib().nf4_norm_residual_fwd(ctypes.byref(d), None if same else z.data_ptr(), H, _ptr(h), H,
                                                stats.data_ptr(), _stream()), "nf4_norm_residual_fwd")
    return z, h, stats


def norm_residual_bwd(gz: Optional[torch.Tensor], gh: Optional[torch.Tensor], y: torch.Tensor,
                      residual: Optional[torch.Tensor], stats: torch.Tensor, *, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, w_pre: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, need_y: bool = True, need_residual: bool = True, need_vectors: bool = True):
    """nf4_norm_residual_bwd: from gz = dL/dz and gh = dL/dh (None: zero) the gradients
    (gy, gresidual, gw_post, ggate, gw_pre) of norm_residual_fwd's inputs, None for absent or unwanted
    ones (`need_vectors` covers the two gains and the gate).  gw_* and a channel gate's gradient are
    fp32 [H]; a token gate's has the gate's shape and dtype."""
    name = "norm_residual_bwd"
    d = _norm(name, y, residual, w_post, gate, scale, w_pre, eps, (gz, gh, stats))
    _rows(name, "gz", gz, y)
    _rows(name, "gh", gh, y)
    T, H = y.shape
    if stats.dtype != torch.float32 or tuple(stats.shape) != (2, T) or not stats.is_contiguous():
        raise ValueError(f"{name}: stats must be the contiguous fp32 [2, T] of the forward")
    if gh is not None and w_pre is None:
        raise ValueError(f"{name}: gh without w_pre")

    def rows(want):
        return torch.empty((T, H), dtype=y.dtype, device=y.device) if want else None

    def vector(want):
        return torch.empty(H, dtype=torch.float32, device=y.device) if want and need_vectors else None

    gy, gr = rows(need_y), rows(need_residual and residual is not None)
    gw_post, gw_pre = vector(w_post is not None), vector(w_pre is not None)
    ggate = rows(need_vectors) if d.gate_kind == _lib.GATE_TOKEN else vector(gate is not None)
    ws, need = None, 0
    if gw_post is not None or gw_pre is not None or (ggate is not None and d.gate_kind == _lib.GATE_CHANNEL):
        need = workspace_size(_lib.OP_NORM_RESIDUAL_BWD, T, H, 0)
        ws = torch.empty(need, dtype=torch.uint8, device=y.device)
    _lib.check(_lib.lib().nf4_norm_residual_bwd(
        ctypes.byref(d), stats.data_ptr(), _ptr(gz), _pitch(gz), _ptr(gh), _pitch(gh), _ptr(gy), H, _ptr(gr), H,
        _ptr(gw_post), _ptr(ggate), H, _ptr(gw_pre), _ptr(ws), need, _stream()), "nf4_norm_residual_bwd")
    return gy, gr, gw_post, ggate, gw_pre


# ----------------------------------------------------------------------- AdamW --

class AdamWState:
    """The two moments of a list of tensors, in fp32 or in 8 bits, kept in one flat buffer each.

    Tensor i occupies `slices[i]` of `exp_avg` and `exp_avg_sq` (fp32 values, or uint8 codes), starting at
    a multiple of 256; with 8 bits, every 256 values share a scale in `exp_avg_absmax` and
    `exp_avg_sq_absmax`.  `step` is the number of steps taken."""

    def __init__(self, params: Sequence[torch.Tensor], bits: int = 8):
        name = "adamw_state"
        if bits not in (8, 32):
            raise ValueError(f"{name}: bits must be 8 or 32")
        params = list(params)
        if not params:
            raise ValueError(f"{name}: no tensors")
        _one_device(name, *params)
        self.bits, self.step, self.device = bits, 0, params[0].device
        self.numels = [p.numel() for p in params]
        self.slices, at = [], 0
        for n in self.numels:
            self.slices.append(slice(at, at + n))
            at += -(-n // _lib.ADAMW_BLOCK) * _lib.ADAMW_BLOCK
        self.exp_avg_absmax = self.exp_avg_sq_absmax = None
        self.levels = (None, None)
        if bits == 32:
            self.exp_avg, self.exp_avg_sq = (torch.zeros(at, dtype=torch.float32, device=self.device) for _ in range(2))
        else:
            self.levels = (_device_codebook("dynamic8", self.device, codebooks.dynamic_code8),
                           _device_codebook("dynamic8_unsigned", self.device, codebooks.dynamic_code8_unsigned))
            zero = [int((c == 0).nonzero()[0]) for c in (codebooks.dynamic_code8(), codebooks.dynamic_code8_unsigned())]
            self.exp_avg, self.exp_avg_sq = (torch.full((at,), z, dtype=torch.uint8, device=self.device) for z in zero)
            self.exp_avg_absmax, self.exp_avg_sq_absmax = (
                torch.zeros(at // _lib.ADAMW_BLOCK, dtype=torch.float32, device=self.device) for _ in range(2))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.exp_avg, self.exp_avg_sq, self.exp_avg_absmax, self.exp_avg_sq_absmax) if t is not None)

    def _table(self):
        """The C table with the states' pointers; param and grad are filled in by each call."""
        tab = (_lib.nf4_adamw_tensor * len(self.numels))()
        size = self.exp_avg.element_size()
        for row, n, sl in zip(tab, self.numels, self.slices):
            row.m = self.exp_avg.data_ptr() + sl.start * size
            row.v = self.exp_avg_sq.data_ptr() + sl.start * size
            if self.bits == 8:
                row.m_absmax = self.exp_avg_absmax.data_ptr() + sl.start // _lib.ADAMW_BLOCK * 4
                row.v_absmax = self.exp_avg_sq_absmax.data_ptr() + sl.start // _lib.ADAMW_BLOCK * 4
            row.n = n
        return tab


def adamw_state(params: Sequence[torch.Tensor], bits: int = 8) -> AdamWState:
    """Zero moments for `params`, in 8 or 32 bits."""
    return AdamWState(params, bits)


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[Optional[torch.Tensor]], state: AdamWState, *, lr: float,
               betas: tuple = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: Optional[torch.Tensor] = None) -> None:
    """nf4_adamw_step: one AdamW step over all tensors in place (params, state; state.step advances).
    Parameters and gradients are contiguous and of one dtype; a gradient of None leaves its tensor and
    states alone.  `grad_scale`, a device fp32 scalar, multiplies the gradients (a clipping factor)."""
    name = "adamw_step"
    if len(params) != len(state.numels) or len(grads) != len(params):
        raise ValueError(f"{name}: {len(params)} tensors and {len(grads)} gradients for a state of {len(state.numels)}")
    dtype = params[0].dtype
    dt = _dtype(name, params[0])
    tab = state._table()
    for i, (p, g) in enumerate(zip(params, grads)):
        row = tab[i]
        if p.dtype != dtype or p.device != state.device or not p.is_contiguous() or p.numel() != row.n:
            raise ValueError(f"{name}: tensor {i} must be contiguous, {dtype}, on {state.device} and of {row.n} values")
        if g is None:
            row.n = 0
            continue
        if g.dtype != dtype or g.device != p.device or not g.is_contiguous() or g.shape != p.shape:
            raise ValueError(f"{name}: gradient {i} must be contiguous and of its tensor's shape, dtype and device")
        row.param, row.grad = p.data_ptr(), g.data_ptr()
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.device != state.device):
        raise ValueError(f"{name}: grad_scale must be one fp32 value on {state.device}")
    _lib.check(_lib.lib().nf4_adamw_step(tab, len(params), dt, state.bits, _ptr(state.levels[0]), _ptr(state.levels[1]),
                                         float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay),
                                         state.step + 1, _ptr(grad_scale), _stream()), "nf4_adamw_step")
    state.step += 1


def adamw_state_values(state: AdamWState):
    """The moments as fp32 values, (exp_avg, exp_avg_sq), laid out as the state's flat buffers: the
    buffers themselves for fp32 states, nf4_adamw_state_values of 8-bit ones."""
    if state.bits == 32:
        return state.exp_avg, state.exp_avg_sq
    m, v = (torch.empty(state.exp_avg.numel(), dtype=torch.float32, device=state.device) for _ in range(2))
    _lib.check(_lib.lib().nf4_adamw_state_values(
        _ptr(state.exp_avg), _ptr(state.exp_avg_sq), _ptr(state.exp_avg_absmax), _ptr(state.exp_avg_sq_absmax),
        _ptr(state.levels[0]), _ptr(state.levels[1]), m.numel(), m.data_ptr(), v.data_ptr(), _stream()),
        "nf4_adamw_state_values")
    return m, v
