"""Torch-facing wrappers of the training-block entry points of ``include/nf4.h``: causal
attention over packed sequences, the gated residual norm, and the AdamW step.

As in ``ops``: PyTorch supplies device memory and the current stream, every step of
the computation runs in the library's kernels, and there is no CPU path.
"""
from __future__ import annotations

import contextlib
import functools
import itertools
import struct
from typing import Optional, Sequence

import torch

from . import _lib, codebooks
from .ops import _device_codebook, _need_cuda, _ptr, workspace_size

# The calls of a training step are short next to what the host spends on them, so the
# wrappers check their arguments in single expressions (a failed one is then explained by a
# slower function), pass structs as packed bytes and look the library's functions up once.

_DTYPES = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16, torch.float16: _lib.DTYPE_F16}
_ATTENTION = struct.Struct("@3P6qP2q4if4xP")     # nf4_attention
_NORM = struct.Struct("@PqPqPqPP2q2i2f")        # nf4_norm_residual
_FNS = {}


def _fn(name: str):
    f = _FNS.get(name)
    if f is None:
        f = _FNS[name] = getattr(_lib.lib(), name)
    return f


def _raw_stream(device: torch.device) -> int:
    """The current stream of `device`."""
    return torch._C._cuda_getCurrentRawStream(device.index)


_written = torch._C._increment_version  # torch.autograd.graph.increment_version of a list
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # None: a torch without CUDA, which gets no further
_guard, _HERE = torch.cuda.device, contextlib.nullcontext()


def _on(device: torch.device):
    """A context in which `device` is the current one, as the library's launches and size queries need it."""
    return _HERE if _current_device() == device.index else _guard(device)


@functools.lru_cache(maxsize=4096)
def _workspace(op: int, M: int, N: int, device: torch.device) -> int:
    return workspace_size(op, M, N, 0)


@functools.lru_cache(maxsize=64)
def _workspace5(op: int, M: int, N: int, K: int, E: int, device: torch.device) -> int:
    return workspace_size(op, M, N, K, E)


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

def _heads(name: str, what: str, t: torch.Tensor, like: torch.Tensor, shape: tuple):
    """Explains why t is no [T, heads, D] operand; `shape` may hold None for a free size."""
    if t.dim() != 3 or any(n is not None and n != s for n, s in zip(shape, t.shape)):
        raise ValueError(f"{name}: {what} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != like.dtype:
        raise ValueError(f"{name}: {what} must have q's dtype")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: {what} must have unit stride within a head")


def _explain_attention(name, q, k, v, cu_seqlens, like_q):
    _one_device(name, q, k, v, cu_seqlens, *(t for _, t in like_q))
    _dtype(name, q)
    _heads(name, "q", q, q, (None, None, None))
    T, Hq, D = q.shape
    _heads(name, "k", k, q, (T, None, D))
    _heads(name, "v", v, q, tuple(k.shape))
    for what, t in like_q:
        _heads(name, what, t, q, (T, Hq, D))
    Hk = k.shape[1]
    if Hk == 0 or Hq == 0 or Hq % Hk != 0:
        raise ValueError(f"{name}: {Hq} query heads do not divide into groups over {Hk} key heads")
    raise ValueError(f"{name}: cu_seqlens must be a contiguous int32 [sequences + 1] tensor")


def _attention(name, q, k, v, cu_seqlens, scale, rest, like_q=()):
    """The packed nf4_attention of checked arguments; like_q: (what, tensor) of q's shape and dtype."""
    dt, dev, qs, ks, qt, kt, vt = q.dtype, q.device, q.shape, k.shape, q.stride(), k.stride(), v.stride()
    ok = (dt in _DTYPES and dev.type == "cuda" and k.dtype is dt and v.dtype is dt and k.device == dev and v.device == dev
          and len(qs) == 3 and len(ks) == 3 and ks == v.shape and ks[0] == qs[0] and ks[2] == qs[2] and ks[1] > 0
          and qs[1] > 0 and qs[1] % ks[1] == 0 and (qs[2] == 1 or qt[2] == kt[2] == vt[2] == 1))
    for _, t in like_q if ok else ():
        ok = ok and t.dtype is dt and t.device == dev and t.shape == qs and (qs[2] == 1 or t.stride(2) == 1)
    nseq = cu = 0
    if cu_seqlens is not None:
        nseq = cu_seqlens.numel() - 1
        cu = cu_seqlens.data_ptr()
        ok = (ok and cu_seqlens.dtype is torch.int32 and cu_seqlens.dim() == 1 and nseq > 0 and cu_seqlens.stride(0) == 1
              and cu_seqlens.device == dev)
    if not ok:
        _explain_attention(name, q, k, v, cu_seqlens, like_q)
    T, Hq, D = qs
    return _ATTENTION.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), qt[0], qt[1], kt[0], kt[1], vt[0], vt[1], cu, nseq, T,
                           Hq, ks[1], D, _DTYPES[dt], D ** -0.5 if scale is None else scale,
                           0 if rest is None else rest.data_ptr())


def _share_storage(t: torch.Tensor) -> bool:
    """Whether two rows of a [T, heads, D] tensor meet in memory."""
    (T, H, D), (st, sh, _) = t.shape, t.stride()
    reach = D
    for stride, n in sorted((s, n) for s, n in ((st, T), (sh, H)) if n > 1):
        if stride < reach and T > 0:
            break
        reach += stride * (n - 1)
    else:
        return False  # one dimension inside the other's steps
    # interleaved: heads dh apart meet tokens dt apart where dh sh - dt st is less than a row
    return (T > 1 and st < D) or any(abs(dh * sh - dt * st) < D for dh in range(1, H) for dt in
                                     ({min(T - 1, dh * sh // st), min(T - 1, dh * sh // st + 1)} if st else {0}))


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, for_backward: bool = True):
    """nf4_attention_fwd: causal attention of packed sequences, q [T, Hq, D] over k, v [T, Hk, D]
    (any token and head strides).  `cu_seqlens` int32 [sequences + 1] holds the row offsets (None:
    one sequence); rows outside them give zeros.  Returns (o [T, Hq, D], lse fp32 [Hq, T]).  With
    `for_backward` and a 16-bit dtype, `lse.o_rest` is a tensor of o's shape with what o's rounding
    left over, for attention_bwd; a caller that wants no gradients saves its memory with False.  `out` takes o
    in place of a new tensor: any token and head strides whose rows do not share storage."""
    rest = None
    if for_backward and q.dtype is not torch.float32 and q.dim() == 3 and q.is_cuda:
        rest = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    d = _attention("attention_fwd", q, k, v, cu_seqlens, scale, rest, () if out is None else (("out", out),))
    if out is not None and _share_storage(out):
        raise ValueError("attention_fwd: rows of out share storage")
    T, Hq, D = q.shape
    o = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device) if out is None else out
    lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    ot, oh, _ = o.stride()
    with _on(q.device):
        rc = _fn("nf4_attention_fwd")(d, o.data_ptr(), ot, oh, lse.data_ptr(), _raw_stream(q.device))
    if rc:
        _lib.check(rc, "nf4_attention_fwd")
    if out is not None:
        _written((out,))
    lse.o_rest = rest
    return o, lse


def attention_bwd(go: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                  lse: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  o_rest: Optional[torch.Tensor] = None):
    """nf4_attention_bwd: the gradients (gq, gk, gv) of attention_fwd from its o, lse and go = dL/do.  `o_rest`
    is the forward's `lse.o_rest` (taken from lse where it still carries it); without it the row sums do . o
    see the rounded o."""
    rest = getattr(lse, "o_rest", None) if o_rest is None else o_rest
    if rest is not None and (rest.shape != q.shape or rest.dtype is not q.dtype or not rest.is_contiguous() or rest.device != q.device
                             or q.dtype is torch.float32):
        raise ValueError("attention_bwd: o_rest must be the forward's, contiguous and of q's shape and 16-bit dtype")
    d = _attention("attention_bwd", q, k, v, cu_seqlens, scale, rest, (("go", go), ("o", o)))
    T, Hq, D = q.shape
    dev, dt = q.device, q.dtype
    if lse.dtype is not torch.float32 or lse.shape != (Hq, T) or not lse.is_contiguous() or lse.device != dev:
        raise ValueError("attention_bwd: lse must be the contiguous fp32 [Hq, T] of the forward")
    Hk = k.shape[1]
    gq = torch.empty((T, Hq, D), dtype=dt, device=dev)
    gk = torch.empty((T, Hk, D), dtype=dt, device=dev)
    gv = torch.empty((T, Hk, D), dtype=dt, device=dev)
    ot, oh, _ = o.stride()
    gt, gh, _ = go.stride()
    # A gradient that no bulk copy can load (broadcast over tokens or heads, off 16 bytes) is copied: two passes over
    # it, where the kernels for any layout would take some hundred times the products' time.
    if dt is not torch.float32 and D <= 128 and D % 8 == 0 and (gt < 1 or gh < 1 or (gt | gh) & 7 or go.data_ptr() & 15):
        go = go.clone(memory_format=torch.contiguous_format)
        gt, gh, _ = go.stride()
    with _on(dev):
        need = _workspace(_lib.OP_ATTENTION_BWD, T, Hq, dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = _fn("nf4_attention_bwd")(d, o.data_ptr(), ot, oh, lse.data_ptr(), go.data_ptr(), gt, gh, gq.data_ptr(), Hq * D, D,
                                      gk.data_ptr(), Hk * D, D, gv.data_ptr(), Hk * D, D, ws.data_ptr(), need, _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_attention_bwd")
    return gq, gk, gv


# --------------------------------------------------------- gated residual norm --

def _explain_norm(name, y, w_post, gate, w_pre, rows):
    _one_device(name, y, w_post, gate, w_pre, *(t for _, t in rows))
    _dtype(name, y)
    if y.dim() != 2 or y.shape[1] < 1:
        raise ValueError(f"{name}: y must be [tokens, width]")
    H = y.shape[1]
    for what, t in (("y", y), ("a token gate", gate if gate is not None and gate.dim() != 1 else None), *rows):
        if t is not None and (t.shape != y.shape or t.dtype != y.dtype or (H > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name}: {what} must be a {y.dtype} {tuple(y.shape)} tensor with unit column stride")
    for what, w in (("w_post", w_post), ("w_pre", w_pre), ("a channel gate", gate)):
        if w is not None and w.dim() == 1 and (w.dtype != torch.float32 or tuple(w.shape) != (H,) or not w.is_contiguous()):
            raise ValueError(f"{name}: {what} must be a contiguous fp32 [{H}] tensor")
    raise ValueError(f"{name}: the gains must be contiguous fp32 [{H}] tensors")


def _norm(name, y, w_post, gate, scale, w_pre, eps, rows):
    """The packed nf4_norm_residual of checked arguments, the gate's kind, the row pitches of `rows`, which starts
    with the residual ((what, tensor or None) of y's shape and dtype), and the tensors that the pointers lie in: those
    of `rows`, y and the gate.  A pitch is the row width at least, so rows that share storage (broadcast over the
    tokens, or overlapping) are copied; the pitch of a single row is never used."""
    dt, dev, ys = y.dtype, y.device, y.shape
    H = ys[-1] if len(ys) == 2 else 0
    ok = dt in _DTYPES and dev.type == "cuda" and H > 0 and (H == 1 or y.stride(1) == 1)
    kind, gp, gl = _lib.GATE_NONE, 0, 0
    wp = wn = 0
    pitches, held = [], []
    if ok:
        T = ys[0]
        if T > 1 and y.stride(0) < H:
            y = y.contiguous()
        for _, t in rows:
            if t is not None:
                ok = ok and t.dtype is dt and t.device == dev and t.shape == ys and (H == 1 or t.stride(1) == 1)
                if ok and T > 1 and t.stride(0) < H:
                    t = t.contiguous()
            held.append(t)
            pitches.append(0 if t is None or not ok else t.stride(0) if T > 1 else H)
        if w_post is not None:
            wp = w_post.data_ptr()
            ok = (ok and w_post.dtype is torch.float32 and w_post.shape == (H,) and w_post.device == dev
                  and w_post.is_contiguous())
        if w_pre is not None:
            wn = w_pre.data_ptr()
            ok = ok and w_pre.dtype is torch.float32 and w_pre.shape == (H,) and w_pre.device == dev and w_pre.is_contiguous()
        if gate is not None:
            if gate.dim() == 1:
                kind = _lib.GATE_CHANNEL
                ok = ok and gate.dtype is torch.float32 and gate.shape == (H,) and gate.device == dev and gate.is_contiguous()
            else:
                kind = _lib.GATE_TOKEN
                ok = ok and gate.dtype is dt and gate.device == dev and gate.shape == ys and (H == 1 or gate.stride(1) == 1)
                if ok and T > 1 and gate.stride(0) < H:
                    gate = gate.contiguous()
                gl = gate.stride(0) if ok and T > 1 else H
            gp = gate.data_ptr()
    if not ok:
        _explain_norm(name, y, w_post, gate, w_pre, rows)
    residual = held[0]
    d = _NORM.pack(y.data_ptr(), y.stride(0) if T > 1 else H, 0 if residual is None else residual.data_ptr(), pitches[0], gp, gl,
                   wp, wn, T, H, kind, _DTYPES[dt], scale, eps)
    return d, kind, pitches, (*held, y, gate)


def norm_residual_fwd(y: torch.Tensor, residual: Optional[torch.Tensor] = None, *, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, w_pre: Optional[torch.Tensor] = None,
                      eps: float = 1e-6):
    """nf4_norm_residual_fwd: z = residual + scale * gate * norm(y; w_post) and h = norm(z; w_pre), the
    norms being x / sqrt(mean(x^2) + eps) * w.  y, residual [T, H]; w_post, w_pre fp32 [H] (w_post None:
    y itself; w_pre None: no h); gate fp32 [H], or [T, H] in y's dtype, or None.  Rows may lie at any distance;
    those that share storage (an expanded row) are copied first.  Returns (z, h, stats);
    z is y itself where nothing changes it, and stats (fp32 [2, T]) is what the backward needs."""
    d, _, _, _held = _norm("norm_residual_fwd", y, w_post, gate, scale, w_pre, eps, (("residual", residual),))
    same = residual is None and w_post is None and gate is None and scale == 1.0
    (T, H), dt, dev = y.shape, y.dtype, y.device
    z = y if same else torch.empty((T, H), dtype=dt, device=dev)
    h = None if w_pre is None else torch.empty((T, H), dtype=dt, device=dev)
    stats = torch.empty((2, T), dtype=torch.float32, device=dev)
    with _on(dev):
        rc = _fn("nf4_norm_residual_fwd")(d, None if same else z.data_ptr(), H, _ptr(h), H, stats.data_ptr(), _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_norm_residual_fwd")
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
    d, kind, (_, pitch_z, pitch_h), held = _norm(name, y, w_post, gate, scale, w_pre, eps,
                                                 (("residual", residual), ("gz", gz), ("gh", gh)))
    (T, H), dt, dev = y.shape, y.dtype, y.device
    if stats.dtype is not torch.float32 or stats.shape != (2, T) or not stats.is_contiguous() or stats.device != dev:
        raise ValueError(f"{name}: stats must be the contiguous fp32 [2, T] of the forward")
    if gh is not None and w_pre is None:
        raise ValueError(f"{name}: gh without w_pre")
    f32 = torch.float32
    gy = torch.empty((T, H), dtype=dt, device=dev) if need_y else None
    gr = torch.empty((T, H), dtype=dt, device=dev) if need_residual and residual is not None else None
    gw_post = torch.empty(H, dtype=f32, device=dev) if need_vectors and w_post is not None else None
    gw_pre = torch.empty(H, dtype=f32, device=dev) if need_vectors and w_pre is not None else None
    ggate = None
    if need_vectors and kind != _lib.GATE_NONE:
        ggate = torch.empty((T, H), dtype=dt, device=dev) if kind == _lib.GATE_TOKEN else torch.empty(H, dtype=f32, device=dev)
    ws, need = None, 0
    with _on(dev):
        if gw_post is not None or gw_pre is not None or (ggate is not None and kind == _lib.GATE_CHANNEL):
            need = _workspace(_lib.OP_NORM_RESIDUAL_BWD, T, H, dev)
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = _fn("nf4_norm_residual_bwd")(d, stats.data_ptr(), _ptr(held[1]), pitch_z, _ptr(held[2]), pitch_h, _ptr(gy), H,
                                          _ptr(gr), H, _ptr(gw_post), _ptr(ggate), H, _ptr(gw_pre), _ptr(ws), need,
                                          _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_norm_residual_bwd")
    return gy, gr, gw_post, ggate, gw_pre


# ----------------------------------------------------------------------- AdamW --

class AdamWState:
    """The two moments of a list of tensors, in fp32 or in 8 bits, kept in one flat buffer each.

    Tensor i occupies `slices[i]` of `exp_avg` and `exp_avg_sq` (fp32 values, or uint8 codes), starting at
    a multiple of 256; with 8 bits, every 256 values share a scale in `exp_avg_absmax` and
    `exp_avg_sq_absmax`.  `step` is the number of steps taken, and `missed` says in how many of them a tensor
    had no gradient (index: count; tensors that missed none are not in it)."""

    def __init__(self, params: Sequence[torch.Tensor], bits: int = 8):
        name = "adamw_state"
        if bits not in (8, 32):
            raise ValueError(f"{name}: bits must be 8 or 32")
        params = list(params)
        if not params:
            raise ValueError(f"{name}: no tensors")
        _one_device(name, *params)
        self.bits, self.step, self.missed, self.device = bits, 0, {}, params[0].device
        self.shapes = [p.size() for p in params]
        self._rows, self._held = struct.Struct("@" + "6Pq" * len(params)), None  # nf4_adamw_tensor
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

    def __getstate__(self):  # a Struct cannot be pickled, and the addresses are those of this state's buffers
        return {k: v for k, v in self.__dict__.items() if k not in ("_rows", "_held")}

    def __setstate__(self, state):
        self.__dict__.update(state, _rows=struct.Struct("@" + "6Pq" * len(state["numels"])), _held=None)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._buffers() if t is not None)

    def _buffers(self):
        return self.exp_avg, self.exp_avg_sq, self.exp_avg_absmax, self.exp_avg_sq_absmax

    def _columns(self):
        """The C table's columns that lie in the state's own buffers: a pointer to each moment and scale of every
        tensor, and its size."""
        m, v, ma, va = base = tuple(0 if t is None else t.data_ptr() for t in self._buffers())
        if self._held is None or self._held[0] != base:  # the buffers were replaced
            size, per = self.exp_avg.element_size(), 4 if self.bits == 8 else 0
            at = [s.start for s in self.slices]
            block = [a // _lib.ADAMW_BLOCK * per for a in at]
            self._held = (base, [m + a * size for a in at], [v + a * size for a in at], [ma + b for b in block],
                          [va + b for b in block])
        return self._held[1:]

    def _table(self, params, grads) -> bytes:
        """The packed nf4_adamw_tensor rows from the tensors' addresses; a gradient of 0 makes an empty row."""
        n = self.numels if 0 not in grads else [n if g else 0 for n, g in zip(self.numels, grads)]
        return self._rows.pack(*itertools.chain.from_iterable(zip(params, grads, *self._columns(), n)))


def adamw_state(params: Sequence[torch.Tensor], bits: int = 8) -> AdamWState:
    """Zero moments for `params`, in 8 or 32 bits."""
    return AdamWState(params, bits)


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[Optional[torch.Tensor]], state: AdamWState, *, lr: float,
               betas: tuple = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: Optional[torch.Tensor] = None, per_tensor: bool = False) -> None:
    """nf4_adamw_step: one AdamW step over all tensors in place (params, state; state.step advances).
    Parameters and gradients are contiguous and of one dtype; a gradient of None leaves its tensor and
    states alone.  The step is number state.step + 1 for every tensor; with `per_tensor` a tensor's number
    counts its own gradients only (a launch for each number), so that moments which start late get the bias
    correction of their start.  The number is fixed at the launch: a replayed CUDA graph repeats it, and
    `state` does not count replays.  `grad_scale`, a device fp32 scalar, multiplies the gradients (a
    clipping factor)."""
    name = "adamw_step"
    n = len(state.numels)
    if len(params) != n or len(grads) != n:
        raise ValueError(f"{name}: {len(params)} tensors and {len(grads)} gradients for a state of {n}")
    T, dtype, dev = torch.Tensor, params[0].dtype, state.device
    some = [g for g in grads if g is not None]
    full = len(some) == n
    every = [*params, *some]
    shapes = state.shapes if full else [s for s, g in zip(state.shapes, grads) if g is not None]
    if not (dtype in _DTYPES and all(map(T.is_contiguous, every)) and list(map(T.size, params)) == state.shapes
            and list(map(T.size, some)) == shapes and {t.dtype for t in every} == {dtype} and set(map(T.get_device, every)) == {dev.index}):
        _explain_adamw(name, params, grads, state)
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.device != dev):
        raise ValueError(f"{name}: grad_scale must be one fp32 value on {dev}")
    ptrs = list(map(T.data_ptr, some))
    if not full:
        it = iter(ptrs)
        ptrs = [0 if g is None else next(it) for g in grads]
    numbers = {state.step + 1: ptrs}
    if per_tensor and state.missed:
        own = [state.step + 1 - state.missed.get(i, 0) for i in range(n)]
        numbers = {s: [p if s == m else 0 for p, m in zip(ptrs, own)] for s in {m for m, g in zip(own, grads) if g is not None}}
    at = list(map(T.data_ptr, params))
    with _on(dev):
        for step, ptrs in numbers.items():
            rc = _fn("nf4_adamw_step")(state._table(at, ptrs), n, _DTYPES[dtype], state.bits, _ptr(state.levels[0]),
                                       _ptr(state.levels[1]), lr, betas[0], betas[1], eps, weight_decay, step, _ptr(grad_scale),
                                       _raw_stream(dev))
            if rc:
                _lib.check(rc, "nf4_adamw_step")
    # autograd's record of writes that it did not see
    _written(params if full else [p for p, g in zip(params, grads) if g is not None])
    state.step += 1
    if not full:
        for i, g in enumerate(grads):
            if g is None:
                state.missed[i] = state.missed.get(i, 0) + 1


def _explain_adamw(name, params, grads, state):
    dtype = params[0].dtype
    _dtype(name, params[0])
    for i, (p, g, shape) in enumerate(zip(params, grads, state.shapes)):
        if p.dtype != dtype or p.device != state.device or not p.is_contiguous() or p.shape != shape:
            raise ValueError(f"{name}: tensor {i} must be contiguous, {dtype}, on {state.device} and of shape {tuple(shape)}")
        if g is not None and (g.dtype != dtype or g.device != p.device or not g.is_contiguous() or g.shape != p.shape):
            raise ValueError(f"{name}: gradient {i} must be contiguous and of its tensor's shape, dtype and device")
    raise ValueError(f"{name}: tensors and gradients do not fit the state")


def adamw_state_values(state: AdamWState):
    """The moments as fp32 values, (exp_avg, exp_avg_sq), laid out as the state's flat buffers: the
    buffers themselves for fp32 states, nf4_adamw_state_values of 8-bit ones."""
    if state.bits == 32:
        return state.exp_avg, state.exp_avg_sq
    m, v = (torch.empty(state.exp_avg.numel(), dtype=torch.float32, device=state.device) for _ in range(2))
    with _on(state.device):
        rc = _fn("nf4_adamw_state_values")(
            _ptr(state.exp_avg), _ptr(state.exp_avg_sq), _ptr(state.exp_avg_absmax), _ptr(state.exp_avg_sq_absmax),
            _ptr(state.levels[0]), _ptr(state.levels[1]), m.numel(), m.data_ptr(), v.data_ptr(), _raw_stream(state.device))
    _lib.check(rc, "nf4_adamw_state_values")
    return m, v
