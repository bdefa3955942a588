"""AdamW for the trained tensors beside the frozen weights, over the library's many-tensor step."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib, block_ops


class NF4AdamW(torch.optim.Optimizer):
    """AdamW whose step is one launch per parameter group and dtype (nf4_adamw_step), with the two moments
    in 8 bits (256-value blocks of the dynamic map) or in fp32.  A parameter's steps count its own gradients;
    where the counts of a group differ, each count is a launch.

    Options per group as in torch.optim.AdamW: lr, betas, eps, weight_decay; `state_bits` is 8 or 32.  A
    group's parameters are contiguous CUDA tensors on one device, of fp32, bf16 or fp16.  The state of a group
    is made at its first step and lies in `group_state` (one AdamWState per group and dtype)."""

    def __init__(self, params, lr: float = 2e-4, betas: tuple = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 8):
        if state_bits not in (8, 32):
            raise ValueError("NF4AdamW: state_bits must be 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits))
        self.group_state = {}

    def _sets(self):
        """(key, group, parameters) of each group and dtype."""
        for i, group in enumerate(self.param_groups):
            by = {}
            for p in group["params"]:
                by.setdefault(p.dtype, []).append(p)
            for dtype, ps in by.items():
                yield (i, str(dtype)), group, ps

    def _state(self, key, group, ps) -> block_ops.AdamWState:
        st = self.group_state.get(key)
        if st is None:
            st = self.group_state[key] = block_ops.adamw_state([p.detach() for p in ps], bits=group["state_bits"])
        return st

    @torch.no_grad()
    def step(self, closure=None, grad_scale: Optional[torch.Tensor] = None):
        """One step; `grad_scale`, a device fp32 scalar, multiplies every gradient (a clipping factor).  A
        parameter without a gradient is left alone.  Not to be captured in a CUDA graph: the number of the step,
        and with it the bias correction, is fixed at the launch, and a replay would repeat it."""
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("NF4AdamW: a step cannot be captured in a CUDA graph (its number is fixed at the launch)")
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for key, group, ps in self._sets():
            grads = [None if p.grad is None else p.grad.contiguous() for p in ps]
            if all(g is None for g in grads):
                continue
            block_ops.adamw_step([p.detach() for p in ps], grads, self._state(key, group, ps), lr=group["lr"],
                                 betas=group["betas"], eps=group["eps"], weight_decay=group["weight_decay"],
                                 grad_scale=grad_scale, per_tensor=True)
        return loss

    def __getstate__(self):
        return dict(super().__getstate__(), group_state=self.group_state)

    def __setstate__(self, state):
        super().__setstate__(state)
        self.__dict__.setdefault("group_state", {})  # a copy made without one

    def state_dict(self):
        d = super().state_dict()
        d["group_state"] = {key: dict(bits=st.bits, step=st.step, missed=dict(st.missed),
                                      shapes=[tuple(s) for s in st.shapes], buffers=list(st._buffers()))
                            for key, st in self.group_state.items()}
        return d

    def load_state_dict(self, state_dict):
        """Takes over a state_dict's options and moments.  Every saved state has to belong to a group and dtype of
        this optimiser, with tensors of the saved shapes; a group that had not stepped when it was saved has none and
        starts anew.  A refusal changes nothing."""
        state_dict = dict(state_dict)
        held = state_dict.pop("group_state")
        sets = {key: ps for key, _, ps in self._sets()}
        for key, rec in held.items():
            shapes = [tuple(p.shape) for p in sets.get(key, ())]
            size = sum(-(-p.numel() // _lib.ADAMW_BLOCK) * _lib.ADAMW_BLOCK for p in sets.get(key, ()))
            scales = size // _lib.ADAMW_BLOCK if rec["bits"] == 8 else None
            # records from before the shapes were kept: the buffers' lengths are all there is
            if (key not in sets or list(map(tuple, rec.get("shapes", shapes))) != shapes
                    or [None if b is None else b.numel() for b in rec["buffers"]] != [size, size, scales, scales]):
                raise ValueError(f"NF4AdamW: the saved state of group {key[0]}, {key[1]} belongs to other parameters")
        super().load_state_dict(state_dict)
        self.group_state = {}
        for key, rec in held.items():
            st = self.group_state[key] = block_ops.adamw_state([p.detach() for p in sets[key]], bits=rec["bits"])
            st.step, st.missed = int(rec["step"]), dict(rec.get("missed", {}))
            for saved, own in zip(rec["buffers"], st._buffers()):
                if own is not None:
                    own.copy_(saved)
