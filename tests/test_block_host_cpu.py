"""The host side of the training-block wrappers, without a GPU: what they hand to the library for tensors of unusual
layout, seen through stand-ins that say they lie on a device."""
import pytest
import torch

from bit_nf4_quantized_linear_gb300 import _lib, block_ops


class OnDevice:
    """A CPU tensor that names a CUDA device as its own; `made` lists these with their copies."""

    def __init__(self, t, made, index=0):
        self.t, self.made, self.device, self.is_cuda, self.dtype, self.shape = t, made, torch.device("cuda", index), True, t.dtype, t.shape
        made.append(self)

    def stride(self, *a):
        return self.t.stride(*a)

    def dim(self):
        return self.t.dim()

    def data_ptr(self):
        return self.t.data_ptr()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def contiguous(self):
        return self if self.t.is_contiguous() else OnDevice(self.t.contiguous(), self.made, self.device.index)


class OnCpu:
    """torch, with device memory taken from the host."""

    def __getattr__(self, name):
        return getattr(torch, name)

    @staticmethod
    def empty(*shape, dtype, device):
        return torch.empty(*shape, dtype=dtype)


@pytest.fixture
def calls(monkeypatch):
    """The library calls that the wrappers make, as (name, arguments); none reaches the library."""
    seen = []

    def fn(name):
        def call(*args):
            seen.append((name, args))
            return 0
        return call

    monkeypatch.setattr(block_ops, "_fn", fn)
    monkeypatch.setattr(block_ops, "torch", OnCpu())
    monkeypatch.setattr(block_ops, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(block_ops, "_workspace", lambda *a: 16)
    monkeypatch.setattr(block_ops, "_current_device", lambda: 0, raising=False)
    return seen


def rows(kind, T, H):
    """[T, H] rows of unit column stride: apart, broadcast, or overlapping by half."""
    if kind == "apart":
        return torch.zeros(T, H, dtype=torch.bfloat16)
    if kind == "broadcast":
        return torch.zeros(H, dtype=torch.bfloat16).expand(T, H)
    return torch.zeros(T * (H // 2) + H, dtype=torch.bfloat16).as_strided((T, H), (H // 2, 1))


@pytest.mark.parametrize("which", ["y", "residual", "gate", "gz", "gh"])
@pytest.mark.parametrize("kind", ["apart", "broadcast", "overlapping"])
@pytest.mark.parametrize("T,H", [(37, 640), (1, 640), (5, 1)])
def test_norm_pitches_stay_inside_the_tensors(calls, which, kind, T, H):
    """Rows that share storage (pitch 0, or below the width) are never read with a larger pitch than their own."""
    made = []
    t = {n: OnDevice(rows(kind if n == which else "apart", T, H), made) for n in ("y", "residual", "gate", "gz", "gh")}
    kw = dict(gate=t["gate"], w_pre=OnDevice(torch.ones(H), made))
    block_ops.norm_residual_fwd(t["y"], t["residual"], **kw)
    stats = OnDevice(torch.ones(2, T), made)
    block_ops.norm_residual_bwd(t["gz"], t["gh"], t["y"], t["residual"], stats, **kw)
    for _, args in calls:
        y, ld_y, r, ld_r, g, ld_g, *_ = block_ops._NORM.unpack(args[0])
        places = [("y", y, ld_y), ("residual", r, ld_r), ("gate", g, ld_g)]
        if args is calls[1][1]:
            places += [("gz", args[2], args[3]), ("gh", args[4], args[5])]
        for name, ptr, pitch in places:
            own = next(x.t for x in made if x.data_ptr() == ptr)
            left = own.untyped_storage().nbytes() // 2 - own.storage_offset()
            assert pitch >= H and (T - 1) * pitch + H <= left, (name, pitch, left)
            assert T == 1 or pitch == own.stride(0), name
    assert len(calls) == 2


def test_rows_that_share_storage_are_recognised():
    """Against every element's address, over all small strides."""
    for T, H, D in ((1, 1, 2), (3, 1, 2), (1, 3, 2), (3, 2, 2), (2, 3, 1), (4, 3, 3), (0, 2, 2)):
        for st in range(0, 14):
            for sh in range(0, 14):
                t = torch.zeros(200).as_strided((T, H, D), (st, sh, 1))
                at = [i * st + h * sh + d for i in range(T) for h in range(H) for d in range(D)]
                assert block_ops._share_storage(t) == (len(set(at)) < len(at)), (T, H, D, st, sh)
