"""Layouts and values of the training-block operators that programs meet beside the ordinary ones: rows that share
storage, gradients of unusual size, infinities that are seen."""
import math

import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from tests import block_refs as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    nf4.device_status(clear=True)
    yield
    assert nf4.device_status() == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device=DEV)


# ---------------------------------------------------------------- residual norm --

def overlapping(n, T, H, dtype):
    """Rows whose pitch is half their width."""
    return n(T * (H // 2) + H).to(dtype).as_strided((T, H), (H // 2, 1))


@pytest.mark.parametrize("which", ["y", "residual", "gate", "gz", "gh"])
@pytest.mark.parametrize("kind", ["broadcast", "overlapping"])
@pytest.mark.parametrize("T,H,dtype", [(37, 640, BF16), (400, 512, F32), (9, 333, F16)])
def test_norm_rows_that_share_storage(which, kind, T, H, dtype):
    """A row broadcast over the tokens, or rows that overlap, give what their copies give, in both directions."""
    n = gen(1)
    c = {x: n(T, H).to(dtype) for x in ("y", "residual", "gate", "gz", "gh")}
    c[which] = n(H).to(dtype).expand(T, H) if kind == "broadcast" else overlapping(n, T, H, dtype)
    w_post, w_pre = 1 + 0.2 * n(H), 1 + 0.2 * n(H)

    def both(t):
        kw = dict(w_post=w_post, gate=t["gate"], scale=0.5, w_pre=w_pre)
        z, h, stats = nf4.norm_residual_fwd(t["y"], t["residual"], **kw)
        return (z, h, *nf4.norm_residual_bwd(t["gz"], t["gh"], t["y"], t["residual"], stats, **kw))

    for got, want in zip(both(c), both({k: t.contiguous() for k, t in c.items()})):
        assert torch.equal(got, want)
    if which in ("gz", "gh"):
        return
    # through autograd a broadcast input's gradient is the sum over the tokens
    leaves = {k: c[k].detach().clone() if k != which else (c[k][0].clone() if kind == "broadcast" else c[k].detach().clone())
              for k in ("y", "residual", "gate")}
    leaves = {k: t.requires_grad_() for k, t in leaves.items()}
    t = {k: x.expand(T, H) for k, x in leaves.items()}
    z, h = nf4.nf4_norm_residual(t["y"], t["residual"], w_post=w_post, gate=t["gate"], scale=0.5, w_pre=w_pre)
    torch.autograd.backward([z, h], [c["gz"], c["gh"]])
    want, mag = ref.norm_residual(c["y"], c["residual"], w_post, c["gate"], 0.5, w_pre, 1e-6, c["gz"], c["gh"])
    for name, key in (("y", "gy"), ("residual", "gr"), ("gate", "ggate")):
        bound = ref.norm_bound(want[key], mag[key], dtype, T, H, False)
        w = want[key]
        if leaves[name].dim() == 1:
            # the T rounded rows are added in fp32 and rounded once more
            w, bound = w.sum(0), bound.sum(0) + 1.1 * ref.UNIT[dtype] * w.sum(0).abs() + T * 2.0 ** -23 * w.abs().sum(0) + ref.TINY[dtype]
        assert ((leaves[name].grad.double() - w).abs() <= bound).all(), name


def test_norm_plain_norm_of_a_broadcast_row():
    """y alone with w_pre, broadcast: z is y itself, h every row the same."""
    n = gen(2)
    row, w = n(256).to(BF16), 1 + 0.2 * n(256)
    y = row.expand(50, 256)
    z, h, _ = nf4.norm_residual_fwd(y, w_pre=w)
    one = nf4.norm_residual_fwd(row[None], w_pre=w)[1]
    assert z is y and torch.equal(h, one.expand(50, 256))
