"""Second derivatives of the training-block operators, and the device that their calls run on."""
import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from bit_nf4_quantized_linear_gb300 import block_ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


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


@pytest.mark.parametrize("op", ["attention", "norm"])
def test_second_derivatives_are_refused(op):
    """The gradients are no functions of autograd's: with create_graph they are right, and a derivative of them is an
    error, not a silently missing part, whether or not the incoming gradient asks for one itself."""
    n = gen(8)
    if op == "attention":
        leaves = [n(20, 2, 64).to(BF16).requires_grad_() for _ in range(3)]
        out = nf4.nf4_attention(*leaves)
    else:
        leaves = [n(20, 64).to(BF16).requires_grad_(), (1 + 0.1 * n(64)).requires_grad_()]
        out = nf4.nf4_norm_residual(leaves[0], w_pre=leaves[1])[1]
    for seed in (torch.ones_like(out), torch.ones_like(out).requires_grad_()):
        plain = torch.autograd.grad(out, leaves, seed, retain_graph=True)
        grads = torch.autograd.grad(out, leaves, seed, create_graph=True)
        for a, b in zip(plain, grads):
            assert torch.equal(a, b) and b.requires_grad
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(sum(g.float().square().sum() for g in grads), leaves)


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    """With another device current, every call makes its tensors' device current around its launches and queries."""
    entered = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *a):
            entered.pop()

    seen = []
    library, workspace = block_ops._fn, block_ops._workspace

    def fn(name):
        def call(*args):
            seen.append((name, list(entered)))
            return library(name)(*args)
        return call

    monkeypatch.setattr(block_ops, "_fn", fn)
    monkeypatch.setattr(block_ops, "_workspace", lambda *a: (seen.append(("workspace", list(entered))), workspace(*a))[1])
    monkeypatch.setattr(block_ops, "_guard", Guard)
    n = gen(9)
    q = n(20, 2, 64).to(BF16)
    y, w = n(20, 64).to(BF16), torch.ones(64, device=DEV)
    p, g = torch.ones(300, device=DEV), torch.ones(300, device=DEV)
    for current in (0, 1):
        monkeypatch.setattr(block_ops, "_current_device", lambda: current)
        seen.clear()
        o, lse = block_ops.attention_fwd(q, q, q)
        block_ops.attention_bwd(q, q, q, q, o, lse)
        _, _, stats = block_ops.norm_residual_fwd(y, w_pre=w)
        block_ops.norm_residual_bwd(y, y, y, None, stats, w_pre=w)
        state = block_ops.adamw_state([p])
        block_ops.adamw_step([p], [g], state, lr=0.1)
        block_ops.adamw_state_values(state)
        assert len(seen) == 8
        for name, devices in seen:
            assert devices == ([torch.device(DEV)] if current else []), name
