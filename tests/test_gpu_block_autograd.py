"""Second derivatives of the training-block operators."""
import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4

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
