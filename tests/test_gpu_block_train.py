"""The training-block operators as a program uses them: autograd, the optimiser with its saved state, and the
example that runs them together."""
import os
import sys

import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from tests import block_refs as ref

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


def test_attention_autograd_matches_the_calls():
    n = gen(0)
    fused = n(120, 8, 64).to(BF16).requires_grad_()
    q, k, v = fused.split([4, 2, 2], 1)
    cu = torch.tensor([0, 50, 120], dtype=torch.int32, device=DEV)
    o = nf4.nf4_attention(q, k, v, cu)
    go = n(120, 4, 64).to(BF16)
    o.backward(go)
    with torch.no_grad():
        o2, lse = nf4.attention_fwd(q, k, v, cu)
        want = torch.cat(nf4.attention_bwd(go, q, k, v, o2, lse, cu), 1)
    assert torch.equal(o, o2) and torch.equal(fused.grad, want)


def test_attention_autograd_with_an_expanded_gradient():
    n = gen(1)
    q, k, v = (n(40, 2, 64).to(BF16).requires_grad_() for _ in range(3))
    nf4.nf4_attention(q, k, v).sum().backward()  # the gradient is one value with strides 0
    with torch.no_grad():
        o, lse = nf4.attention_fwd(q, k, v)
        want = nf4.attention_bwd(torch.ones_like(o), q, k, v, o, lse)
    for t, w in zip((q, k, v), want):
        assert torch.equal(t.grad, w)


@pytest.mark.parametrize("use", ["z", "h", "both"])
def test_norm_autograd_matches_the_definition(use):
    n = gen(2)
    t = dict(y=n(30, 256).to(BF16), residual=n(30, 256).to(BF16), w_post=1 + 0.1 * n(256), gate=n(256), w_pre=1 + 0.1 * n(256))
    leaves = {k: x.clone().requires_grad_() for k, x in t.items()}
    z, h = nf4.nf4_norm_residual(leaves["y"], leaves["residual"], w_post=leaves["w_post"], gate=leaves["gate"], scale=0.5,
                                 w_pre=leaves["w_pre"])
    gz, gh = n(30, 256).to(BF16), n(30, 256).to(BF16)
    gz, gh = (gz if use != "h" else None), (gh if use != "z" else None)
    torch.autograd.backward([x for x, g in ((z, gz), (h, gh)) if g is not None], [g for g in (gz, gh) if g is not None])
    want, mag = ref.norm_residual(t["y"], t["residual"], t["w_post"], t["gate"], 0.5, t["w_pre"], 1e-6, gz, gh)
    for name, key in (("y", "gy"), ("residual", "gr"), ("w_post", "gw_post"), ("gate", "ggate"), ("w_pre", "gw_pre")):
        g = leaves[name].grad
        bound = ref.norm_bound(want[key], mag[key], BF16, 30, 256, g.dim() == 1)
        assert ((g.double() - want[key]).abs() <= bound).all(), name


def test_norm_autograd_plain_norm_and_frozen_parts():
    n = gen(3)
    x = n(9, 128).to(BF16).requires_grad_()
    w = torch.ones(128, device=DEV)
    z, h = nf4.nf4_norm_residual(x, w_pre=w)
    assert torch.equal(z, x)
    (z.float().sum() + h.float().sum()).backward()
    _, _, st = nf4.norm_residual_fwd(x.detach(), w_pre=w)
    ones = torch.ones(9, 128, dtype=BF16, device=DEV)
    assert torch.equal(x.grad, nf4.norm_residual_bwd(ones, ones, x.detach(), None, st, w_pre=w)[0])
    assert w.grad is None


def test_checkpointed_recompute_gives_the_same_gradients():
    from torch.utils.checkpoint import checkpoint
    n = gen(4)
    base = [n(100, 4, 64).to(BF16), n(100, 2, 64).to(BF16), n(100, 2, 64).to(BF16)]

    def run(wrap):
        leaves = [t.clone().requires_grad_() for t in base]
        out = checkpoint(nf4.nf4_attention, *leaves, use_reentrant=False) if wrap else nf4.nf4_attention(*leaves)
        out.float().square().sum().backward()
        return [t.grad for t in leaves]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [8, 32])
def test_optimiser_follows_its_step_and_its_saved_state(bits):
    """NF4AdamW steps as adamw_step does, over mixed dtypes and groups; a state saved and loaded continues bit for bit."""
    n = gen(5)

    def params():
        g = gen(6)
        return [torch.nn.Parameter(g(300, 7)), torch.nn.Parameter(g(1000).to(BF16)), torch.nn.Parameter(g(5, 5).to(BF16))]

    def make(ps):
        return nf4.NF4AdamW([dict(params=ps[:2], lr=1e-2), dict(params=ps[2:], weight_decay=0.1)], lr=1e-3, state_bits=bits)

    grads = [[n(300, 7), n(1000).to(BF16), n(5, 5).to(BF16)] for _ in range(4)]
    a, b = params(), params()
    opt = make(a)

    def step(ps, o, gs):
        for p, g in zip(ps, gs):
            p.grad = g.clone()
        o.step()

    for gs in grads[:2]:
        step(a, opt, gs)
    flat = [p.detach() for p in params()]
    states = [nf4.adamw_state([p], bits=bits) for p in flat]
    for gs in grads[:2]:
        for p, g, st, hyper in zip(flat, gs, states, ((1e-2, 0.01), (1e-2, 0.01), (1e-3, 0.1))):
            nf4.adamw_step([p], [g], st, lr=hyper[0], weight_decay=hyper[1])
    for p, q in zip(a, flat):
        assert torch.equal(p.detach(), q)
    with torch.no_grad():
        for p, q in zip(b, a):
            p.copy_(q)
    second = make(b)
    second.load_state_dict(opt.state_dict())
    for gs in grads[2:]:
        step(a, opt, gs)
        step(b, second, gs)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert [st.step for st in second.group_state.values()] == [4, 4, 4]
    other = nf4.NF4AdamW(params(), state_bits=40 - bits)
    with pytest.raises(ValueError):
        other.load_state_dict(opt.state_dict())


def test_optimiser_skips_parameters_without_gradients():
    ps = [torch.nn.Parameter(torch.ones(10, device=DEV)) for _ in range(2)]
    opt = nf4.NF4AdamW(ps, lr=0.1)
    opt.step()
    ps[0].grad = torch.ones(10, device=DEV)
    opt.step()
    assert (ps[0] < 1).all() and (ps[1] == 1).all()


def test_example_learns():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_block
    losses = train_block.train(steps=40, tokens=512, hidden=512)
    assert losses[-1] < 0.5 * losses[0]


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, torch.float16), (40, BF16), (37, BF16)])
def test_attention_rest_of_the_output(D, dtype):
    """o plus its rest is the unrounded output (to the rest's own rounding); a forward that no gradient follows makes none,
    and a backward without it stays within the bounds that count o's rounding."""
    n = gen(7)
    q, k, v, go = (n(150, 2, D).to(dtype) for _ in range(4))
    o, lse = nf4.attention_fwd(q, k, v)
    want, mag = ref.attention(q, k, v, [0, 150], D ** -0.5, go)
    u = ref.UNIT[dtype]
    # the probabilities are rounded once (u of their products), o + rest to u * u
    bound = (1.1 * u + 2.0 ** -12) * mag["o"] + 1.1 * u * u * want["o"].abs() + ref.TINY[dtype]
    assert ((o.double() + lse.o_rest.double() - want["o"]).abs() <= bound).all()
    o2, lse2 = nf4.attention_fwd(q, k, v, for_backward=False)
    assert torch.equal(o, o2) and lse2.o_rest is None
    smax = D ** -0.5 * (q.double().norm(dim=2).max() * k.double().norm(dim=2).max()).item()
    for got, name in zip(nf4.attention_bwd(go, q, k, v, o2, lse2), ("gq", "gk", "gv")):
        assert ((got.double() - want[name]).abs() <= ref.attention_bound(name, want[name], mag[name], dtype, smax)).all()
    with pytest.raises(ValueError):
        nf4.attention_bwd(go, q, k, v, o2, lse2, o_rest=lse.o_rest[:, :1])
