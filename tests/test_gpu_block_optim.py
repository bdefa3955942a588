"""NF4AdamW beside torch.optim.AdamW, and what a program does to an optimiser between steps: late gradients, saved
and loaded states, copies, graphs."""
import copy
import io

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


def params(dtype=torch.float32):
    n = gen(0)
    return [torch.nn.Parameter(n(s).to(dtype)) for s in (300, 1000, 5, 77)]


def test_steps_of_a_parameter_count_its_own_gradients():
    """Parameters whose first gradient comes late, or that miss some, step as torch.optim.AdamW's do."""
    n = gen(1)
    a, b = params(), params()
    kw = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
    own, other = nf4.NF4AdamW(a, state_bits=32, **kw), torch.optim.AdamW(b, **kw)
    for step in range(12):
        for i, (p, q) in enumerate(zip(a, b)):
            present = (True, step >= 7, step % 3 == 0, step != 4)[i]
            p.grad = n(p.numel()) if present else None
            q.grad = None if p.grad is None else p.grad.clone()
        own.step()
        other.step()
        for p, q in zip(a, b):
            # each step's error is a few units of its size (lr) and one rounding of the parameter, at most 12 times over
            assert ((p - q).abs() <= 12 * (2.0 ** -23 * q.abs() + 32 * 2.0 ** -24 * kw["lr"])).all(), step


@pytest.mark.parametrize("bits", [8, 32])
def test_step_counts_are_saved(bits):
    """A state saved while the counts of its parameters differ continues bit for bit, and a record without the counts
    (saved before there were any) loads with one count for all."""
    n = gen(2)
    a = params()
    opt = nf4.NF4AdamW(a, lr=1e-2, state_bits=bits)
    grads = [[n(p.numel()) for p in a] for _ in range(6)]

    def step(ps, o, t):
        for i, (p, g) in enumerate(zip(ps, grads[t])):
            p.grad = None if i == 1 and t < 3 else g
        o.step()

    for t in range(4):
        step(a, opt, t)
    saved = io.BytesIO()
    torch.save(opt.state_dict(), saved)
    saved.seek(0)
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    second = nf4.NF4AdamW(b, lr=1e-2, state_bits=bits)
    second.load_state_dict(torch.load(saved))
    for t in (4, 5):
        step(a, opt, t)
        step(b, second, t)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    old = opt.state_dict()
    old["group_state"] = {k: {x: r[x] for x in ("bits", "step", "buffers")} for k, r in old["group_state"].items()}
    third = nf4.NF4AdamW(b, lr=1e-2, state_bits=bits)
    third.load_state_dict(old)
    step(b, third, 0)


def test_raw_step_counts():
    """adamw_step numbers a call's step for all tensors, or each tensor's by its own gradients."""
    n = gen(3)
    g = [n(300), n(40)]
    hyper = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0)
    ps = [torch.zeros(300, device=DEV), torch.zeros(40, device=DEV)]
    state = nf4.adamw_state(ps, bits=32)
    for _ in range(4):
        nf4.adamw_step(ps, [g[0], None], state, per_tensor=True, **hyper)
    nf4.adamw_step(ps, g, state, per_tensor=True, **hyper)
    # the first step from zero moments goes lr along each gradient's sign
    assert (ps[1] + hyper["lr"] * g[1].sign()).abs().max() <= 1e-5 * hyper["lr"] + 2 * hyper["lr"] * 1e-8 / g[1].abs().min()
    shared = [torch.zeros(300, device=DEV), torch.zeros(40, device=DEV)]
    state = nf4.adamw_state(shared, bits=32)
    for _ in range(4):
        nf4.adamw_step(shared, [g[0], None], state, **hyper)
    nf4.adamw_step(shared, g, state, **hyper)
    assert state.step == 5 and torch.equal(shared[0], ps[0]) and not torch.equal(shared[1], ps[1])


def stepped(ps, **kw):
    opt = nf4.NF4AdamW(ps, **kw)
    n = gen(4)
    for p in opt.param_groups[0]["params"]:
        p.grad = n(*p.shape).to(p.dtype)
    opt.step()
    return opt


def test_a_saved_state_that_fits_no_parameters_is_refused():
    """Of parameters of another dtype, or of other shapes in buffers of the same size; the refusal changes nothing."""
    saved = stepped(params()).state_dict()
    other = stepped(params(BF16))
    before = copy.deepcopy(other.state_dict())
    with pytest.raises(ValueError, match="state"):
        other.load_state_dict(saved)
    after = other.state_dict()
    assert before["param_groups"] == after["param_groups"] and before["group_state"].keys() == after["group_state"].keys()
    for key, rec in before["group_state"].items():
        assert rec["step"] == after["group_state"][key]["step"]
        for x, y in zip(rec["buffers"], after["group_state"][key]["buffers"]):
            assert (x is None and y is None) or torch.equal(x, y)
    swapped = params()
    swapped = [swapped[i] for i in (3, 2, 1, 0)]  # 77, 5, 1000, 300: as many blocks in all
    with pytest.raises(ValueError, match="state"):
        nf4.NF4AdamW(swapped).load_state_dict(saved)


def test_a_group_that_never_stepped_loads_without_a_state():
    ps, qs = params(), params()
    opt = nf4.NF4AdamW([dict(params=ps[:2]), dict(params=ps[2:])])
    for p in ps[:2]:
        p.grad = torch.ones_like(p)
    opt.step()
    second = nf4.NF4AdamW([dict(params=qs[:2]), dict(params=qs[2:])])
    second.load_state_dict(opt.state_dict())
    assert list(second.group_state) == list(opt.group_state)
    for q in qs:
        q.grad = torch.ones_like(q)
    second.step()


def test_a_captured_step_is_refused():
    """The step's number is fixed when it is launched: a replayed graph would repeat one bias correction."""
    ps = params()
    opt = nf4.NF4AdamW(ps)
    for p in ps:
        p.grad = torch.ones_like(p)
    opt.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ps[0].grad.mul_(1)  # a graph with something in it
        with pytest.raises(RuntimeError, match="captur"):
            opt.step()
    opt.step()
    assert [st.step for st in opt.group_state.values()] == [2]


def test_a_step_moves_the_version_counters_of_what_it_writes():
    """A backward through a graph kept from before the step is an error, as with torch's optimisers."""
    ps = params()
    opt = nf4.NF4AdamW(ps)
    loss = sum(p.square().sum() for p in ps)
    loss.backward(retain_graph=True)
    ps[2].grad = None
    seen = [p._version for p in ps]
    opt.step()
    assert [p._version > s for p, s in zip(ps, seen)] == [True, True, False, True]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    x = torch.zeros(9, 2, 64, dtype=BF16, device=DEV)
    out = torch.zeros_like(x)
    before = out._version
    nf4.attention_fwd(x, x, x, out=out)
    assert out._version > before
    with torch.inference_mode():
        p, g = torch.ones(10, device=DEV), torch.ones(10, device=DEV)
        nf4.adamw_step([p], [g], nf4.adamw_state([p]), lr=0.1)
        assert (p < 1).all()


@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_copies_of_an_optimiser_step_like_it(how):
    n = gen(6)
    ps = params()
    opt = nf4.NF4AdamW(ps, lr=1e-2)
    grads = [[n(p.numel()) for p in ps] for _ in range(3)]

    def step(o, t):
        for p, g in zip(o.param_groups[0]["params"], grads[t]):
            p.grad = g.clone()
        o.step()

    step(opt, 0)
    step(opt, 1)
    if how == "deepcopy":
        twin = copy.deepcopy(opt)
    else:
        held = io.BytesIO()
        torch.save(opt, held)
        held.seek(0)
        twin = torch.load(held, weights_only=False)
    step(opt, 2)
    step(twin, 2)
    for p, q in zip(ps, twin.param_groups[0]["params"]):
        assert p is not q and torch.equal(p, q)
