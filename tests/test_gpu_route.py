"""The router on the GPU against its definition: choices and tables exactly, weights and gradients within error bounds
computed from the reference's own magnitudes."""
import math
import random

import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from tests import decode_refs as ref
from tests.block_refs import TINY, UNIT

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


def spread(x):
    """Distance of each finite logit from the row's largest, and its size: what an exponential's argument loses."""
    y = x.double().masked_fill(x == -math.inf, 0.0)
    return (y.amax(1) - y.amin(1)).abs() + y.abs().amax(1)


def weight_bound(x, w):
    """A dozen fp32 operations, a sum of E terms in runs of E / 32 and a tree, and exponentials of arguments up to the
    spread, each rounded once."""
    return w.abs() * ((96 + 4 * spread(x)) * 2.0 ** -24)[:, None] + 1e-37


def check(x, k, live=None, grads=True, **how):
    T, E = x.shape
    kind, renorm, scale = how.get("score", "softmax"), how.get("renormalise", False), how.get("scale", 1.0)
    groups = how.get("groups", 1)
    r = nf4.route_experts(x, k, live=live, **how)
    on = torch.ones(T, dtype=torch.bool, device=DEV) if live is None else live.bool()
    want = ref.choose(x, k, kind, how.get("bias"), groups, how.get("top_groups") or groups, how.get("group_top", 1))
    assert r.experts.dtype == torch.int32 and torch.equal(r.experts, want.int().masked_fill(~on[:, None], -1))
    xd = x.double().requires_grad_()
    w = ref.weights(xd, want, kind, renorm, scale)
    wm = w.detach() * on[:, None]
    assert r.weights.dtype == F32 and ((r.weights.double() - wm).abs() <= weight_bound(x, wm)).all()
    for got, tab in zip((r.offsets, r.row_token, r.token_rows, r.row_weight), ref.tables(r.experts, r.weights, E)):
        assert torch.equal(got, tab)
    bare = nf4.route_experts(x, k, live=live, tables=False, **how)
    assert torch.equal(bare.experts, r.experts) and torch.equal(bare.weights, r.weights) and bare.offsets is None
    if not grads:
        return r
    n = gen(T + E + k)
    gw, gr = n(T, k), n(T * k)
    used = torch.where(r.token_rows >= 0, gr[r.token_rows.clamp(min=0).long()], 0.0)
    bwd = dict(score=kind, renormalise=renorm, scale=scale)
    for a, b in ((gw, None), (None, gr), (gw, gr)):
        g = nf4.route_experts_bwd(x, r, grad_weights=a, grad_row_weight=b, **bwd)
        up = ((0 if a is None else a.double()) + (0 if b is None else used.double())) * on[:, None]
        wg, = torch.autograd.grad((w * up).sum(), xd, retain_graph=True)
        wg = wg.nan_to_num(nan=0.0)
        # each term is scale p (g - sum g p), p the share of the term's expert
        p = (ref.scores(x.double(), kind).nan_to_num(nan=0.0) if not renorm else torch.zeros_like(wg).scatter_(1, want, w.detach() / scale))
        full = torch.zeros_like(wg).scatter_(1, want, up.abs())
        mag = abs(scale) * p * (full + (up.abs() * (w.detach() / scale).abs()).sum(1, keepdim=True))
        # p g - p sum g p cancels where p is 1: the error is relative to the magnitudes
        bound = 1.02 * UNIT[x.dtype] * wg.abs() + ((256 + 8 * spread(x)) * 2.0 ** -24)[:, None] * mag + TINY[x.dtype] + 1e-37
        assert g.dtype == x.dtype and torch.isfinite(g).all()
        over = ((g.double() - wg).abs() / bound).max().item()
        assert over <= 1, f"gradient: {over:.3g} of its bound"
        assert (g[~on] == 0).all()
    return r


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (5, 3), (8, 8), (32, 4), (33, 2), (60, 4), (64, 8), (65, 6), (128, 2), (200, 10), (256, 8),
                                 (257, 1), (512, 32), (40, 32)])
@pytest.mark.parametrize("T", [1, 32, 33, 300])
def test_route_sizes(E, k, T):
    rng = random.Random(E * 1000 + T)
    for dtype in (F32, BF16, F16):
        x = (1.5 * gen(T + E)(T, E)).to(dtype)
        check(x, k, score=rng.choice(["softmax", "sigmoid"]), renormalise=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
              bias=rng.choice([None, 0.1 * gen(3)(E)]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_forms(score, renormalise, biased):
    for T in (7, 2000):
        x = 2 * gen(T)(T, 64)
        check(x, 6, score=score, renormalise=renormalise, scale=1.7, bias=0.2 * gen(1)(64) if biased else None)


@pytest.mark.parametrize("E,groups,top_groups,k", [(16, 4, 2, 3), (64, 8, 3, 8), (60, 5, 1, 4), (256, 8, 4, 8), (512, 32, 7, 10), (32, 32, 5, 5),
                                                   (96, 2, 2, 12)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, groups, top_groups, k, group_top, score):
    for biased in (False, True):
        x = 1.5 * gen(E + k)(700, E)
        check(x, k, score=score, groups=groups, top_groups=top_groups, group_top=group_top, renormalise=True,
              bias=0.1 * gen(2)(E) if biased else None)


def test_route_large_batch():
    x = gen(0)(20011, 64)
    check(x, 8, grads=True, score="sigmoid", bias=0.1 * gen(1)(64), renormalise=True)
    # more tokens than fit the counts' bytes, none of them, or all, with one expert
    x = gen(2)(40001, 48)
    x[:, 7] += 20
    x[:, 9] -= 20
    r = check(x, 2, grads=False)
    assert r.offsets[8] - r.offsets[7] == 40001 and r.offsets[10] == r.offsets[9]


@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(biased):
    """Few distinct logits, so that equal candidates lie on both sides of the border everywhere."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for E, groups in ((64, 1), (128, 8), (60, 4)):
        x = torch.randint(-2, 3, (500, E), generator=g, device=DEV).float()
        bias = torch.randint(0, 2, (E,), generator=g, device=DEV).float() / 4 if biased else None
        for score in ("softmax", "sigmoid"):
            for group_top in (1, 2) if groups > 1 else (1,):
                check(x, 5, score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2), group_top=group_top)
        check(torch.zeros(50, E, device=DEV, dtype=BF16), 4, bias=None if bias is None else torch.zeros(E, device=DEV))
    x = torch.tensor([[0.0, -0.0, 1.0, -0.0, 0.0]], device=DEV)
    assert nf4.route_experts(x, 3).experts.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_borders_nearer_than_fp32(score):
    """Candidates whose s + bias differ by less than fp32 can tell: the choice is still that of the definition."""
    T, E = 400, 32
    x = gen(4)(T, E)
    s = ref.scores(x.double(), score)
    # a bias that levels one row's scores to within a rounding; in that row every order is a near tie
    for row in range(0, T, 40):
        bias = (0.75 - s[row]).float()
        c = s[row] + bias.double()
        assert (c.max() - c.min()) < 1.3e-7
        for k in (1, 5, 16):
            check(x[row:row + 40], k, score=score, bias=bias, grads=False)
        check(x[row:row + 40], 3, score=score, bias=bias, groups=8, top_groups=3, group_top=2, grads=False)


def test_route_hidden_experts_and_empty_rows():
    """Experts of logit -inf come after all others and weigh nothing; a row of -inf alone has weights 0 and gradient 0."""
    x = gen(5)(300, 24)
    x[torch.rand(300, 24, device=DEV) < 0.7] = -math.inf
    x[17], x[18] = -math.inf, -math.inf
    x[18, 20] = 1.0
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            for kw in ({}, dict(bias=gen(6)(24)), dict(groups=6, top_groups=3, group_top=2), dict(groups=6, top_groups=3)):
                r = check(x, 5, score=score, renormalise=renormalise, **kw)
                assert (r.weights[17] == 0).all() and torch.isfinite(r.weights).all()
                assert (r.weights[torch.isinf(x.gather(1, r.experts.long()))] == 0).all()


@pytest.mark.parametrize("T", [5, 32, 400])
def test_route_padding(T):
    x = gen(T)(T, 16)
    for live in (torch.arange(T, device=DEV) < T - 3, torch.arange(T, device=DEV) % 3 != 0, torch.zeros(T, dtype=torch.bool, device=DEV),
                 (torch.arange(T, device=DEV) % 2).to(torch.uint8)):
        x2 = x.clone()
        x2[~live.bool()] = math.nan  # what padding holds is not read for anything
        r = check(x, 4, live=live)
        r2 = nf4.route_experts(x2, 4, live=live)
        for a, b in zip(r, r2):
            assert torch.equal(a, b)
        g = nf4.route_experts_bwd(x2, r2, grad_row_weight=torch.ones(T * 4, device=DEV))
        assert (g[~live.bool()] == 0).all() and torch.isfinite(g).all()


def test_route_nan_rows_stay_in_range():
    """A NaN logit makes its own row's weights NaN at most; the choice stays k distinct experts."""
    x = gen(7)(100, 48)
    clean = nf4.route_experts(x, 6)
    x[3, 5], x[4], x[5, 7] = math.nan, math.nan, math.inf
    for kw in ({}, dict(bias=gen(8)(48)), dict(groups=8, top_groups=4, group_top=2), dict(score="sigmoid", bias=gen(8)(48))):
        r = nf4.route_experts(x, 6, **kw)
        assert ((r.experts >= 0) & (r.experts < 48)).all() and (r.experts[:, 1:] > r.experts[:, :-1]).all()
        assert torch.equal(r.token_rows.flatten().sort().values, torch.arange(600, device=DEV, dtype=torch.int32))
        nf4.route_experts_bwd(x, r, grad_weights=torch.ones(100, 6, device=DEV))
    r = nf4.route_experts(x, 6)
    rest = torch.ones(100, dtype=torch.bool, device=DEV)
    rest[3:6] = False
    assert torch.equal(r.experts[rest], clean.experts[rest]) and torch.equal(r.weights[rest], clean.weights[rest])
    assert 5 in r.experts[3].tolist() and 7 in r.experts[5].tolist()


@pytest.mark.parametrize("E", [24, 200, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_extreme_biases(score, E):
    """Experts of an infinite bias come first, or last but for those of logit -inf; equal ones by the lower index."""
    x = gen(11)(120, E)
    x[torch.rand(120, E, device=DEV) < 0.2] = -math.inf
    some = torch.randperm(E, device=DEV)
    for high in (1, 4, 6, 12, E):
        for value in (math.inf, 3e38, 1e30):
            bias = gen(E + high)(E)
            bias[some[:high]] = value
            bias[some[-3:]] = -value
            for kw in ({}, dict(groups=4, top_groups=2), dict(groups=8, top_groups=3)):
                check(x, 5, score=score, bias=bias, grads=False, **kw)
            if value != 3e38:  # twice that is no fp32 number
                check(x, 5, score=score, bias=bias, groups=4, top_groups=2, group_top=2, grads=False)
    bias = gen(12)(E)
    bias[3] = math.nan
    for kw in ({}, dict(groups=4, top_groups=2, group_top=2)):
        r = nf4.route_experts(x, 5, score=score, bias=bias, **kw)
        assert ((r.experts >= 0) & (r.experts < E)).all() and (r.experts[:, 1:] > r.experts[:, :-1]).all()


def test_route_extreme_logits():
    """Sigmoid scores that leave fp32's range, and softmax rows with one giant: weights stay those of the definition."""
    x = torch.linspace(-300, 60, 37 * 20, device=DEV).view(20, 37)
    for score in ("softmax", "sigmoid"):
        check(x, 4, score=score, renormalise=True)
    x = gen(9)(30, 16)
    x[:, 3] += 200
    check(x, 4, renormalise=True)
    check(x, 4)
    check(x, 4, bias=10 * gen(1)(16), renormalise=True)


def test_route_layouts():
    wide = gen(10)(90, 100)
    check(wide[:, 10:57], 5)
    check(wide[:, 3:50].to(BF16)[::2], 5)
    row = gen(11)(1, 40)
    check(row.expand(50, 40), 3, grads=False)
    r = nf4.route_experts(wide[:0], 4)
    assert r.offsets.tolist() == [0] * 101 and r.experts.shape == (0, 4) and r.row_token.numel() == 0
    assert nf4.route_experts_bwd(wide[:0], r, grad_weights=torch.zeros(0, 4, device=DEV)).shape == (0, 100)


def test_route_gradient_against_differences():
    """Central differences of the weights themselves.  h = 2^-7: the remainder is h^2 / 6 of a third derivative (at most
    8 scale sum |g|), the weights' rounding 64 ULP of scale sum |g| over h."""
    T, E, k, h = 6, 12, 4, 2.0 ** -7
    x, gw = gen(12)(T, E), gen(13)(T, k)
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            how = dict(score=score, renormalise=renormalise, scale=1.5)
            r = nf4.route_experts(x, k, **how)
            # the border is away from the step
            border = x.sort(dim=1, descending=True).values
            assert (border[:, k - 1] - border[:, k] > 2 * h).all()
            g = nf4.route_experts_bwd(x, r, grad_weights=gw, **how)
            for e in range(E):
                up, down = x.clone(), x.clone()
                up[:, e] += h
                down[:, e] -= h
                a, b = (nf4.route_experts(y, k, **how) for y in (up, down))
                assert torch.equal(a.experts, r.experts) and torch.equal(b.experts, r.experts)
                diff = ((a.weights.double() - b.weights.double()) * gw.double()).sum(1) / (up[:, e].double() - down[:, e].double())
                size = 1.5 * gw.abs().sum(1).double()
                assert ((g[:, e].double() - diff).abs() <= size * (8 * h * h / 6 + 64 * 2.0 ** -24 / h)).all()


def test_route_repeats_bit_for_bit_on_streams_and_in_graphs():
    x = 1.5 * gen(14)(3000, 96)
    bias = 0.1 * gen(15)(96)

    def both(x):
        r = nf4.route_experts(x, 6, score="sigmoid", bias=bias, renormalise=True)
        return (*r, nf4.route_experts_bwd(x, r, grad_weights=r.weights, score="sigmoid", renormalise=True))

    first = both(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = [both(x) for _ in range(4)]
    here = [both(x) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for got in other + here:
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    for T in (3000, 20):
        y = x[:T].clone()
        both(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = both(y)
        for s in (1, 2):
            y.copy_(1.5 * gen(s)(T, 96))
            graph.replay()
            for a, b in zip(both(y), held):
                assert torch.equal(a, b)


def test_route_refusals():
    """Every argument that does not fit is refused with a message, before anything is launched."""
    x = gen(19)(10, 24)
    r = nf4.route_experts(x, 4)
    before = nf4.path_counters()["total"]

    def fwd(message, x=x, k=4, **kw):
        with pytest.raises(ValueError, match=message):
            nf4.route_experts(x, k, **kw)

    fwd("logits", x=x[0])
    fwd("logits", x=x[:, :0])
    fwd("logits", x=x.T.contiguous().T)
    fwd("fp32, bf16 or fp16", x=x.double())
    fwd("CUDA", x=x.cpu())
    fwd("score", score="relu")
    for kw in (dict(groups=0), dict(groups=5), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(group_top=3)):
        fwd("groups", **kw)
    fwd("experts of the", k=0)
    fwd("experts of the", k=25)
    fwd("experts of the", groups=6, top_groups=1, k=5)
    fwd("bias", bias=torch.zeros(23, device=DEV))
    fwd("bias", bias=torch.zeros(24, device=DEV, dtype=BF16))
    fwd("CUDA", bias=torch.zeros(24))
    fwd("live", live=torch.zeros(9, dtype=torch.bool, device=DEV))
    fwd("live", live=torch.zeros(10, device=DEV))
    for E, k, kw in ((513, 4, {}), (64, 33, {}), (64, 4, dict(groups=64))):
        with pytest.raises(nf4._lib.NF4Error, match="UNSUPPORTED_SHAPE"):
            nf4.route_experts(torch.zeros(2, E, device=DEV), k, **kw)

    def bwd(message, x=x, r=r, **kw):
        with pytest.raises(ValueError, match=message):
            nf4.route_experts_bwd(x, r, **kw)

    g = torch.zeros(10, 4, device=DEV)
    bwd("routes.experts", r=r._replace(experts=r.experts.long()), grad_weights=g)
    bwd("routes.experts", x=x[:5], grad_weights=g)
    bwd("grad_weights", grad_weights=g[:, :3])
    bwd("grad_weights", grad_weights=g.half())
    bwd("grad_row_weight", grad_row_weight=g)
    bwd("token_rows", r=r._replace(token_rows=None), grad_row_weight=g.flatten())
    bwd("score", grad_weights=g, score="none")
    bwd("CUDA", grad_weights=g.cpu())
    assert nf4.path_counters()["total"] == before


def test_route_autograd():
    """Through nf4_route: gradients by weight and by row, none asked for, second derivatives refused."""
    x = gen(16)(70, 24).requires_grad_()
    r = nf4.nf4_route(x, 4, renormalise=True, scale=2.0)
    n = gen(17)
    gw, gr = n(70, 4), n(280)
    g, = torch.autograd.grad((r.weights * gw).sum() + (r.row_weight * gr).sum(), x)
    assert torch.equal(g, nf4.route_experts_bwd(x.detach(), r, grad_weights=gw, grad_row_weight=gr, renormalise=True, scale=2.0))
    r = nf4.nf4_route(x, 4, score="sigmoid", tables=False)
    assert r.offsets is None
    g, = torch.autograd.grad(r.weights.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    assert not nf4.nf4_route(x.detach(), 4).weights.requires_grad
    assert not r.experts.requires_grad


def test_route_backward_in_a_graph():
    """Forward and backward captured together, as a training step is, and replayed on new logits."""
    x = gen(18)(64, 16).requires_grad_()

    def step():
        r = nf4.nf4_route(x, 2, renormalise=True)
        return torch.autograd.grad(r.weights.square().sum() + (r.row_weight ** 3).sum(), x)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step()
    for s in (1, 2):
        with torch.no_grad():
            x.copy_(gen(s)(64, 16))
        graph.replay()
        assert torch.equal(g, step())


@pytest.mark.parametrize("E", [130, 300, 512])
@pytest.mark.parametrize("spread_by", [0.3, 1.0, 5.0])
def test_route_borders_nearer_than_fp32_of_many_experts(E, spread_by):
    """Softmax scores whose sum is of many terms, levelled to within a rounding by the bias."""
    x = spread_by * gen(E)(60, E)
    s = ref.scores(x.double(), "softmax")
    for row in range(0, 60, 10):
        bias = (0.75 - s[row]).float()
        assert (s[row] + bias.double()).sub(0.75).abs().max() < 6.1e-8
        for k in (1, 7, 32):
            check(x[row:row + 10], k, bias=bias, grads=False)
        check(x[row:row + 10], 5, bias=bias, groups=10 if E % 10 == 0 else 8, top_groups=3, group_top=2, grads=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_hidden_experts_equal_those_of_an_infinite_bias(score):
    """A logit of -inf and a bias of -inf give the same c, -inf: behind all others, and by the index among each other."""
    x = gen(20)(1, 8)
    x[0, [1, 6]] = -math.inf
    bias = torch.zeros(8, device=DEV)
    bias[[0, 2, 7]] = -math.inf
    live = [3, 4, 5]
    for k in range(1, 9):
        r = check(x, k, score=score, bias=bias, grads=False)
        if k >= 3:
            assert r.experts[0].tolist() == sorted((live + [0, 1, 2, 6, 7])[:k])
    assert r.weights[0, 1] == 0 and r.weights[0, 6] == 0 and (r.weights[0, [0, 2, 7]] > 0).all()
