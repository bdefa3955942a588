"""The router and the paged cache together with the operators that they stand beside: a trained mixture-of-experts layer,
and a decoding step of a whole block, against plain torch over the same dequantised weights."""
import math

import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from tests.helpers import ELEM, REL_FRO

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


def near(got, want, what, stages):
    """Each stage of bf16 products is held to the products' own bounds, REL_FRO in all and ELEM by element."""
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), what
    assert (got - want).norm() <= stages * REL_FRO * want.norm(), (what, ((got - want).norm() / want.norm()).item())
    assert ((got - want).abs() <= stages * ELEM * (want.abs() + want.square().mean().sqrt())).all(), what


class Experts:
    """E experts of hidden H and intermediate I, quantised; and their dense values."""

    def __init__(self, E, H, I, seed):
        n = gen(seed)
        gate, up, down = 0.05 * n(E * I, H), 0.05 * n(E * I, H), 0.05 * n(E * H, I)
        self.E, self.I = E, I
        self.gate_up = nf4.quantize(nf4.interleave_gate_up(gate, up, E))
        self.down = nf4.quantize(down)
        gu = nf4.dequantize(self.gate_up).view(E, I // 64, 2, 64, H)
        self.dense = [gu[:, :, i].reshape(E, I, H).double() for i in range(2)] + [nf4.dequantize(self.down).view(E, H, I).double()]

    def layer(self, x, r):
        """The layer as nf4_route's documentation gives it."""
        h = nf4.nf4_grouped_swiglu(nf4.nf4_dispatch(x, r.token_rows), r.offsets, self.gate_up, self.E, r.row_weight)
        return nf4.nf4_combine(nf4.nf4_grouped(h, r.offsets, self.down, self.E), r.token_rows)

    def plain(self, x, experts, weights):
        """In float64, with the routes given; -1 for none."""
        gate, up, down = self.dense
        y = torch.zeros_like(x)
        for e in range(self.E):
            t, j = (experts == e).nonzero(as_tuple=True)
            if t.numel():
                h = torch.nn.functional.silu(x[t] @ gate[e].T) * (x[t] @ up[e].T) * weights[t, j][:, None]
                y = y.index_add(0, t, h @ down[e].T)
        return y


@pytest.mark.parametrize("T,pad", [(1, 0), (48, 0), (300, 37)])
@pytest.mark.parametrize("renormalise", [False, True])
def test_moe_layer_with_gradients(T, pad, renormalise):
    """Router, dispatch, grouped experts and combine: output and the gradients of activations and router weights."""
    E, H, I, k = 16, 256, 128, 4
    ex = Experts(E, H, I, T)
    n = gen(T + 1)
    x, wr = n(T, H).to(BF16).requires_grad_(), (0.1 * n(E, H)).requires_grad_()
    live = torch.arange(T, device=DEV) < T - pad
    gy = n(T, H).to(BF16) * live[:, None]
    r = nf4.nf4_route(x.float() @ wr.T, k, renormalise=renormalise, live=live)
    y = ex.layer(x, r)
    gx, gw = torch.autograd.grad(y, (x, wr), gy)
    xd, wd = x.detach().double().requires_grad_(), wr.detach().double().requires_grad_()
    logits = xd @ wd.T
    held = r.experts.clamp(min=0).long()
    w = torch.softmax(logits, 1).gather(1, held)
    w = (w / w.sum(1, keepdim=True) if renormalise else w) * live[:, None]
    want = ex.plain(xd, r.experts, w)
    wx, ww = torch.autograd.grad(want, (xd, wd), gy.double())
    assert (y[~live] == 0).all() and (gx[~live] == 0).all()
    near(y, want, "y", 3)
    near(gx, wx, "gx", 5)
    near(gw, ww, "gw", 5)


def test_moe_route_tables_are_those_of_route_rows():
    x = gen(3)(130, 32)
    r = nf4.route_experts(x, 4)
    assert torch.equal(r.token_rows, nf4.route_rows(r.row_token, 130, 4))


def test_decoding_steps_of_a_block():
    """A prompt through the prompt attention with its keys appended, then steps of one token for three sequences and an idle
    one, captured in a graph: norm, fused q, k, v, append, paged attention, output projection, norm, experts."""
    H, heads, kv, D, E, I, k, B, page = 256, 8, 2, 64, 8, 128, 2, 4, 16
    n = gen(0)
    ex = Experts(E, H, I, 1)
    dense = [0.06 * n(r, H) for r in (heads * D, kv * D, kv * D)] + [0.05 * n(H, heads * D)]
    ws = [nf4.quantize(w) for w in dense]
    wd = [nf4.dequantize(w).double() for w in ws]
    gain1, gain2, wr = 1 + 0.1 * n(H), 1 + 0.1 * n(H), 0.1 * n(E, H)
    prompts, steps = [37, 0, 5, 64], 20
    lens = [m + (steps if m else 0) for m in prompts]
    need = [-(-m // page) for m in lens]
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    at = 0
    for i, m in enumerate(need):
        table[i, :m], at = ids[at:at + m], at + m
    table = table.to(DEV)
    kp, vp = (torch.full((sum(need), page, kv, D), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    lengths = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    live = lengths > 0

    def block(x, attend):
        stream, h = nf4.nf4_norm_residual(x, w_pre=gain1)
        q, key, val = (t.view(x.shape[0], -1, D) for t in nf4.linear_fwd_multi([h] * 3, ws[:3]))
        stream, h = nf4.nf4_norm_residual(nf4.linear_fwd(attend(q, key, val).flatten(1), ws[3]), stream, w_pre=gain2)
        return stream, h

    def experts(stream, h, live=None):
        r = nf4.route_experts(h.float() @ wr.T, k, renormalise=True, live=live)
        return stream + ex.layer(h, r), r

    # the prompts, packed
    cu = torch.tensor([sum(prompts[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
    xp = n(sum(prompts), H).to(BF16)
    kept = {}

    def attend_prompt(q, key, val):
        nf4.paged_append(key, val, kp, vp, table, lengths, cu)
        return nf4.nf4_attention(q, key, val, cu)

    yp, _ = experts(*block(xp, attend_prompt))
    assert torch.isfinite(yp).all()

    x = torch.zeros(B, H, dtype=BF16, device=DEV)

    def attend_token(q, key, val):
        nf4.paged_append(key, val, kp, vp, table, lengths)
        kept["q"] = q
        return nf4.paged_attention(q, kp, vp, table, lengths)[0]

    def step():
        stream, h = block(x, attend_token)
        y, r = experts(stream, h, live)
        return y, r

    lengths += live.int()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, r = step()
    lengths -= live.int()

    history = [xp[cu[i]:cu[i + 1]].double() for i in range(B)]

    def norm(t, gain):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * gain.double()

    for s in range(steps):
        lengths += live.int()
        x.copy_(gen(100 + s)(B, H))
        graph.replay()
        for i in range(B):
            if not live[i]:
                continue
            history[i] = torch.cat([history[i], x[i:i + 1].double()])
            if s % 7:
                continue
            h = norm(history[i], gain1)
            q, key, val = (h @ w.T for w in wd[:3])
            q, key, val = q[-1].view(heads, D), *(t.view(-1, kv, D).repeat_interleave(heads // kv, 1) for t in (key, val))
            p = torch.softmax(torch.einsum("hd,lhd->hl", q, key) / math.sqrt(D), 1)
            stream = x[i].double() + torch.einsum("hl,lhd->hd", p, val).flatten() @ wd[3].T
            want = stream + ex.plain(norm(stream, gain2)[None], r.experts[i:i + 1], r.weights[i:i + 1].double())[0]
            near(y[i], want, f"step {s}, sequence {i}", 4)
        assert torch.equal(r.experts[1], torch.full_like(r.experts[1], -1)) and torch.isfinite(y).all()
    assert lengths.tolist() == lens


def test_dispatch_refuses_tables_that_do_not_fit():
    """Fewer or more tokens than the table, another type, layout or device: refused before anything is launched."""
    x = gen(8)(6, 64).to(BF16)
    t = nf4.route_experts(gen(9)(6, 8), 2).token_rows
    before = nf4.path_counters()["total"]
    for f in (lambda x, t: nf4.nf4_dispatch(x, t), lambda x, t: nf4.moe_combine_bwd(x, t, t.numel())):
        for bad, message in ((x[:5], "6 tokens for 5 rows"), (x[:0], "6 tokens for 0 rows"), (torch.cat([x, x]), "6 tokens for 12 rows"),
                             (x.half(), "bf16"), (x[0], "bf16"), (x.cpu(), "CUDA")):
            with pytest.raises(ValueError, match=message):
                f(bad, t)
        for bad, message in ((t.long(), "int32"), (t.T.contiguous().T, "contiguous"), (t.flatten(), "int32"), (t.cpu(), "CUDA")):
            with pytest.raises(ValueError, match=message):
                f(x, bad)
    assert nf4.path_counters()["total"] == before
    rows = nf4.nf4_dispatch(x, t)
    assert torch.equal(rows[t.long()], x[:, None].expand(6, 2, 64))


def test_dispatch_and_combine_second_derivatives():
    """A penalty on the gradient of a squared path through dispatch and combine, on the kernels.  The values are small whole
    numbers, so that every sum is exact in bf16."""
    T, k, H = 9, 2, 64
    t = nf4.route_experts(gen(10)(T, 6), k, live=torch.arange(T, device=DEV) < 7).token_rows
    x = torch.randint(-2, 3, (T, H), generator=torch.Generator().manual_seed(1)).to(DEV, BF16).requires_grad_()
    y = nf4.nf4_combine(nf4.nf4_dispatch(x, t).square(), t)  # k x^2 of the live tokens
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    g2, = torch.autograd.grad(g.square().sum(), x)  # of (2 k x)^2
    live = (t[:, :1] >= 0)
    assert torch.equal(g, 2 * k * x.detach() * live) and torch.equal(g2, 8 * k * k * x.detach() * live)


@pytest.mark.parametrize("counts,pad", [((0, 0, 0), 3), ((0, 0, 0), 300), ((1, 0, 0), 1), ((5, 40, 0), 7), ((0, 200, 133), 260)])
@pytest.mark.parametrize("bits", [4, 8])
def test_rows_of_no_expert_are_zero_in_new_tensors(counts, pad, bits):
    """Rows behind the last expert's, in memory that held NaN: zeros in what the calls return, left as they were in `out`."""
    E, N_e, K = 3, 384, 256
    n = gen(sum(counts) + pad)
    wt = 0.05 * n(E * N_e, K)
    w = nf4.quantize(wt, quant_type="int8" if bits == 8 else "nf4")
    used = sum(counts)
    T = used + pad
    offsets = torch.tensor([sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device=DEV)
    x, gy, gh = n(T, K).to(BF16), n(T, N_e).to(BF16), n(T, N_e // 2).to(BF16)
    scale = torch.rand(T, device=DEV)

    def dirty(*shapes):
        held = [torch.full(s, math.nan, dtype=dt, device=DEV) for s, dt in shapes]
        del held

    calls = {"fwd": (N_e, lambda **kw: nf4.grouped_fwd(x, offsets, w, E, **kw)),
             "scaled": (N_e, lambda **kw: nf4.grouped_fwd(x, offsets, w, E, row_scale=scale, **kw)),
             "swiglu": (N_e // 2, lambda **kw: nf4.grouped_fwd(x, offsets, w, E, row_scale=scale, swiglu=True, **kw)),
             "dgrad": (K, lambda **kw: nf4.grouped_dgrad(gy, offsets, w, E, **kw))}
    for name, (width, call) in calls.items():
        held = torch.full((T, width), 7.0, dtype=BF16, device=DEV)
        call(out=held)
        assert (held[used:] == 7).all(), name
        dirty(((T, width), BF16))
        y = call()
        assert torch.equal(y[:used], held[:used]) and (y[used:] == 0).all(), name
    if bits == 4:
        dirty(((T, K), BF16), ((T,), torch.float32))
        gx, gs = nf4.grouped_swiglu_bwd(x, offsets, w, E, gh, row_scale=scale, need_row_scale_grad=True)
        assert torch.isfinite(gx).all() and (gx[used:] == 0).all() and (gs[used:] == 0).all()


def test_an_adapter_between_dispatch_and_combine_with_padding():
    """A trained low-rank path beside the frozen experts, over all rows: its weights' gradients see no row of padding."""
    E, H, I, k, T, pad = 8, 256, 128, 2, 60, 23
    ex = Experts(E, H, I, 5)
    n = gen(6)
    x, wr = n(T, H).to(BF16), 0.1 * n(E, H)
    live = torch.arange(T, device=DEV) < T - pad
    r = nf4.nf4_route(x.float() @ wr.T, k, live=live)
    down, up = (0.05 * n(I, 4)).requires_grad_(), (0.05 * n(4, H)).requires_grad_()
    for shape in ((T * k, I), (T * k, H)):
        held = torch.full(shape, math.nan, dtype=BF16, device=DEV)
        del held
    h = nf4.nf4_grouped_swiglu(nf4.nf4_dispatch(x, r.token_rows), r.offsets, ex.gate_up, E, r.row_weight)
    y = nf4.nf4_combine(nf4.nf4_grouped(h, r.offsets, ex.down, E) + (h.float() @ down @ up).to(BF16), r.token_rows)
    gd, gu = torch.autograd.grad(y.float().sum(), (down, up))
    assert torch.isfinite(gd).all() and torch.isfinite(gu).all() and torch.isfinite(y).all() and (y[~live] == 0).all()


@pytest.mark.parametrize("T,pad", [(0, 0), (5, 5), (1, 1)])
def test_moe_layer_of_no_tokens(T, pad):
    """No tokens, or none that is live: an output and gradients of zeros, from an expanded gradient as sum() gives it."""
    ex = Experts(8, 256, 128, 1)
    n = gen(11)
    x, wr = n(T, 256).to(BF16).requires_grad_(), n(8, 256).requires_grad_()
    r = nf4.nf4_route(x.float() @ wr.T, 2, live=torch.arange(T, device=DEV) < T - pad)
    y = ex.layer(x, r)
    for total in (y.sum(), y.float().sum()):
        gx, gw = torch.autograd.grad(total, (x, wr), retain_graph=True)
        assert y.shape == gx.shape == (T, 256) and (y == 0).all() and (gx == 0).all() and (gw == 0).all()
