"""The training-block operators on the GPU against their 64-bit definitions, at the sizes, layouts and values where
they can go wrong.  Every tolerance is an error bound computed from the reference's own magnitudes."""
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


def within(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert over <= 1.0, f"{what}: {over:.3g} of its error bound"


# ------------------------------------------------------------------ attention --

def qkv(T, Hq, Hk, D, dtype, seed=0):
    n = gen(seed)
    q, k = 1.3 * n(T, Hq, D), 1.3 * n(T, Hk, D)
    return [x.to(dtype) for x in (q, k, n(T, Hk, D) + 0.3, n(T, Hq, D))]


def check_attention(q, k, v, go, cu_list, cu, scale=None):
    o, lse = nf4.attention_fwd(q, k, v, cu, scale=scale)
    got = dict(zip(("gq", "gk", "gv"), nf4.attention_bwd(go, q, k, v, o, lse, cu, scale=scale)), o=o)
    sc = q.shape[2] ** -0.5 if scale is None else scale
    want, mag = ref.attention(q, k, v, cu_list, sc, go)
    smax = abs(sc) * (q.double().norm(dim=2).max() * k.double().norm(dim=2).max()).item()
    live = want["lse"] > -math.inf
    assert torch.equal(live, lse > -math.inf)
    assert ((lse.double() - want["lse"])[live].abs() <= (64 + 8 * smax) * 2.0 ** -24 * (1 + want["lse"][live].abs())).all()
    for name in got:
        assert got[name].dtype == q.dtype
        within(got[name], want[name], ref.attention_bound(name, want[name], mag[name], q.dtype, smax), name)


LENS = [[1], [2], [16], [63], [64], [65], [127], [128], [129], [255], [256], [257], [383], [600], [1, 1, 1], [0, 5, 0, 130, 1, 0],
        [128, 128], [100, 28, 256, 3], [31] * 9]


@pytest.mark.parametrize("lens", LENS, ids=lambda l: "-".join(map(str, l)))
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_attention_lengths(lens, D, dtype):
    q, k, v, go = qkv(sum(lens), 4, 2, D, dtype)
    b = ref.bounds_of(lens)
    check_attention(q, k, v, go, b, torch.tensor(b, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (8, 1), (6, 6), (10, 2), (8, 4)])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 112, 128, 136, 256, 37])
def test_attention_heads_and_widths(Hq, Hk, D):
    for dtype in (BF16, F16) if Hq == 3 else (BF16,):
        q, k, v, go = qkv(331, Hq, Hk, D, dtype, seed=D)
        check_attention(q, k, v, go, [0, 331], None)


@pytest.mark.parametrize("D", [5, 64, 128, 200])
def test_attention_fp32(D):
    q, k, v, go = qkv(150, 4, 2, D, F32, seed=D)
    check_attention(q, k, v, go, [0, 70, 150], torch.tensor([0, 70, 150], dtype=torch.int32, device=DEV), scale=0.1)


def test_attention_many_sequences():
    """More sequences than a warp has lanes, empty ones among them; many tiles."""
    lens = [(7 * i) % 23 for i in range(150)] + [300] + [0] * 40 + [1]
    q, k, v, go = qkv(sum(lens), 2, 1, 64, BF16)
    b = ref.bounds_of(lens)
    check_attention(q, k, v, go, b, torch.tensor(b, dtype=torch.int32, device=DEV))


def test_attention_long_sequence():
    q, k, v, go = qkv(2500, 4, 1, 128, BF16, seed=3)
    check_attention(q, k, v, go, [0, 2500], None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_rows_outside_the_sequences(dtype):
    """Rows before the first and after the last offset: zeros, whatever they hold, and no trace of them elsewhere."""
    T, cu_list = 400, [37, 120, 341]
    q, k, v, go = qkv(T, 4, 2, 64, dtype)
    cu = torch.tensor(cu_list, dtype=torch.int32, device=DEV)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    clean = (o, *nf4.attention_bwd(go, q, k, v, o, lse, cu))
    check_attention(q, k, v, go, cu_list, cu)
    for t in (q, k, v, go):
        t[:37], t[341:] = math.nan, math.inf
    o2, lse2 = nf4.attention_fwd(q, k, v, cu)
    for a, b in zip(clean, (o2, *nf4.attention_bwd(go, q, k, v, o2, lse2, cu))):
        assert torch.equal(a, b)
        assert (b[:37] == 0).all() and (b[341:] == 0).all()
    assert torch.equal(lse, lse2) and (lse2[:, :37] == -math.inf).all()


@pytest.mark.parametrize("at", [0, 5, 127, 128, 200, 299])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_nan_reaches_later_rows_only(at, bad):
    """A NaN or infinity in the key or value of token `at` of a sequence changes no earlier row and no other sequence."""
    lens = [90, 300, 50]
    b = ref.bounds_of(lens)
    cu = torch.tensor(b, dtype=torch.int32, device=DEV)
    q, k, v, go = qkv(sum(lens), 4, 2, 128, BF16)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    gq = nf4.attention_bwd(go, q, k, v, o, lse, cu)[0]
    t = b[1] + at
    fine = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    fine[t:b[2]] = False
    for x in (v, k):
        keep = x[t, 1, 3].clone()
        x[t, 1, 3] = bad
        o2, lse2 = nf4.attention_fwd(q, k, v, cu)
        gq2, gk2, gv2 = nf4.attention_bwd(go, q, k, v, o2, lse2, cu)
        assert torch.equal(o[fine], o2[fine])
        assert torch.equal(gq[fine], gq2[fine])
        assert torch.equal(o[:, :2], o2[:, :2])  # the heads of the other group
        other = torch.ones_like(fine)
        other[b[1]:b[2]] = False
        assert torch.isfinite(gk2[other].float()).all() and torch.isfinite(gv2[other].float()).all()
        if x is v:  # the value enters each later row with a positive weight
            want = torch.full_like(o2[t:b[2], 2:, 3].float(), bad)
            assert torch.equal(torch.nan_to_num(o2[t:b[2], 2:, 3].float(), nan=7.0), torch.nan_to_num(want, nan=7.0))
            assert torch.equal(o[:, 2:, 4:], o2[:, 2:, 4:])
        x[t, 1, 3] = keep


def test_attention_nan_gradient_rows_reach_earlier_keys_only():
    """A NaN in go of row i reaches the gradients of keys 0 .. i of its sequence and of no later key."""
    lens = [300, 60]
    b = ref.bounds_of(lens)
    cu = torch.tensor(b, dtype=torch.int32, device=DEV)
    q, k, v, go = qkv(sum(lens), 2, 2, 64, BF16)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    base = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    go[140, 1, 9] = math.nan
    gq, gk, gv = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    for got, want in ((gk, base[1]), (gv, base[2])):
        assert torch.equal(got[141:], want[141:]) and torch.equal(got[:, 0], want[:, 0])
    assert torch.isnan(gv[:141, 1, 9].float()).all()
    rows = torch.ones(360, dtype=torch.bool, device=DEV)
    rows[140] = False
    assert torch.equal(gq[rows], base[0][rows])


def test_attention_large_scores_and_equal_scores():
    """Scores of several hundred (a softmax that is nearly one-hot), and rows whose scores are all equal."""
    q, k, v, go = qkv(200, 2, 1, 64, BF16)
    check_attention(8 * q, 8 * k, v, go, [0, 200], None)
    check_attention(torch.zeros_like(q), k, v, go, [0, 200], None)
    check_attention(q, k, v, go, [0, 200], None, scale=-0.2)
    check_attention(q, k, v, go, [0, 200], None, scale=0.0)


def test_attention_strides():
    """Views of a fused projection output, head-major storage, a padded and a misaligned token stride."""
    T, Hq, Hk, D = 210, 4, 2, 64
    q, k, v, go = qkv(T, Hq, Hk, D, BF16)
    o, lse = nf4.attention_fwd(q, k, v)
    want = (o, *nf4.attention_bwd(go, q, k, v, o, lse))

    def same(q2, k2, v2, go2, exact=True):
        o2, lse2 = nf4.attention_fwd(q2, k2, v2)
        for a, b in zip(want, (o2, *nf4.attention_bwd(go2, q2, k2, v2, o2, lse2))):
            assert torch.equal(a, b) if exact else torch.allclose(a.float(), b.float(), atol=0.05, rtol=0.05)

    fused = torch.cat([q, k, v], 1).reshape(T, -1)
    same(*(x.view(T, -1, D) for x in fused.split([Hq * D, Hk * D, Hk * D], 1)), go)
    same(*(x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, go)))
    same(*(torch.cat([x, x], 2)[..., :D] for x in (q, k, v, go)))
    # a token stride of an odd number of elements takes the general kernels
    same(*(torch.cat([x.reshape(T, -1), torch.zeros(T, 3, dtype=BF16, device=DEV)], 1)[:, :x.shape[1] * D].view(T, -1, D)
           if False else torch.as_strided(torch.cat([x.reshape(T, -1), torch.zeros(T, 3, dtype=BF16, device=DEV)], 1),
                                          x.shape, (x.shape[1] * D + 3, D, 1)) for x in (q, k, v, go)), exact=False)


def test_attention_repeats_bit_for_bit_and_on_another_stream():
    q, k, v, go = qkv(700, 8, 2, 128, BF16)
    cu = torch.tensor([0, 333, 700], dtype=torch.int32, device=DEV)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    first = (o, lse, *nf4.attention_bwd(go, q, k, v, o, lse, cu))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = nf4.attention_fwd(q, k, v, cu)
        second = (o2, lse2, *nf4.attention_bwd(go, q, k, v, o2, lse2, cu))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_attention_graph_replay():
    """Captured in a CUDA graph, with the offsets changed between replays (they are read on the device)."""
    q, k, v, go = qkv(500, 4, 2, 64, BF16)
    cu = torch.tensor([0, 250, 500], dtype=torch.int32, device=DEV)

    def step():
        o, lse = nf4.attention_fwd(q, k, v, cu)
        return (o, lse, *nf4.attention_bwd(go, q, k, v, o, lse, cu))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for bounds in ([0, 250, 500], [0, 1, 480], [10, 400, 400]):
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_attention_gradient_against_differences():
    """The gradients of the library's own fp32 forward against central differences of it."""
    q, k, v, go = qkv(61, 4, 2, 16, F32)
    cu = torch.tensor([0, 20, 61], dtype=torch.int32, device=DEV)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    grads = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    n = gen(9)
    eps = 1e-2
    for i, g in enumerate(grads):
        d = n(*g.shape)
        val = []
        for s in (eps, -eps):
            args = [q, k, v]
            args[i] = args[i] + s * d
            val.append((nf4.attention_fwd(*args, cu)[0].double() * go.double()).sum().item())
        want, got = (val[0] - val[1]) / (2 * eps), (g.double() * d.double()).sum().item()
        # truncation is O(eps^2) of third derivatives of order one, the two values' rounding about 1e-7 of their size / eps
        assert abs(want - got) <= 5e-3 * (g.double() * d.double()).abs().sum().item() ** 0.5 + 2e-3 * abs(got)


def test_attention_bad_offsets_are_recorded():
    q, k, v, _ = qkv(100, 2, 1, 64, BF16)
    for bad in ([0, 200], [-5, 100], [60, 40]):
        o, _ = nf4.attention_fwd(q, k, v, torch.tensor(bad, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert nf4.device_status(clear=True) == 8


def test_attention_empty():
    q, k, v, go = qkv(0, 2, 1, 64, BF16)
    o, lse = nf4.attention_fwd(q, k, v)
    assert o.shape == q.shape and lse.shape == (2, 0)
    assert all(g.numel() == 0 for g in nf4.attention_bwd(go, q, k, v, o, lse))


def test_attention_refusals():
    q, k, v, go = qkv(10, 4, 2, 64, BF16)
    for args in ((q, k[:9], v), (q, k.half(), v), (q, k, v[:, :1]), (q[:, :3], k, v), (q[..., ::2], k[..., ::2], v[..., ::2]),
                 (q.double(), k.double(), v.double()), (q.cpu(), k.cpu(), v.cpu()), (q[0], k[0], v[0])):
        with pytest.raises(ValueError):
            nf4.attention_fwd(*args)
    for cu in (torch.tensor([0, 10], device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV),
               torch.tensor([0, 10], dtype=torch.int32)):
        with pytest.raises(ValueError):
            nf4.attention_fwd(q, k, v, cu)
    wide = torch.zeros(4, 1, 264, dtype=BF16, device=DEV)
    with pytest.raises(RuntimeError, match="NF4_ERR_UNSUPPORTED_SHAPE"):
        nf4.attention_fwd(wide, wide, wide)
    o, lse = nf4.attention_fwd(q, k, v)
    with pytest.raises(ValueError):
        nf4.attention_bwd(go, q, k, v, o, lse[:, :5])
    with pytest.raises(ValueError):
        nf4.attention_bwd(go[:9], q, k, v, o, lse)


# ---------------------------------------------------------------- residual norm --

def norm_case(T, H, dtype, kinds, seed=0):
    n = gen(seed)
    r = (1.5 * n(T, H)).to(dtype) if "r" in kinds else None
    w_post = 1 + 0.2 * n(H) if "p" in kinds else None
    w_pre = 1 + 0.2 * n(H) if "n" in kinds else None
    gate = 0.5 + 0.2 * n(H) if "c" in kinds else torch.sigmoid(n(T, H)).to(dtype) if "t" in kinds else None
    return dict(y=(0.7 * n(T, H)).to(dtype), residual=r, w_post=w_post, gate=gate, w_pre=w_pre,
                gz=(0.3 * n(T, H)).to(dtype), gh=n(T, H).to(dtype) if w_pre is not None else None)


def check_norm(c, scale=0.5, eps=1e-6):
    T, H = c["y"].shape
    dtype = c["y"].dtype
    kw = dict(w_post=c["w_post"], gate=c["gate"], scale=scale, w_pre=c["w_pre"], eps=eps)
    z, h, stats = nf4.norm_residual_fwd(c["y"], c["residual"], **kw)
    gy, gr, gw_post, ggate, gw_pre = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], stats, **kw)
    got = {k: x for k, x in dict(z=z, h=h, gy=gy, gr=gr, gw_post=gw_post, ggate=ggate, gw_pre=gw_pre).items() if x is not None}
    want, mag = ref.norm_residual(c["y"], c["residual"], c["w_post"], c["gate"], scale, c["w_pre"], eps, c["gz"], c["gh"])
    assert set(got) == set(want)
    for name, x in got.items():
        summed = x.dim() == 1
        assert x.dtype == (F32 if summed else dtype)
        within(x, want[name], ref.norm_bound(want[name], mag[name], dtype, T, H, summed), name)
    return got


@pytest.mark.parametrize("H", [1, 3, 8, 100, 255, 256, 1000, 1024, 2047, 2048, 4096, 5120, 8191, 8192, 16384, 20001])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_widths(H, dtype):
    check_norm(norm_case(5, H, dtype, "rpcn", seed=H))
    check_norm(norm_case(5, H, dtype, "rptn", seed=H))


@pytest.mark.parametrize("T", [1, 2, 151, 152, 153, 304, 305, 700, 2500])
def test_norm_token_counts(T):
    check_norm(norm_case(T, 512, BF16, "rpcn", seed=T))


@pytest.mark.parametrize("kinds", ["n", "rn", "p", "rp", "pn", "rpn", "rcn", "rtn", "rc", "rpt", "rpc", "cpn", "ptn", "r"])
@pytest.mark.parametrize("dtype,H", [(BF16, 768), (F32, 333)])
def test_norm_parts(kinds, dtype, H):
    c = norm_case(40, H, dtype, kinds)
    check_norm(c)
    check_norm(dict(c, gz=None, gh=c["gh"]) if c["gh"] is not None else c, scale=1.0)


def test_norm_plain_input_is_returned_as_it_is():
    c = norm_case(6, 256, BF16, "n")
    z, h, _ = nf4.norm_residual_fwd(c["y"], w_pre=c["w_pre"])
    assert z is c["y"]
    check_norm(dict(c, gz=None), scale=1.0)


def test_norm_strides_and_alignment():
    """Row pitches larger than the width, rows that start off 16 bytes, and gradients of a broadcast row (pitch 0)."""
    c = norm_case(37, 640, BF16, "rptn")
    want = check_norm(c)

    def pitched(x, pad, off):
        return None if x is None else torch.nn.functional.pad(x, (off, pad))[:, off:off + 640]

    for pad, off in ((8, 0), (24, 8), (1, 0), (0, 1), (5, 3)):
        d = {k: pitched(x, pad, off) if x is not None and x.dim() == 2 else x for k, x in c.items()}
        got = check_norm(d)
        if pad % 8 == 0 and off % 8 == 0:
            for k in got:
                assert torch.equal(got[k], want[k])
    check_norm(dict(c, gz=None, gh=torch.ones(1, 1, dtype=BF16, device=DEV).expand(37, 640).contiguous()))


def test_norm_values_at_the_edges():
    """Zero rows (rstd is 1/sqrt(eps)), rows of one large value, a negative scale, a zero gate."""
    c = norm_case(8, 512, F32, "rpcn")
    c["y"][0] = 0
    c["residual"][0] = 0
    c["y"][1] = 0
    c["y"][2], c["residual"][2] = 0, 0
    c["y"][2, 7] = 1e4
    c["gate"][:5] = 0
    check_norm(c)
    check_norm(c, scale=-1.25)
    check_norm(c, scale=0.0)


def test_norm_nan_stays_in_its_row():
    c = norm_case(9, 384, BF16, "rptn")
    kw = dict(w_post=c["w_post"], gate=c["gate"], w_pre=c["w_pre"])
    z, h, st = nf4.norm_residual_fwd(c["y"], c["residual"], **kw)
    base = (z, h, *nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, **kw)[:2])
    c["y"][4, 100] = math.nan
    z, h, st = nf4.norm_residual_fwd(c["y"], c["residual"], **kw)
    after = (z, h, *nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, **kw)[:2])
    rows = torch.arange(9, device=DEV) != 4
    for a, b in zip(base, after):
        assert torch.equal(a[rows], b[rows])
        assert torch.isnan(b[4].float()).all()


def test_norm_wanted_outputs_only():
    c = norm_case(20, 256, BF16, "rpcn")
    kw = dict(w_post=c["w_post"], gate=c["gate"], w_pre=c["w_pre"])
    _, _, st = nf4.norm_residual_fwd(c["y"], c["residual"], **kw)
    full = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, **kw)
    part = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, need_vectors=False, need_residual=False, **kw)
    assert torch.equal(part[0], full[0]) and part[1:] == (None, None, None, None)
    part = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, need_y=False, **kw)
    assert part[0] is None and all(torch.equal(a, b) for a, b in zip(part[1:], full[1:]))


def test_norm_repeats_bit_for_bit():
    c = norm_case(1000, 2048, BF16, "rpcn")
    a, b = check_norm(c), check_norm(c)
    for k in a:
        assert torch.equal(a[k], b[k])


def test_norm_gradient_against_differences():
    c = norm_case(7, 96, F32, "rpcn")
    kw = dict(w_post=c["w_post"], gate=c["gate"], w_pre=c["w_pre"])
    names = ("y", "residual", "w_post", "gate", "w_pre")
    _, _, st = nf4.norm_residual_fwd(c["y"], c["residual"], scale=0.5, **kw)
    grads = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st, scale=0.5, **kw)
    n = gen(4)
    for name, g in zip(names, grads):
        d = n(*g.shape)
        val = []
        for s in (1e-2, -1e-2):
            a = dict(c, **{name: c[name] + s * d})
            z, h, _ = nf4.norm_residual_fwd(a["y"], a["residual"], w_post=a["w_post"], gate=a["gate"], scale=0.5, w_pre=a["w_pre"])
            val.append(((z.double() * c["gz"].double()).sum() + (h.double() * c["gh"].double()).sum()).item())
        want, got = (val[0] - val[1]) / 2e-2, (g.double() * d.double()).sum().item()
        # truncation O(1e-4) of third derivatives, rounding about 1e-7 / 1e-2 of the summed terms
        assert abs(want - got) <= 2e-3 * (g.double() * d.double()).abs().sum().item()


def test_norm_empty_and_refusals():
    c = norm_case(0, 64, BF16, "rpcn")
    got = check_norm(c)
    assert (got["gw_pre"] == 0).all() and (got["gw_post"] == 0).all() and (got["ggate"] == 0).all()
    c = norm_case(4, 64, BF16, "rpcn")
    for bad in (dict(residual=c["residual"].float()), dict(residual=c["residual"][:3]), dict(w_pre=c["w_pre"].to(BF16)),
                dict(w_post=c["w_post"][:60]), dict(gate=c["gate"].to(BF16)), dict(gate=c["gate"][:32]),
                dict(y=c["y"].cpu(), residual=None), dict(y=c["y"].double(), residual=None), dict(y=c["y"].t(), residual=None)):
        d = dict(c, **bad)
        with pytest.raises(ValueError):
            nf4.norm_residual_fwd(d["y"], d["residual"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    _, _, st = nf4.norm_residual_fwd(c["y"], c["residual"], w_pre=c["w_pre"])
    with pytest.raises(ValueError):
        nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st)
    with pytest.raises(ValueError):
        nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], st[:, :3], w_pre=c["w_pre"])
    with pytest.raises(RuntimeError, match="NF4_ERR_INVALID_ARG"):
        nf4.norm_residual_fwd(c["y"], w_pre=c["w_pre"], eps=-1.0)


# ------------------------------------------------------------------------ AdamW --

HYPER = dict(lr=3e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.02)


def flat_views(state, flat):
    return [flat[s] for s in state.slices]


def adam_reference(ps, gs, state, scale=None):
    """Expected parameters (float64) and state buffers after one step, by the definition."""
    b1, b2 = HYPER["betas"]
    out = []
    for i, (p, g, sl) in enumerate(zip(ps, gs, state.slices)):
        if g is None:
            out.append(None)
            continue
        gf = g.float().flatten()
        if scale is not None:
            gf = gf * scale
        mv = []
        for flat, top, lev in ((state.exp_avg, state.exp_avg_absmax, state.levels[0]),
                               (state.exp_avg_sq, state.exp_avg_sq_absmax, state.levels[1])):
            x = flat[sl]
            if state.bits == 8:
                idx = torch.arange(sl.start, sl.stop, device=DEV) // 256
                x = lev[x.long()] * top[idx]
            mv.append(x)
        pd, m, v = ref.adamw(p.flatten(), gf, *mv, state.step + 1, HYPER["lr"], b1, b2, HYPER["eps"], HYPER["weight_decay"])
        rec = {"p": pd, "m": m, "v": v}
        if state.bits == 8:
            for key, x, lev in (("m", m, state.levels[0]), ("v", v, state.levels[1])):
                pad = torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)
                codes, top = ref.encode8(pad, lev)
                rec[key], rec[key + "_top"] = codes.flatten()[:x.numel()], top
        out.append(rec)
    return out


def check_adam(ps, gs, state, grad_scale=None):
    want = adam_reference(ps, gs, state, grad_scale)
    before = [p.clone() for p in ps]
    held = (state.exp_avg.clone(), state.exp_avg_sq.clone())
    nf4.adamw_step(ps, gs, state, grad_scale=grad_scale, **HYPER)
    for i, (p, w, sl) in enumerate(zip(ps, want, state.slices)):
        if w is None:
            assert torch.equal(p, before[i]) and torch.equal(state.exp_avg[sl], held[0][sl])
            continue
        u = ref.UNIT[p.dtype]
        step = (w["p"] - before[i].double().flatten()).abs() + HYPER["lr"] * HYPER["weight_decay"] * before[i].double().flatten().abs()
        bound = (u if p.dtype != F32 else 2 * u) * w["p"].abs() * 1.01 + 16 * 2.0 ** -24 * step + 1e-30
        if p.dtype == F16:
            bound = bound + 2.0 ** -25  # subnormals
        within(p.flatten(), w["p"], bound, f"p{i}")
        assert torch.equal(state.exp_avg[sl], w["m"]), f"m{i}"
        assert torch.equal(state.exp_avg_sq[sl], w["v"]), f"v{i}"
        if state.bits == 8:
            blocks = slice(sl.start // 256, sl.start // 256 + -(-p.numel() // 256))
            assert torch.equal(state.exp_avg_absmax[blocks], w["m_top"])
            assert torch.equal(state.exp_avg_sq_absmax[blocks], w["v_top"])


SHAPES = [(1,), (255,), (256,), (257,), (33, 47), (1024, 16), (3, 5, 7), (4096,), (0,), (511,)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_adamw_steps(bits, dtype):
    """Several steps from zero states over tensors of every shape, gradients of very different sizes."""
    n = gen(bits)
    ps = [(0.05 * n(*s)).to(dtype) for s in SHAPES]
    state = nf4.adamw_state(ps, bits=bits)
    for step in range(5):
        gs = [(10.0 ** (i % 5 - 3) * n(*s)).to(dtype) for i, s in enumerate(SHAPES)]
        gs[3] = None if step == 2 else gs[3]
        check_adam(ps, gs, state)
    assert state.step == 5


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_adamw_codes_over_the_whole_map(dtype):
    """Moments that visit every level, both signs, values at and next to the midpoints, tiny and huge scales."""
    n = gen(11)
    for size in (1e-18, 1e-9, 1e-3, 1.0, 1e6, 1e15):
        g = (size * n(64, 256) * torch.exp(4 * n(64, 256)).clamp(1e-7, 1e2)).to(dtype)
        ps = [torch.zeros(64, 256, dtype=dtype, device=DEV)]
        state = nf4.adamw_state(ps, bits=8)
        check_adam(ps, [g], state)
        check_adam(ps, [g.flip(0)], state)


def test_adamw_midpoint_ties_take_the_lower_level():
    """m = 0.1 g exactly representable ratios: g holds the block maximum 1 and the fp32 midpoints themselves."""
    for which, lev in ((0, nf4.dynamic_code8()), (1, nf4.dynamic_code8_unsigned())):
        lev = lev.to(DEV)
        mid = ((lev[:-1].double() + lev[1:].double()) / 2).float()
        x = torch.cat([mid, torch.ones(1, device=DEV)]).view(1, 256)
        near = torch.stack([torch.nextafter(x, torch.full_like(x, s)) for s in (-9.0, 9.0)]).view(2, 256)
        near[:, -1] = 1
        x = torch.cat([x, near]).contiguous()
        ps = [torch.zeros_like(x)]
        state = nf4.adamw_state(ps, bits=8)
        # the values reach the encoder unchanged: zero gradient, decay factors 1 are not allowed, so betas near it
        codes, top = ref.encode8(x, lev)
        target, tops = (state.exp_avg, state.exp_avg_absmax) if which == 0 else (state.exp_avg_sq, state.exp_avg_sq_absmax)
        # a first step from zero states has m = g (1 - b1): choose b1 = 0.5 so that the factor is exact
        g = 2 * x if which == 0 else torch.sqrt(2 * x)
        nf4.adamw_step(ps, [g], state, lr=0.0, betas=(0.5, 0.5), eps=1e-8, weight_decay=0.0)
        if which == 1:  # what the fp32 squares give
            codes, top = ref.encode8((g * g) * 0.5, lev)
        assert torch.equal(target.view(3, 256), codes) and torch.equal(tops, top)


def test_adamw_grad_scale_and_many_tensors():
    """More tensors than one launch's table holds, and a clipping factor on the device."""
    n = gen(2)
    ps = [(0.1 * n(1 + (37 * i) % 700)).to(BF16) for i in range(900)]
    gs = [n(*p.shape).to(BF16) for p in ps]
    state = nf4.adamw_state(ps, bits=8)
    check_adam(ps, gs, state, grad_scale=torch.tensor(0.37, device=DEV))


def test_adamw_unaligned_tensors():
    """Parameters and gradients that start off 16 bytes."""
    n = gen(3)
    for bits in (8, 32):
        base, grads = n(5000).to(BF16), n(5000).to(BF16)
        ps, gs = [base[1:700], base[703:2800], base[3001:5000]], [grads[3:702], grads[800:2897], grads[3001:5000]]
        state = nf4.adamw_state(ps, bits=bits)
        guard = base[700:703].clone()
        check_adam(ps, gs, state)
        assert torch.equal(base[700:703], guard)


def test_adamw_zero_and_nonfinite_gradients():
    ps = [torch.ones(600, device=DEV)]
    state = nf4.adamw_state(ps, bits=8)
    check_adam(ps, [torch.zeros(600, device=DEV)], state)
    m, v = nf4.adamw_state_values(state)
    assert (m == 0).all() and (v == 0).all()
    g = torch.ones(600, device=DEV)
    g[300] = math.nan
    nf4.adamw_step(ps, [g], state, **HYPER)
    m, v = (x[:600] for x in nf4.adamw_state_values(state))
    # the NaN's block (256 .. 511) reads as NaN; the others do not notice
    assert torch.isnan(m[256:512]).all() and torch.isnan(v[256:512]).all()
    assert torch.isfinite(m[:256]).all() and torch.isfinite(m[512:]).all()
    assert torch.isnan(ps[0][300]) and torch.isfinite(ps[0][:300]).all() and torch.isfinite(ps[0][301:]).all()


def test_adamw_state_values():
    n = gen(6)
    ps = [n(1000), n(37, 53)]
    state = nf4.adamw_state(ps, bits=8)
    for _ in range(3):
        nf4.adamw_step(ps, [n(1000), n(37, 53)], state, **HYPER)
    m, v = nf4.adamw_state_values(state)
    for got, codes, top, lev in ((m, state.exp_avg, state.exp_avg_absmax, state.levels[0]),
                                 (v, state.exp_avg_sq, state.exp_avg_sq_absmax, state.levels[1])):
        assert torch.equal(got, lev[codes.long()] * top.repeat_interleave(256))


def test_adamw_refusals():
    p, g = torch.zeros(10, device=DEV), torch.zeros(10, device=DEV)
    state = nf4.adamw_state([p], bits=8)
    for ps, gs in (([p], [g, g]), ([p.to(BF16)], [g]), ([p], [g[:5]]), ([torch.zeros(20, device=DEV)[::2]], [g]),
                   ([p.cpu()], [g.cpu()]), ([p.double()], [g.double()])):
        with pytest.raises(ValueError):
            nf4.adamw_step(ps, gs, state, **HYPER)
    with pytest.raises(ValueError):
        nf4.adamw_state([p], bits=4)
    with pytest.raises(ValueError):
        nf4.adamw_state([p.cpu()])
    with pytest.raises(ValueError):
        nf4.adamw_step([p], [g], state, grad_scale=torch.ones(2, device=DEV), **HYPER)
    with pytest.raises(RuntimeError, match="NF4_ERR_INVALID_ARG"):
        nf4.adamw_step([p], [g], state, **dict(HYPER, betas=(1.0, 0.9)))
    assert state.step == 0
