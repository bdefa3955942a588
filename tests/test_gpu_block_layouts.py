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


# -------------------------------------------------------------------- attention --

def qkv(T, Hq, Hk, D, dtype, seed=0):
    n = gen(seed)
    q, k = 1.3 * n(T, Hq, D), 1.3 * n(T, Hk, D)
    return [x.to(dtype) for x in (q, k, n(T, Hk, D) + 0.3, n(T, Hq, D))]


def offsets(lens):
    b = ref.bounds_of(lens)
    return b, torch.tensor(b, dtype=torch.int32, device=DEV)


# Relative rms error of one rounding to fp16: 2^-11 / sqrt(3) of the binade's start, over mantissas spread evenly in
# their logarithm a factor sqrt(3 / (8 ln 2)).
ROUND16 = 2.0 ** -11 / math.sqrt(3) * math.sqrt(3 / (8 * math.log(2)))


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def check_relative(grads, want, unit=ROUND16):
    """Relative error of each whole gradient: one rounding of the result (subnormal where it is), one of the weights or
    score gradients of its product, one of the probabilities that o, and so the row sums, are made of.  They are
    independent, so their squares add; a tenth on top."""
    for got, name in zip(grads, ("gq", "gk", "gv")):
        assert torch.isfinite(got).all(), name
        one = relative(want[name].to(got.dtype), want[name])
        assert relative(got, want[name]) <= 1.1 * math.sqrt(one ** 2 + 2 * unit ** 2), (name, relative(got, want[name]) / one)


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 3e-4, 1e-4, 3e-5])
@pytest.mark.parametrize("Hq,Hk,D,lens", [(4, 2, 128, [1500, 37]), (2, 2, 64, [2100]), (3, 1, 80, [700, 1, 900])])
def test_attention_fp16_gradients_of_any_size(size, Hq, Hk, D, lens):
    q, k, v, go = qkv(sum(lens), Hq, Hk, D, F16)
    go = (size * go.float()).half()
    b, cu = offsets(lens)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    grads = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    check_relative(grads, ref.attention(q, k, v, b, D ** -0.5, go)[0])


@pytest.mark.parametrize("Hq,Hk,D,lens", [(2, 1, 64, [2500]), (2, 2, 128, [2500]), (4, 1, 96, [1, 700, 0, 33, 1200])])
def test_attention_bf16_error_of_whole_gradients(Hq, Hk, D, lens):
    """Beside the bounds of single elements, which grow with the sum of their terms' sizes, one for each gradient."""
    q, k, v, go = qkv(sum(lens), Hq, Hk, D, BF16)
    b, cu = offsets(lens)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    grads = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    check_relative(grads, ref.attention(q, k, v, b, D ** -0.5, go)[0], 8 * ROUND16)


def test_attention_fp16_large_score_gradients():
    """Score gradients beyond fp16's largest value whose sums, times small queries and keys, fit."""
    q, k, v, go = qkv(300, 2, 1, 128, F16)
    q, k, v, go = ((f * x.float()).half() for f, x in ((1e-3, q), (1e-3, k), (40, v), (4e3, go)))
    o, lse = nf4.attention_fwd(q, k, v)
    check_relative(nf4.attention_bwd(go, q, k, v, o, lse), ref.attention(q, k, v, [0, 300], 128 ** -0.5, go)[0])


def test_attention_fp16_rows_of_different_size():
    """Output gradients from 1e-5 to 10 in neighbouring rows: each row's gq is as good as on its own."""
    T = 1200
    q, k, v, go = qkv(T, 2, 2, 128, F16)
    size = 10.0 ** (torch.arange(T, device=DEV) * 0.37 % 6 - 5)
    go = (size[:, None, None] * go.float()).half()
    o, lse = nf4.attention_fwd(q, k, v)
    gq = nf4.attention_bwd(go, q, k, v, o, lse)[0].double()[1:]  # row 0 sees one key: its gradient is 0
    want = ref.attention(q, k, v, [0, T], 128 ** -0.5, go)[0]["gq"][1:]

    def mean_square(x):
        return ((x - want).square().sum(-1) / want.square().sum(-1)).mean().item()

    assert mean_square(gq) <= 1.21 * (mean_square(want.half().double()) + 2 * ROUND16 ** 2)


@pytest.mark.parametrize("at", [3, 127, 128, 200])
def test_attention_fp16_masked_values_leave_no_trace(at):
    """The scale that fp16 score gradients are held at comes from what a row sees: a large value or output gradient
    behind the mask, or in another sequence, changes no bit."""
    lens = [300, 150]
    b, cu = offsets(lens)
    q, k, v, go = qkv(sum(lens), 4, 2, 64, F16)
    go = (1e-4 * go.float()).half()

    def both():
        o, lse = nf4.attention_fwd(q, k, v, cu)
        return nf4.attention_bwd(go, q, k, v, o, lse, cu)

    base = both()
    v[at] *= 4096
    gq = both()[0]
    assert torch.equal(gq[:at], base[0][:at]) and torch.equal(gq[300:], base[0][300:])
    v[at] /= 4096
    go[at] *= 4096
    gq, gk, gv = both()
    assert torch.equal(gk[at + 1:], base[1][at + 1:]) and torch.equal(gv[at + 1:], base[2][at + 1:])
    rows = torch.arange(450, device=DEV) != at
    assert torch.equal(gq[rows], base[0][rows])


def test_attention_fp16_zero_and_nonfinite_gradients():
    """go of zero gives zero gradients; a NaN in go reaches the keys that its row sees and no others."""
    b, cu = offsets([300, 60])
    q, k, v, go = qkv(360, 2, 2, 64, F16)
    o, lse = nf4.attention_fwd(q, k, v, cu)
    for g in nf4.attention_bwd(torch.zeros_like(go), q, k, v, o, lse, cu):
        assert (g == 0).all()
    base = nf4.attention_bwd(go, q, k, v, o, lse, cu)
    for bad in (math.nan, math.inf):
        x = go.clone()
        x[140, 1, 9] = bad
        gq, gk, gv = nf4.attention_bwd(x, q, k, v, o, lse, cu)
        assert torch.equal(gk[141:], base[1][141:]) and torch.equal(gv[141:], base[2][141:])
        assert not torch.isfinite(gk[:141, 1]).any() and not torch.isfinite(gv[:141, 1, 9]).any()
        rows = torch.arange(360, device=DEV) != 140
        assert torch.equal(gq[rows], base[0][rows]) and not torch.isfinite(gq[140, 1]).any()


@pytest.mark.parametrize("kind", ["tokens", "heads", "both", "misaligned", "odd pitch"])
def test_attention_output_gradient_of_any_layout_stays_on_the_tensor_cores(kind):
    """A gradient broadcast over tokens or heads (of a mean, for instance), or that no bulk copy can load, is copied:
    the backward does not leave the tensor-core kernels for it."""
    T, H, D = 200, 4, 64
    q, k, v, go = qkv(T, H, 2, D, BF16)
    if kind in ("misaligned", "odd pitch"):
        pitch = H * D + (8 if kind == "misaligned" else 3)
        store = torch.zeros(T * pitch + 1, dtype=BF16, device=DEV)
        go = store[1 if kind == "misaligned" else 0:].as_strided((T, H, D), (pitch, D, 1)).copy_(go)
    else:
        go = go[:1 if kind != "heads" else T, :1 if kind != "tokens" else H].expand(T, H, D)
    o, lse = nf4.attention_fwd(q, k, v)
    want = nf4.attention_bwd(go.contiguous(), q, k, v, o, lse)
    nf4.reset_path_counters()
    got = nf4.attention_bwd(go, q, k, v, o, lse)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    nf4.nf4_attention(*leaves).backward(go)
    counts = nf4.path_counters()
    assert counts["attention_any"] == 0 and counts["attention"] == 3
    for a, b, leaf in zip(got, want, leaves):
        assert torch.equal(a, b) and torch.equal(leaf.grad, b)


@pytest.mark.parametrize("gate", ["channel", "token", None])
@pytest.mark.parametrize("T", [5, 400])
@pytest.mark.parametrize("y,r,w,gz", [(1e-14, 1e-14, 1e-14, 1.0), (1e-18, 1.0, 1.0, 1e5)])
def test_norm_rows_of_tiny_values(y, r, w, gz, gate, T):
    """Tiny rows with eps = 0: the powers of a row's 1 / rms leave fp32, the gradients do not."""
    n, H = gen(3), 512
    c = dict(y=y * n(T, H), residual=r * n(T, H), gz=gz * n(T, H), gh=n(T, H), w_post=w * (1 + 0.2 * n(H)), w_pre=1 + 0.2 * n(H))
    g = n(H) if gate == "channel" else n(T, H) if gate == "token" else None
    kw = dict(w_post=c["w_post"], gate=g, scale=0.5, w_pre=c["w_pre"], eps=0.0)
    z, h, stats = nf4.norm_residual_fwd(c["y"], c["residual"], **kw)
    gy, gr, gw_post, ggate, gw_pre = nf4.norm_residual_bwd(c["gz"], c["gh"], c["y"], c["residual"], stats, **kw)
    want, mag = ref.norm_residual(c["y"], c["residual"], c["w_post"], g, 0.5, c["w_pre"], 0.0, c["gz"], c["gh"])
    for name, x in dict(z=z, h=h, gy=gy, gr=gr, gw_post=gw_post, ggate=ggate, gw_pre=gw_pre).items():
        if x is None:
            continue
        bound = ref.norm_bound(want[name], mag[name], F32, T, H, x.dim() == 1)
        assert torch.isfinite(x).all(), name
        assert ((x.double() - want[name]).abs() <= bound).all(), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("at", [5, 127, 128, 200, 299])
def test_attention_key_of_minus_infinity(at, dtype):
    """A key whose scores are -inf takes no part: outputs and gradients are those without it, but for gq in the
    channel where 0 meets the infinity."""
    q, k, v, go = qkv(300, 4, 2, 128, dtype)
    q[..., 3] = q[..., 3].abs() + 0.5
    k[at, 1, 3] = -6e4  # as good as -inf: every weight underflows to 0 in 64 bits
    smax = 128 ** -0.5 * (q.double().norm(dim=2).max() * k[torch.arange(300, device=DEV) != at].double().norm(dim=2).max()).item()
    want, mag = ref.attention(q, k, v, [0, 300], 128 ** -0.5, go)
    k[at, 1, 3] = -math.inf
    o, lse = nf4.attention_fwd(q, k, v)
    got = dict(zip(("gq", "gk", "gv"), nf4.attention_bwd(go, q, k, v, o, lse)), o=o)
    assert torch.isnan(got["gq"][at:, 2:, 3]).all()
    got["gq"][at:, 2:, 3] = want["gq"][at:, 2:, 3].to(dtype)
    for name, x in got.items():
        assert torch.isfinite(x).all(), name
        bound = ref.attention_bound(name, want[name], mag[name], dtype, smax)
        assert ((x.double() - want[name]).abs() <= bound).all(), name


def test_attention_out_must_not_share_storage():
    """Rows of `out` that share storage would be written by several blocks at once: refused; any other view is filled."""
    q, k, v, _ = qkv(50, 4, 2, 64, BF16)
    o, _ = nf4.attention_fwd(q, k, v)
    row = torch.zeros(1, 4, 64, dtype=BF16, device=DEV)
    for out in (row.expand(50, 4, 64), torch.zeros(50, 1, 64, dtype=BF16, device=DEV).expand(50, 4, 64),
                torch.zeros(50 * 128 + 128, dtype=BF16, device=DEV).as_strided((50, 4, 64), (128, 64, 1))):
        with pytest.raises(ValueError, match="out"):
            nf4.attention_fwd(q, k, v, out=out)
    wide = torch.zeros(50, 6, 72, dtype=BF16, device=DEV)
    for out in (wide[:, 1:5, :64], torch.zeros(4, 50, 64, dtype=BF16, device=DEV).transpose(0, 1)):
        assert nf4.attention_fwd(q, k, v, out=out)[0] is out and torch.equal(out, o)
    one = torch.zeros(1, 1, 64, dtype=BF16, device=DEV).expand(1, 4, 64).contiguous()[:, :1].expand(1, 1, 64)
    nf4.attention_fwd(q[:1, :1], k[:1, :1], v[:1, :1], out=one)


@pytest.mark.parametrize("backward", [False, True])
def test_norm_copies_that_never_complete(backward):
    """A streamed row's wait that runs out is recorded, the launch ends, other blocks' rows and later calls are right."""
    from bit_nf4_quantized_linear_gb300 import _lib
    n, T, H = gen(5), 6000, 512
    y, r, gz, gh = (n(T, H).to(BF16) for _ in range(4))
    w = 1 + 0.2 * n(H)

    def call():
        z, h, stats = nf4.norm_residual_fwd(y, r, w_post=w, w_pre=w)
        if not backward:
            return z, h
        if armed:
            _lib.inject_norm_timeout()
        return nf4.norm_residual_bwd(gz, gh, y, r, stats, w_post=w, w_pre=w)[:2]

    armed = False
    want = call()
    armed = True
    if not backward:
        _lib.inject_norm_timeout()
    got = call()
    torch.cuda.synchronize()
    assert nf4.device_status(clear=True) == 6
    for a, b in zip(got, want):
        # the failing block walks rows 0, grid, 2 grid, ...: a small part
        assert (a == b).all(1).float().mean() > 0.9 and torch.equal(a[1:100], b[1:100])
    armed = False
    for a, b in zip(call(), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert nf4.device_status() == 0
