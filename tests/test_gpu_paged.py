"""The paged cache on the GPU: append and attention against their definitions, at the lengths, pages, layouts and values
where they can go wrong.  Tolerances are error bounds computed from the reference's own magnitudes."""
import math
import random

import pytest
import torch

import bit_nf4_quantized_linear_gb300 as nf4
from tests import decode_refs as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BAD_OFFSETS = 8


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


def cache(lengths, Hk, D, dtype, page=16, order="token", seed=0, spare=2, extra_pages=1):
    """(k_pages, v_pages, page_table, lengths): shuffled pages, leftovers in every slot, -1 past each sequence's pages."""
    n = gen(seed)
    need = [-(-m // page) for m in lengths]
    total = sum(need) + spare
    ids = list(range(total))
    random.Random(seed).shuffle(ids)
    table = torch.full((len(lengths), max([1, *need]) + extra_pages), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += m
    if order == "token":
        kp, vp = (1.3 * n(total, page, Hk, D)).to(dtype), (n(total, page, Hk, D) + 0.3).to(dtype)
    else:
        kp, vp = ((x.to(dtype)).transpose(1, 2) for x in (1.3 * n(total, Hk, page, D), n(total, Hk, page, D) + 0.3))
    return kp, vp, table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV)


def queries(n, Hq, D, dtype, seed=1):
    return (1.3 * gen(seed)(n, Hq, D)).to(dtype)


def check(q, kp, vp, table, lengths, scale=None, path=None, out=None):
    before = nf4.path_counters()
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths, scale=scale, out=out)
    after = nf4.path_counters()
    assert path is None or after[path] == before[path] + 1, path
    lens, D = lengths.tolist(), q.shape[2]
    want, wl, mag, smag = ref.paged_attention(q, kp, vp, table, lens, D ** -0.5 if scale is None else scale)
    bo, bl = ref.paged_bounds(want, wl, mag, smag, lens, D, q.dtype)
    assert o.dtype == q.dtype and lse.dtype == F32
    live = lengths > 0
    assert torch.isfinite(o).all() and torch.equal(lse == -math.inf, (~live)[:, None].expand_as(lse))
    assert (o[~live] == 0).all()
    over = ((o.double() - want).abs() / bo).max().item()
    assert over <= 1, f"o: {over:.3g} of its bound"
    if live.any():
        over = ((lse.double() - wl)[live].abs() / bl[live]).max().item()
        assert over <= 1, f"lse: {over:.3g} of its bound"
    return o, lse


LENGTHS = [[1], [2], [15], [16], [17], [48], [63], [64], [65], [128], [129], [1000], [0], [0, 5, 0, 130, 1, 0], [64, 64, 64], [3000, 1],
           [1] * 40, [257, 0, 511, 512, 513]]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda l: "-".join(map(str, l[:6])))
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16), (80, F32)])
def test_attention_lengths(lens, D, dtype):
    kp, vp, table, lengths = cache(lens, 2, D, dtype)
    check(queries(len(lens), 8, D, dtype), kp, vp, table, lengths)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (4, 4), (10, 2), (8, 1), (18, 2), (16, 1), (20, 1), (40, 1)])
@pytest.mark.parametrize("D", [1, 8, 37, 40, 64, 72, 96, 128, 136, 192, 256])
def test_attention_heads_and_widths(Hq, Hk, D):
    for dtype in (BF16, F16) if Hq in (3, 18) else (BF16,):
        kp, vp, table, lengths = cache([331, 7, 64], Hk, D, dtype, seed=D)
        check(queries(3, Hq, D, dtype), kp, vp, table, lengths, path="paged_attention" if D % 8 == 0 else "paged_attention_any")


@pytest.mark.parametrize("Hq,Hk,D", [(3, 1, 5), (8, 8, 64), (10, 2, 128), (9, 1, 200), (6, 3, 256)])
def test_attention_fp32(Hq, Hk, D):
    kp, vp, table, lengths = cache([200, 0, 33], Hk, D, F32, seed=D)
    check(queries(3, Hq, D, F32), kp, vp, table, lengths, scale=0.1, path="paged_attention_any")


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 333])
@pytest.mark.parametrize("order", ["token", "head"])
def test_attention_pages(page, order):
    kp, vp, table, lengths = cache([700, 99, 1, 0, 333], 2, 64, BF16, page=page, order=order, seed=page)
    check(queries(5, 8, 64, BF16), kp, vp, table, lengths, path="paged_attention")
    for D in (64, 100, 128):
        kp, vp, table, lengths = cache([700, 99, 1, 0, 333], 2, D, F32, page=page, order=order, seed=page)
        check(queries(5, 8, D, F32), kp, vp, table, lengths, path="paged_attention_any")


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (8, 2), (5, 1), (16, 2), (9, 1), (20, 1)])
@pytest.mark.parametrize("D", [4, 20, 64, 68, 128, 132, 200, 256])
def test_attention_fp32_heads(Hq, Hk, D):
    """Groups of one to twenty heads, widths that fill a row of the ring and do not; rows that no 16-byte copy can take."""
    lens = [331, 7, 64, 0, 1500]
    kp, vp, table, lengths = cache(lens, Hk, D, F32, seed=D)
    q = queries(5, Hq, D, F32)
    check(q, kp, vp, table, lengths)
    odd = torch.zeros(kp.numel() + 1, device=DEV)[1:].view(kp.shape)
    odd.copy_(kp)
    check(q, odd, vp, table, lengths)


@pytest.mark.parametrize("n", [33, 300, 1500])
def test_attention_many_sequences(n):
    """More sequences than threads of a CTA, idle ones among them."""
    rng = random.Random(n)
    lens = [rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, 300)]) for _ in range(n)]
    kp, vp, table, lengths = cache(lens, 2, 64, BF16)
    check(queries(n, 4, 64, BF16), kp, vp, table, lengths)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (F32, 64)])
def test_attention_long_sequences(dtype, D):
    """Every (sequence, head) is cut over many CTAs."""
    kp, vp, table, lengths = cache([30001, 9], 1, D, dtype, page=64)
    check(queries(2, 4, D, dtype), kp, vp, table, lengths)


def test_attention_layouts():
    """Views give the bits of contiguous tensors on the tensor cores; unaligned ones are right on the other kernel."""
    lens, Hq, Hk, D = [131, 0, 70], 8, 2, 64
    kp, vp, table, lengths = cache(lens, Hk, D, BF16)
    q = queries(3, Hq, D, BF16)
    want = nf4.paged_attention(q, kp, vp, table, lengths)

    def same(*args, **kw):
        for a, b in zip(want, nf4.paged_attention(*args, **kw)):
            assert torch.equal(a, b)

    both = torch.stack([kp, vp], 1)  # keys and values side by side in one buffer
    same(q, both[:, 0], both[:, 1], table, lengths)
    same(torch.cat([q, q], 2)[:, :, :D], kp, vp, table, lengths)
    same(q.transpose(0, 1).contiguous().transpose(0, 1), kp, vp, table, lengths)
    same(torch.cat([q.view(3, -1), q.view(3, -1)], 1)[:, :Hq * D].view(3, Hq, D), kp, vp, table, lengths)
    wide = torch.full((3, table.shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    same(q, kp, vp, wide[:, :table.shape[1]], lengths)
    same(q, kp, vp, wide, lengths)  # entries past a sequence's pages are not read
    out = torch.zeros(Hq, 3, D, dtype=BF16, device=DEV).transpose(0, 1)
    same(q, kp, vp, table, lengths, out=out)
    odd = torch.zeros(kp.numel() + 1, dtype=BF16, device=DEV)[1:].view(kp.shape)
    odd.copy_(kp)
    check(q, odd, vp, table, lengths, path="paged_attention_any")
    check(q, kp, vp, table, lengths, out=torch.zeros(3, Hq, D + 1, dtype=BF16, device=DEV)[:, :, :D], path="paged_attention_any")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_leftovers_leave_no_trace(dtype, bad):
    """NaN and infinities in slots past a length and in pages of nobody change no bit."""
    lens = [37, 0, 64, 1, 100]
    kp, vp, table, lengths = cache(lens, 2, 64, dtype)
    q = queries(5, 4, 64, dtype)
    want = nf4.paged_attention(q, kp, vp, table, lengths)
    owned = torch.zeros(kp.shape[:2], dtype=torch.bool, device=DEV)
    for i, m in enumerate(lens):
        owned[ref.slots_of(table[i], m, 16)] = True
    kp[~owned], vp[~owned] = bad, bad
    for a, b in zip(want, nf4.paged_attention(q, kp, vp, table, lengths)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("at", [0, 15, 63, 64, 99])
def test_attention_nonfinite_values_reach_their_rows_only(dtype, at):
    lens = [90, 100, 50]
    kp, vp, table, lengths = cache(lens, 2, 64, dtype)
    q = queries(3, 4, 64, dtype)
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    page, slot = table[1, at // 16], at % 16
    for bad in (math.nan, math.inf, -math.inf):
        keep = vp[page, slot, 1, 3].clone()
        vp[page, slot, 1, 3] = bad
        o2, lse2 = nf4.paged_attention(q, kp, vp, table, lengths)
        vp[page, slot, 1, 3] = keep
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[1, 2:, 3] = True
        assert torch.equal(o[~hit], o2[~hit]) and torch.equal(lse, lse2)
        assert torch.equal(o2[hit].isnan(), torch.full_like(o2[hit], bad).isnan()) and not torch.isfinite(o2[hit]).any()
        keep = kp[page, slot, 1].clone()
        kp[page, slot, 1] = bad
        o2, lse2 = nf4.paged_attention(q, kp, vp, table, lengths)
        kp[page, slot, 1] = keep
        rows = torch.ones(3, 4, dtype=torch.bool, device=DEV)
        rows[1, 2:] = False
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[rows], lse2[rows])
        if math.isnan(bad):
            assert o2[1, 2:].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_attention_key_of_minus_infinity_scores(dtype):
    """Tokens of score -inf have no weight, wherever they lie: the answer is that of the sequence without them."""
    D = 64
    kp, vp, table, lengths = cache([200], 1, D, dtype, seed=5)
    q = queries(1, 4, D, dtype).abs() + 0.1
    dead = torch.zeros(200, dtype=torch.bool, device=DEV)
    dead[:70] = dead[130:150] = True
    page, slot = ref.slots_of(table[0], 200, 16)
    kp[page[dead], slot[dead], 0] = -math.inf
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    live = (~dead).nonzero().flatten()
    k2, v2 = kp[page[live], slot[live]][None], vp[page[live], slot[live]][None]
    one = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    check(q, k2, v2, one, torch.tensor([live.numel()], dtype=torch.int32, device=DEV))
    want, wl, mag, smag = ref.paged_attention(q, k2, v2, one, [live.numel()], D ** -0.5)
    bo, bl = ref.paged_bounds(want, wl, mag, smag, [200], D, dtype)
    assert ((o.double() - want).abs() <= bo).all() and ((lse.double() - wl).abs() <= bl).all()


def test_attention_large_and_equal_scores():
    for dtype in (BF16, F16, F32):
        kp, vp, table, lengths = cache([300, 20], 2, 64, dtype)
        q = queries(2, 8, 64, dtype)
        check(8 * q, kp, vp, table, lengths)
        check(torch.zeros_like(q), kp, vp, table, lengths)
        for scale in (-0.2, 0.0, 3.0):
            check(q, kp, vp, table, lengths, scale=scale)


def test_attention_offsets_past_32_bits():
    """A page that lies more than 2^32 elements into the buffer."""
    D, Hk, page = 128, 8, 64
    pages = (1 << 32) // (page * Hk * D) + 3
    big = [torch.empty(pages, page, Hk, D, dtype=BF16, device=DEV) for _ in range(2)]
    kp, vp, _, lengths = cache([page, 5], Hk, D, BF16, page=page, spare=0)
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device=DEV)
    for b, p in zip(big, (kp, vp)):
        b[pages - 1], b[pages - 2] = p[0], p[1]
    q = queries(2, 16, D, BF16)
    check(q, *big, table, lengths)
    for dst in big:
        dst[pages - 1].zero_()
    nf4.paged_append(kp[0], vp[0], *big, table, torch.tensor([page, 0], dtype=torch.int32, device=DEV),
                     torch.tensor([0, page, page], dtype=torch.int32, device=DEV))
    assert torch.equal(big[0][pages - 1], kp[0]) and torch.equal(big[1][pages - 1], vp[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_pages_and_lengths_are_recorded_and_passed_over(dtype):
    kp, vp, table, lengths = cache([100, 40, 16], 2, 64, dtype, extra_pages=0)
    q = queries(3, 4, 64, dtype)
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad  # tokens 16 .. 31 of sequence 1
        o2, lse2 = nf4.paged_attention(q, kp, vp, t, lengths)
        assert nf4.device_status(clear=True) == BAD_OFFSETS
        assert torch.equal(o[::2], o2[::2]) and torch.equal(lse[::2], lse2[::2])
        page, slot = ref.slots_of(table[1], 40, 16)
        have = torch.tensor([i for i in range(40) if not 16 <= i < 32], device=DEV)
        one = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
        want, wl, mag, smag = ref.paged_attention(q[1:2], kp[page[have], slot[have]][None], vp[page[have], slot[have]][None], one, [24], 0.125)
        bo, bl = ref.paged_bounds(want, wl, mag, smag, [40], 64, dtype)
        assert ((o2[1:2].double() - want).abs() <= bo).all() and ((lse2[1:2].double() - wl).abs() <= bl).all()
        k, v = kp[0, :3].clone(), vp[0, :3].clone()
        keep = kp.clone(), vp.clone()
        nf4.paged_append(k, v, kp, vp, t, torch.tensor([0, 30, 0], dtype=torch.int32, device=DEV))
        assert nf4.device_status(clear=True) == BAD_OFFSETS
        assert torch.equal(keep[0], kp) and torch.equal(keep[1], vp)
    for bad in (-5, table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        n = lengths.clone()
        n[2] = bad
        o2, lse2 = nf4.paged_attention(q, kp, vp, table, n)
        assert nf4.device_status(clear=True) == BAD_OFFSETS
        # another length cuts the batch elsewhere, so the other sequences' sums may be grouped anew: within their bounds
        want, wl, mag, smag = ref.paged_attention(q[:2], kp, vp, table, [100, 40], 0.125)
        bo, bl = ref.paged_bounds(want, wl, mag, smag, [100, 40], 64, dtype)
        assert ((o2[:2].double() - want).abs() <= bo).all() and ((lse2[:2].double() - wl).abs() <= bl).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 37])
def test_rows_without_a_weight_are_zero(dtype, D):
    """All scores -inf, all pages missing, a table of no columns: zeros and -inf, beside rows that are as ever."""
    kp, vp, table, lengths = cache([40, 70, 33], 2, D, dtype)
    q = queries(3, 4, D, dtype).abs() + 0.1
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    k2 = kp.clone()
    k2[table[1, :5].long()] = -math.inf
    o2, lse2 = nf4.paged_attention(q, k2, vp, table, lengths)
    assert (o2[1] == 0).all() and (lse2[1] == -math.inf).all() and torch.equal(o2[::2], o[::2]) and torch.equal(lse2[::2], lse[::2])
    t = table.clone()
    t[1] = -1
    o2, lse2 = nf4.paged_attention(q, kp, vp, t, lengths)
    assert nf4.device_status(clear=True) == BAD_OFFSETS
    assert (o2[1] == 0).all() and (lse2[1] == -math.inf).all() and torch.equal(o2[::2], o[::2]) and torch.equal(lse2[::2], lse[::2])
    o2, lse2 = nf4.paged_attention(q, kp, vp, table[:, :0], lengths)
    assert nf4.device_status(clear=True) == BAD_OFFSETS
    assert (o2 == 0).all() and (lse2 == -math.inf).all()
    o2, lse2 = nf4.paged_attention(q, kp[:0], vp[:0], table, lengths)
    nf4.paged_append(kp[0, :3], vp[0, :3], kp[:0], vp[:0], table, lengths)
    assert nf4.device_status(clear=True) == BAD_OFFSETS
    assert (o2 == 0).all() and (lse2 == -math.inf).all()
    o2, lse2 = nf4.paged_attention(q[:0], kp, vp, table[:0], lengths[:0])
    assert o2.shape == (0, 4, D) and lse2.shape == (0, 4)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 128), (F32, 64), (F16, 31)])
def test_out_may_be_the_queries(dtype, D):
    kp, vp, table, lengths = cache([300, 17, 0, 64, 5000], 2, D, dtype)
    q = queries(5, 24, D, dtype)
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    version = q._version
    o2, lse2 = nf4.paged_attention(q, kp, vp, table, lengths, out=q)
    assert o2 is q and q._version > version and torch.equal(o, q) and torch.equal(lse, lse2)


def test_decoding_under_inference_mode():
    with torch.inference_mode():
        kp, vp, table, lengths = cache([40, 17], 2, 64, BF16)
        k, v = queries(2, 2, 64, BF16, 5), queries(2, 2, 64, BF16, 6)
        nf4.paged_append(k, v, kp, vp, table, lengths)
        check(queries(2, 4, 64, BF16), kp, vp, table, lengths)
        last = ref.slots_of(table[0], 40, 16)
        assert torch.equal(kp[last[0][-1], last[1][-1]], k[0])


def test_refusals():
    """Every argument that does not fit is refused with a message, before anything is launched."""
    kp, vp, table, lengths = cache([20, 5], 2, 64, BF16)
    q, k, v = queries(2, 4, 64, BF16), queries(2, 2, 64, BF16), queries(2, 2, 64, BF16)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    before = nf4.path_counters()["total"]

    def attend(message, q=q, kp=kp, vp=vp, table=table, lengths=lengths, **kw):
        with pytest.raises(ValueError, match=message):
            nf4.paged_attention(q, kp, vp, table, lengths, **kw)

    def append(message, k=k, v=v, kp=kp, vp=vp, table=table, lengths=lengths, cu=None):
        with pytest.raises(ValueError, match=message):
            nf4.paged_append(k, v, kp, vp, table, lengths, cu)

    for f in (attend, append):
        f("pages", kp=kp[0])
        f("pages", vp=vp[:, :3])
        f("pages", vp=vp.half())
        f("fp32, bf16 or fp16", kp=kp.double(), vp=vp.double())
        f("unit stride", kp=kp.transpose(2, 3).contiguous().transpose(2, 3))
        f("lengths", lengths=lengths.long())
        f("lengths", lengths=torch.zeros(4, dtype=torch.int32, device=DEV)[::2])
        f("page_table", table=table[:1])
        f("page_table", table=table.long())
        f("page_table", table=table.T.contiguous().T)
        f("CUDA", table=table.cpu())
        f("CUDA", lengths=lengths.cpu())
    attend("q must be", q=q.half())
    attend("q must be", q=q[..., :32])
    attend("does not fit", q=q[:1])
    attend("does not fit", q=queries(2, 3, 64, BF16))
    attend("does not fit", q=q[:, :0])
    attend("unit stride", q=q.transpose(1, 2).contiguous().transpose(1, 2))
    attend("out must", out=torch.zeros(2, 2, 64, dtype=BF16, device=DEV))
    attend("out must be", out=torch.zeros(2, 4, 64, device=DEV))
    attend("storage", out=torch.zeros(4, 64, dtype=BF16, device=DEV).expand(2, 4, 64))
    append("k must be", k=queries(2, 4, 64, BF16))
    append("v must be", v=v.half())
    append("rows of keys", k=queries(3, 2, 64, BF16))
    append("rows of keys", k=queries(3, 2, 64, BF16), v=queries(3, 2, 64, BF16))
    append("cu_seqlens", cu=cu[:2])
    append("cu_seqlens", cu=cu.long())
    append("cu_seqlens", cu=cu.cpu())
    append("share storage", kp=kp[:1].expand(kp.shape))
    append("share storage", vp=vp[:, :1].expand(vp.shape))
    assert nf4.path_counters()["total"] == before


def test_repeats_bit_for_bit_and_on_another_stream():
    kp, vp, table, lengths = cache([5000, 17, 0, 900], 4, 128, BF16)
    q = queries(4, 16, 128, BF16)
    first = nf4.paged_attention(q, kp, vp, table, lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = [nf4.paged_attention(q, kp, vp, table, lengths) for _ in range(5)]
    here = [nf4.paged_attention(q, kp, vp, table, lengths) for _ in range(5)]  # at the same time
    torch.cuda.current_stream().wait_stream(side)
    for got in second + here:
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_graph_of_a_decoding_step(dtype):
    """A captured append and attention, replayed with the lengths growing on the device; two graphs in turn."""
    Hk, D, n = 2, 64, 3
    kp, vp, table, lengths = cache([200, 130, 90], Hk, D, dtype)
    start = torch.tensor([3, 0, 17], dtype=torch.int32, device=DEV)
    q, k, v = queries(n, 8, D, dtype), queries(n, Hk, D, dtype, 2), queries(n, Hk, D, dtype, 3)
    lengths.copy_(start)

    def step():
        nf4.paged_append(k, v, kp, vp, table, lengths)
        return nf4.paged_attention(q, kp, vp, table, lengths)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()
        graphs.append((g, held))
    for i in range(70):
        lengths += (start > 0).int()
        for x, s in ((q, 10 + i), (k, 100 + i), (v, 200 + i)):
            x.copy_(queries(*x.shape, dtype, s))
        g, held = graphs[i % 2]
        g.replay()
        if i % 23 == 0 or i == 69:
            lens = lengths.tolist()
            want, wl, mag, smag = ref.paged_attention(q, kp, vp, table, lens, D ** -0.5)
            bo, _ = ref.paged_bounds(want, wl, mag, smag, lens, D, dtype)
            assert ((held[0].double() - want).abs() <= bo).all()
            last = ref.slots_of(table[2], lens[2], 16)
            assert torch.equal(kp[last[0][-1], last[1][-1]], k[2]) and torch.equal(vp[last[0][-1], last[1][-1]], v[2])


# ------------------------------------------------------------------------------- append --

def plain_append(k, v, kp, vp, table, lengths, cu):
    page = kp.shape[1]
    for i, m in enumerate(lengths):
        rows = range(i, i + 1) if cu is None else range(cu[i], cu[i + 1])
        if m == 0:
            continue
        for j, r in enumerate(rows):
            pos = m - len(rows) + j
            kp[table[i, pos // page], pos % page], vp[table[i, pos // page], pos % page] = k[r], v[r]


@pytest.mark.parametrize("new,before", [([1], [0]), ([17], [30]), ([5, 0, 64, 1, 200], [0, 9, 16, 99, 3]), ([0, 0, 3], [0, 5, 0]),
                                        ([3] * 50, list(range(50))), ([2500, 2501], [1, 0])])
@pytest.mark.parametrize("dtype,D,page,order", [(BF16, 128, 16, "token"), (F32, 37, 24, "token"), (F16, 72, 5, "head"), (BF16, 7, 64, "head")])
def test_append_of_prompts(new, before, dtype, D, page, order):
    lens = [a + b for a, b in zip(new, before)]
    kp, vp, table, lengths = cache(lens, 2, D, dtype, page=page, order=order)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    k, v = (queries(cu[-1] + 4, 2, D, dtype, s) for s in (5, 6))  # four rows past the last sequence
    k2, v2 = kp.clone(), vp.clone()
    plain_append(k, v, k2, v2, table.cpu(), lens, cu)
    nf4.paged_append(k, v, kp, vp, table, lengths, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert torch.equal(kp, k2) and torch.equal(vp, v2)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F32, 3)])
def test_append_of_single_tokens(dtype, D):
    lens = [1, 0, 16, 17, 333, 0]
    kp, vp, table, lengths = cache(lens, 3, D, dtype)
    fused = queries(6, 6, D, dtype, 8)  # keys and values as views of one projection's output
    k, v = fused[:, :3], fused[:, 3:]
    k2, v2 = kp.clone(), vp.clone()
    plain_append(k, v, k2, v2, table.cpu(), lens, None)
    version = kp._version
    nf4.paged_append(k, v, kp, vp, table, lengths)
    assert torch.equal(kp, k2) and torch.equal(vp, v2) and kp._version > version


def test_append_refuses_bad_offsets_on_the_device():
    """Offsets that descend or leave the rows, and more new rows than a sequence has tokens: recorded, and nothing out of
    place is written."""
    kp, vp, table, lengths = cache([40, 40], 2, 64, BF16)
    k, v = queries(20, 2, 64, BF16, 5), queries(20, 2, 64, BF16, 6)
    for cu, lens in (([0, 15, 10], [40, 40]), ([0, 10, 30], [40, 40]), ([-3, 10, 20], [40, 40]), ([0, 10, 20], [40, 3])):
        k2, v2 = kp.clone(), vp.clone()
        nf4.paged_append(k, v, k2, v2, table, torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert nf4.device_status(clear=True) == BAD_OFFSETS
        free = torch.ones(kp.shape[0], dtype=torch.bool, device=DEV)
        free[table[table >= 0].long()] = False
        assert torch.equal(k2[free], kp[free]) and torch.equal(v2[free], vp[free])


def test_append_then_attend_equals_the_attention_of_a_prompt():
    """Token by token through the cache, and the whole prompt through nf4_attention."""
    T, Hq, Hk, D = 67, 8, 2, 64
    q, k, v = queries(T, Hq, D, BF16), queries(T, Hk, D, BF16, 2), queries(T, Hk, D, BF16, 3)
    want = nf4.nf4_attention(q, k, v)
    kp, vp, table, lengths = cache([T], Hk, D, BF16)
    lengths.fill_(60)
    nf4.paged_append(k[:60], v[:60], kp, vp, table, lengths, torch.tensor([0, 60], dtype=torch.int32, device=DEV))
    for t in range(60, T):
        lengths += 1
        nf4.paged_append(k[t:t + 1], v[t:t + 1], kp, vp, table, lengths)
        o, _ = nf4.paged_attention(q[t:t + 1], kp, vp, table, lengths)
        # each side is one rounding of the result and of the weights from it
        assert ((o[0].double() - want[t].double()).abs() <= 2 * 2.0 ** -8 * want[t].double().abs() + 2.0 ** -8 * v[:t + 1].abs().amax().double()).all()


@pytest.mark.parametrize("dtype,D,order", [(BF16, 64, "token"), (F16, 72, "head"), (F32, 3, "token")])
def test_append_past_the_table_overwrites_nothing(dtype, D, order):
    """A length of more tokens than the table's row names: a row whose position has no page is not written, the others go
    to their own positions, and no older token is lost.  A negative length has no new rows."""
    kp, vp, table, _ = cache([32, 32, 32, 32], 2, D, dtype, order=order, extra_pages=0)  # two pages of 16 a sequence, all in use
    for new, lens in ((None, [33, 20, 2 ** 31 - 1, 32]), ([6, 1, 0, 32], [35, 33, 40, 32]), ([3, 40, 5, 2], [-1, 50, 32, -2 ** 31]),
                      ([1, 1, 1, 1], [32, 33, 1, 48])):
        cu = [sum(new[:i]) for i in range(5)] if new else None
        k, v = (queries(cu[-1] if new else 4, 2, D, dtype, s) for s in (5, 6))
        wk, wv = kp.clone(), vp.clone()
        for i, m in enumerate(lens):
            rows = list(range(cu[i], cu[i + 1])) if new else [i]
            for j, r in enumerate(rows):
                pos = m - len(rows) + j
                if 0 <= pos < 32:
                    page = table[i, pos // 16]
                    wk[page, pos % 16], wv[page, pos % 16] = k[r], v[r]
        gk, gv = kp.clone(), vp.clone()
        nf4.paged_append(k, v, gk, gv, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                         None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert nf4.device_status(clear=True) == BAD_OFFSETS
        assert torch.equal(gk, wk) and torch.equal(gv, wv), lens


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_attention_values_without_a_weight_count_nothing(dtype):
    """Tokens of score -inf: the largest finite values there add nothing to the answer of the others."""
    D = 64
    kp, vp, table, lengths = cache([200], 1, D, dtype, seed=5)
    q = queries(1, 4, D, dtype).abs() + 0.1
    dead = torch.zeros(200, dtype=torch.bool, device=DEV)
    dead[:70] = dead[130:150] = True
    page, slot = ref.slots_of(table[0], 200, 16)
    kp[page[dead], slot[dead], 0] = -math.inf
    vp[page[dead], slot[dead], 0] = torch.finfo(dtype).max
    o, lse = nf4.paged_attention(q, kp, vp, table, lengths)
    live = (~dead).nonzero().flatten()
    one = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    want, wl, mag, smag = ref.paged_attention(q, kp[page[live], slot[live]][None], vp[page[live], slot[live]][None], one, [live.numel()],
                                              D ** -0.5)
    bo, bl = ref.paged_bounds(want, wl, mag, smag, [200], D, dtype)
    assert ((o.double() - want).abs() <= bo).all() and ((lse.double() - wl).abs() <= bl).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F16, 64), (F32, 64), (BF16, 37), (F32, 37)])
def test_attention_sums_of_the_largest_values(dtype, D):
    """Values near the type's largest, of which a few add up past fp32's range: their mean is a number.  And such values at
    tokens that lose all their weight to later ones."""
    kp, vp, table, lengths = cache([200, 3, 0, 3000], 2, D, dtype, seed=D)
    q = queries(4, 8, D, dtype)
    big = 0.9 * torch.finfo(dtype).max
    check(q, kp, torch.full_like(vp, big), table, lengths)
    check(0 * q, kp, torch.full_like(vp, -big), table, lengths)
    check(q, kp, (vp.sign() * big).to(dtype), table, lengths)
    page, slot = (torch.cat(t) for t in zip(*(ref.slots_of(table[i], 70, 16) for i in (0, 3))))
    kp[page, slot], vp[page, slot] = -3e4, big
    check(q.abs() + 0.1, kp, vp, table, lengths)


def test_tensors_that_require_a_gradient_are_refused():
    """The calls have no gradients: under grad mode they refuse what asks for one, and take it under no_grad or detached."""
    kp, vp, table, lengths = cache([20, 5], 2, 64, BF16)
    q, k, v = queries(2, 4, 64, BF16), queries(2, 2, 64, BF16, 2), queries(2, 2, 64, BF16, 3)
    before = nf4.path_counters()["total"]

    def leaf(t):
        return t.clone().requires_grad_()

    for args in ((leaf(q), kp, vp), (q, leaf(kp), vp), (q, kp, leaf(vp)), (leaf(q) * 2, kp, vp)):
        with pytest.raises(ValueError, match="no gradients"):
            nf4.paged_attention(*args, table, lengths)
    with pytest.raises(ValueError, match="no gradients"):
        nf4.paged_attention(q, kp, vp, table, lengths, out=leaf(q))
    for args in ((leaf(k), v, kp, vp), (k, leaf(v), kp, vp), (k, v, leaf(kp), vp), (k, v, kp, leaf(vp))):
        with pytest.raises(ValueError, match="no gradients"):
            nf4.paged_append(*args, table, lengths)
    assert nf4.path_counters()["total"] == before
    want = nf4.paged_attention(q, kp, vp, table, lengths)
    with torch.no_grad():
        nf4.paged_append(leaf(k), leaf(v), kp.clone(), vp.clone(), table, lengths)
        got = nf4.paged_attention(leaf(q), kp, vp, table, lengths)
    also = nf4.paged_attention(leaf(q).detach(), kp, vp, table, lengths)
    for a, b, c in zip(want, got, also):
        assert torch.equal(a, b) and torch.equal(a, c) and not b.requires_grad


def test_memory_that_a_call_both_reads_and_writes():
    """out in memory that other CTAs read, and keys and values in one place, are refused; out and q, and keys and values,
    side by side in one buffer are taken."""
    Hq, Hk, D = 8, 2, 64
    kp, vp, table, lengths = cache([131, 40, 70], Hk, D, BF16)
    q, k, v = queries(3, Hq, D, BF16), queries(3, Hk, D, BF16, 2), queries(3, Hk, D, BF16, 3)
    want = nf4.paged_attention(q, kp, vp, table, lengths)
    before = nf4.path_counters()["total"]
    rows, held = torch.zeros(4, Hq, D, dtype=BF16, device=DEV), torch.zeros(3 * Hq * D + 8, dtype=BF16, device=DEV)
    for a, out in ((rows[:3], rows[1:]), (rows[1:], rows[:3]), (held[:-8].view(3, Hq, D), held[8:].view(3, Hq, D)),
                   (q, q.view(Hq, 3, D).transpose(0, 1)), (q, kp.view(-1)[5 * D:][:q.numel()].view(q.shape)),
                   (q, vp.view(-1)[:q.numel()].view(q.shape))):
        with pytest.raises(ValueError, match="share no storage"):
            nf4.paged_attention(a, kp, vp, table, lengths, out=out)
    flat = torch.cat([kp.flatten(), kp.flatten()])
    for apart in (0, 8, 64, kp.numel() - 8):
        with pytest.raises(ValueError, match="share storage"):
            nf4.paged_append(k, v, flat[:kp.numel()].view(kp.shape), flat[apart:apart + kp.numel()].view(kp.shape), table, lengths)
    assert nf4.path_counters()["total"] == before
    both = torch.zeros(3, 2, Hq, D, dtype=BF16, device=DEV)
    both[:, 0] = q
    got = nf4.paged_attention(both[:, 0], kp, vp, table, lengths, out=both[:, 1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(both[:, 0], q)
    assert torch.equal(nf4.paged_attention(both[:, 0], kp, vp, table, lengths, out=both[:, 0])[0], want[0])
    wk, wv = kp.clone(), vp.clone()
    nf4.paged_append(k, v, wk, wv, table, lengths)
    for dim in range(4):
        gk, gv = torch.stack([kp, vp], dim).unbind(dim)
        nf4.paged_append(k, v, gk, gv, table, lengths)
        assert torch.equal(gk, wk) and torch.equal(gv, wv), dim


@pytest.mark.parametrize("Hq,Hk,D", [(4, 4, 4), (8, 2, 64), (16, 2, 80), (5, 1, 128), (9, 1, 200), (8, 2, 256)])
def test_attention_fp32_rows_and_their_kernel(Hq, Hk, D):
    """Aligned fp32 rows go through the rings, everything else of fp32 to the kernel of any layout; one call counts once."""
    kp, vp, table, lengths = cache([331, 7, 64, 0, 150], Hk, D, F32, seed=D)
    q = queries(5, Hq, D, F32)

    def path(call, rings):
        before = nf4.path_counters()
        call()
        after = nf4.path_counters()
        moved = {name: after[name] - before[name] for name in after if after[name] != before[name]}
        assert moved == dict(paged_attention_any=1, total=1, **({"paged_attention_f32": 1} if rings else {}))

    def shifted(t):
        return torch.zeros(t.numel() + 1, device=DEV)[1:].view(t.shape).copy_(t)

    path(lambda: check(q, kp, vp, table, lengths), True)
    path(lambda: check(q, kp, vp, table, lengths, out=shifted(q)), True)  # only what is read in pieces has to be aligned
    for args in ((shifted(q), kp, vp), (q, shifted(kp), vp), (q, kp, shifted(vp))):
        path(lambda: check(*args, table, lengths), False)
    if D > 4:
        path(lambda: check(q[..., :-1], kp[..., :-1], vp[..., :-1], table, lengths), False)


@pytest.mark.parametrize("page", [3, 24, 100])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("D,dtype", [(128, BF16), (136, F16), (256, BF16), (132, F32), (200, F32), (256, F32)])
def test_attention_pages_of_wide_heads(page, order, D, dtype):
    """Pages that no tile fits, for rows that take a warp's whole copy or two."""
    kp, vp, table, lengths = cache([700, 99, 1, 0, 333], 2, D, dtype, page=page, order=order, seed=page)
    check(queries(5, 8, D, dtype), kp, vp, table, lengths, path="paged_attention_f32" if dtype == F32 else "paged_attention")
