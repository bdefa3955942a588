"""Host checks of the paged cache and the router: wrong arguments are refused before any launch (no GPU needed)."""
import ctypes
import itertools

import pytest
import torch

from bit_nf4_quantized_linear_gb300 import _lib, build, decode_ops, route_ops

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
X = ctypes.c_void_p(0x1000)  # never read: every call here is refused or empty


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def cache(**kw):
    c = _lib.nf4_paged_cache(0x1000, 0x1000, 2048, 128, 64, 2048, 128, 64, 0x1000, 4, 0x1000, 3, 10, 4, 16, 2, 64, _lib.DTYPE_BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def route(**kw):
    d = _lib.nf4_route(0x1000, 64, 10, None, None, 64, 8, _lib.DTYPE_F32, 0, 1, 1, 1, 0, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


BAD_CACHES = [dict(dtype=3), dict(nseq=-1), dict(pages=-1), dict(max_pages=-1), dict(page_size=0), dict(Hk=0), dict(D=0), dict(ld_table=-1),
              dict(lengths=None), dict(table=None), dict(k=None), dict(v=None)]


def test_structs_are_packed_as_the_header_lays_them_out():
    assert decode_ops._CACHE.size == ctypes.sizeof(_lib.nf4_paged_cache)
    assert route_ops._ROUTE.size == ctypes.sizeof(_lib.nf4_route)
    packed = decode_ops._CACHE.pack(*range(1, 19))
    c = _lib.nf4_paged_cache.from_buffer_copy(packed)
    assert [getattr(c, n) for n, _ in c._fields_] == list(range(1, 19))
    packed = route_ops._ROUTE.pack(*range(1, 14), 2.5)
    d = _lib.nf4_route.from_buffer_copy(packed)
    assert [getattr(d, n) for n, _ in d._fields_] == [*range(1, 14), 2.5]


def test_append_refusals(L):
    def append(c, k=X, v=X, cu=None, T=3):
        return L.nf4_paged_append(c, k, 128, 64, v, 128, 64, cu, T, None)

    assert append(None) == INVALID
    for kw in BAD_CACHES:
        assert append(cache(**kw)) == INVALID, kw
    for kw in (dict(nseq=2 ** 31), dict(pages=2 ** 31), dict(Hk=65536), dict(D=257), dict(max_pages=2 ** 27 + 1)):
        assert append(cache(**kw), cu=X) == SHAPE, kw
    for kw in (dict(k=0x1001), dict(v=0x1001), dict(table=0x1002), dict(lengths=0x1001)):
        assert append(cache(**kw)) == ALIGN, kw
    assert append(cache(), T=4) == INVALID and append(cache(), T=-1, cu=X) == INVALID and append(cache(), T=2 ** 31, cu=X) == SHAPE
    assert append(cache(), k=None) == INVALID and append(cache(), v=None) == INVALID
    assert append(cache(), k=ctypes.c_void_p(0x1001)) == ALIGN and append(cache(), cu=ctypes.c_void_p(0x1002)) == ALIGN
    assert append(cache(), None, None, X, 0) == 0 and append(cache(nseq=0, lengths=None), None, None, None, 0) == 0


def test_attention_refusals(L):
    def attend(c, q=X, Hq=8, o=X, lse=X, ws=X, n=1 << 40):
        return L.nf4_paged_attention(c, q, 512, 64, Hq, 0.125, o, 512, 64, lse, ws, n, None)

    assert attend(None) == INVALID
    for kw in BAD_CACHES:
        assert attend(cache(**kw)) == INVALID, kw
    for Hq in (0, -8, 7):
        assert attend(cache(), Hq=Hq) == INVALID
    assert attend(cache(), Hq=65536) == SHAPE
    assert attend(cache(), q=None) == INVALID and attend(cache(), o=None) == INVALID
    assert attend(cache(), q=ctypes.c_void_p(0x1001)) == ALIGN and attend(cache(), lse=ctypes.c_void_p(0x1002)) == ALIGN
    assert attend(cache(nseq=0), None, 8, None, None, None, 0) == 0


BAD_ROUTES = [dict(dtype=-1), dict(T=-1), dict(E=0), dict(k=0), dict(ld=63), dict(score=2), dict(groups=0), dict(groups=5), dict(top_groups=0),
              dict(top_groups=2), dict(group_top=0), dict(group_top=3), dict(k=65), dict(groups=8, top_groups=1, k=9), dict(logits=None)]


def test_route_refusals(L):
    def fwd(d, experts=X, weights=X, tables=(X, X, X, X)):
        return L.nf4_route_fwd(d, experts, weights, *tables, X, 1 << 40, None)

    assert fwd(None) == INVALID
    for kw in BAD_ROUTES:
        assert fwd(route(**kw)) == INVALID, kw
    for kw in (dict(E=513, ld=513), dict(k=33), dict(groups=64, top_groups=64), dict(T=2 ** 28)):
        assert fwd(route(**kw)) == SHAPE, kw
    assert fwd(route(logits=0x1002)) == ALIGN and fwd(route(bias=0x1001)) == ALIGN
    assert fwd(route(), experts=None) == INVALID and fwd(route(), weights=None) == INVALID
    for i in range(1, 4):
        assert fwd(route(), tables=[None if j == i else X for j in range(4)]) == INVALID
    assert fwd(route(), tables=(None, None, None, X)) == INVALID
    assert fwd(route(), tables=(X, X, ctypes.c_void_p(0x1002), X)) == ALIGN

    def bwd(d, experts=X, rows=X, gw=X, gr=X, g=X, ld=64):
        return L.nf4_route_bwd(d, experts, rows, gw, gr, g, ld, None)

    assert bwd(None) == INVALID and bwd(route(), ld=63) == INVALID and bwd(route(), rows=None) == INVALID
    assert bwd(route(), experts=None) == INVALID and bwd(route(), g=None) == INVALID
    assert bwd(route(), g=ctypes.c_void_p(0x1002)) == ALIGN and bwd(route(), gr=ctypes.c_void_p(0x1001)) == ALIGN
    for kw in BAD_ROUTES:
        assert bwd(route(**kw)) == INVALID, kw
    assert bwd(route(T=0, logits=None), None, None, None, None, None) == 0


def test_no_cpu_path():
    p, t = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    n, q = torch.ones(1, dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: decode_ops.paged_append(q[:, :2], q[:, :2], p, p, t, n), lambda: decode_ops.paged_attention(q, p, p, t, n),
                 lambda: route_ops.route_experts(torch.zeros(4, 8), 2),
                 lambda: route_ops.route_experts_bwd(torch.zeros(4, 8), route_ops.Routes(torch.zeros(4, 2, dtype=torch.int32), *[None] * 5))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_slots_that_share_storage_are_recognised():
    """Never called free where two addresses are equal; free for the layouts that pages have."""
    share = decode_ops._slots_share
    assert not share((5, 16, 2, 64), (2048, 128, 64, 1)) and not share((5, 16, 2, 64), (2048, 64, 1024, 1))
    assert not share((5, 16, 2, 64), (4096, 128, 64, 1)) and not share((1, 16, 1, 64), (0, 64, 0, 1))
    for shape in ((2, 3, 2, 2), (1, 2, 3, 1), (3, 1, 2, 2)):
        for a in range(0, 13, 2):
            for b in range(0, 13):
                for c in range(0, 9):
                    at = [i * a + j * b + h * c + d for i in range(shape[0]) for j in range(shape[1]) for h in range(shape[2]) for d in range(shape[3])]
                    assert share(shape, (a, b, c, 1)) or len(set(at)) == len(at), (shape, a, b, c)


def test_route_tables_that_do_not_fit_the_activations_are_refused():
    """What the dispatch and the combine would read past their inputs or as other types, before any pointer is taken."""
    from bit_nf4_quantized_linear_gb300 import ops
    x, t = torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(5, 2, dtype=torch.int32)
    ops._check_token_rows("op", t, x, 5)
    ops._check_token_rows("op", t, x)
    for bad in (t.long(), t.float(), t[:, 0], t[None], t.T.contiguous().T, torch.zeros(5, 4, dtype=torch.int32)[:, ::2]):
        with pytest.raises(ValueError, match="op: token_rows must be"):
            ops._check_token_rows("op", bad, x)
    for tokens in (0, 4, 6):
        with pytest.raises(ValueError, match="op: token_rows of 5 tokens"):
            ops._check_token_rows("op", t, x, tokens)
    with pytest.raises(ValueError, match="op: token_rows on meta"):
        ops._check_token_rows("op", t.to("meta"), x)


def test_grouped_epilogue_of_the_input_gradient(L):
    """nf4_grouped_dgrad_ep takes zero_rest alone; the flag lies in what was padding of the struct."""
    assert ctypes.sizeof(_lib.nf4_epilogue) == 24 and _lib.nf4_epilogue(None, None, 1).zero_rest == 0
    w = _lib.nf4_weight(0x1000, 0x1000, None, None, None, 0x1000, None, 384, 256, 64, 256, 0, 4)

    def dgrad(ep, T=10, offsets=X):
        return L.nf4_grouped_dgrad_ep(X, offsets, 3, T, 128, ctypes.byref(w), 128, ep, X, 256, None)

    for ep in (_lib.nf4_epilogue(0x1000, None, 0, 1), _lib.nf4_epilogue(None, 0x1000, 0, 1), _lib.nf4_epilogue(None, None, 1, 1)):
        assert dgrad(ctypes.byref(ep)) == INVALID
    assert dgrad(None, offsets=None) == INVALID and dgrad(ctypes.byref(_lib.nf4_epilogue(None, None, 0, 1)), T=-1) == INVALID
    assert dgrad(ctypes.byref(_lib.nf4_epilogue(None, None, 0, 1)), T=0) == 0 and dgrad(None, T=0) == 0


def test_tensors_that_meet_in_memory_are_recognised():
    """Exactly the common addresses, for tensors of one layout; never called free where two addresses are equal."""
    meet = decode_ops._meet

    def at(shape, stride, first=0):
        return {first + sum(i * s for i, s in zip(index, stride)) for index in itertools.product(*map(range, shape))}

    for shape, stride in (((2, 3, 2, 2), (12, 4, 2, 1)), ((2, 3, 2, 2), (24, 8, 2, 1)), ((2, 3, 2, 2), (24, 2, 12, 1)), ((3, 2, 4), (20, 4, 1)),
                          ((3, 2, 4), (5, 30, 1)), ((1, 3, 2), (0, 7, 1)), ((4, 3), (6, 1))):
        one = at(shape, stride)
        for apart in range(-90, 91):
            assert meet(shape, stride, stride, apart) == bool(one & at(shape, stride, apart)), (shape, stride, apart)
    for one, other in (((12, 4, 2, 1), (24, 4, 2, 1)), ((12, 4, 2, 1), (12, 2, 6, 1)), ((0, 4, 2, 1), (12, 4, 2, 1)), ((4, 4, 2, 1), (4, 4, 2, 1))):
        for apart in range(-70, 71):
            assert meet((2, 3, 2, 2), one, other, apart) or not at((2, 3, 2, 2), one) & at((2, 3, 2, 2), other, apart)
    assert not meet((0, 2, 4), (8, 4, 1), (8, 4, 1), 0)
    w = decode_ops._writable
    token, pages = (2048, 128, 64, 1), (5, 16, 2, 64)
    assert w(pages, token, token, 5 * 2048) and w(pages, token, token, -5 * 2048) and not w(pages, token, token, 0)
    assert not w(pages, token, token, 2048) and w(pages, (4096, 128, 64, 1), (4096, 128, 64, 1), 2048)  # whole pages in turn
    assert w(pages, (4096, 256, 64, 1), (4096, 256, 64, 1), 128) and w(pages, (4096, 256, 128, 1), (4096, 256, 128, 1), 64)
    assert not w(pages, (4096, 256, 128, 1), (4096, 256, 128, 1), 32) and not w(pages, token, (2048, 64, 1024, 1), 64)
