"""Host checks of the training-block entry points: wrong arguments are refused before any launch (no GPU needed), and
the optimiser's level maps."""
import ctypes

import pytest
import torch

from bit_nf4_quantized_linear_gb300 import _lib, block_ops, build, codebooks

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
X = ctypes.c_void_p(0x1000)  # never read: every call here is refused or empty


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def norm(**kw):
    d = _lib.nf4_norm_residual(0x1000, 64, 0x1000, 64, None, 0, 0x1000, 0x1000, 4, 64, _lib.GATE_NONE, _lib.DTYPE_BF16, 1.0, 1e-6)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def attn(**kw):
    d = _lib.nf4_attention(0x1000, 0x1000, 0x1000, 256, 64, 128, 64, 128, 64, None, 0, 10, 4, 2, 64, _lib.DTYPE_BF16, 0.125)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def test_norm_refusals(L):
    def fwd(d, z=X, ldz=64, h=X, ldh=64):
        return L.nf4_norm_residual_fwd(d, z, ldz, h, ldh, X, None)

    assert fwd(None) == INVALID
    for kw in (dict(T=-1), dict(H=0), dict(dtype=3), dict(gate_kind=3), dict(gate_kind=_lib.GATE_CHANNEL), dict(y=None),
               dict(ld_y=63), dict(ld_residual=63), dict(eps=-1.0), dict(eps=float("nan")), dict(w_pre=None),
               dict(gate_kind=_lib.GATE_TOKEN, gate=0x1000, ld_gate=10)):
        assert fwd(norm(**kw)) == INVALID, kw
    assert fwd(norm(), ldz=63) == INVALID and fwd(norm(), ldh=63) == INVALID
    assert fwd(norm(y=0x1001)) == ALIGN and fwd(norm(w_post=0x1002)) == ALIGN
    assert fwd(norm(), z=ctypes.c_void_p(0x1001)) == ALIGN
    assert fwd(norm(T=2 ** 31)) == SHAPE and fwd(norm(H=2 ** 31, ld_y=2 ** 31, ld_residual=2 ** 31)) == SHAPE
    assert fwd(norm(T=0, y=None)) == 0

    def bwd(d, gz=X, gh=X, gr=X, gw_post=X, ggate=None, gw_pre=X):
        return L.nf4_norm_residual_bwd(d, X, gz, 64, gh, 64, X, 64, gr, 64, gw_post, ggate, 64, gw_pre, None, 0, None)

    assert bwd(norm(w_pre=None)) == INVALID and bwd(norm(w_post=None)) == INVALID
    assert bwd(norm(), ggate=X) == INVALID and bwd(norm(residual=None)) == INVALID


def test_attention_refusals(L):
    def fwd(d, o=X, lse=X):
        return L.nf4_attention_fwd(d, o, 256, 64, lse, None)

    assert fwd(None) == INVALID
    for kw in (dict(T=-1), dict(Hk=0), dict(Hq=0), dict(Hq=5), dict(D=0), dict(dtype=-1), dict(q=None), dict(v=None),
               dict(cu_seqlens=0x1000, nseq=0)):
        assert fwd(attn(**kw)) == INVALID, kw
    for kw in (dict(D=257), dict(T=2 ** 31), dict(Hq=65536), dict(cu_seqlens=0x1000, nseq=2 ** 31)):
        assert fwd(attn(**kw)) == SHAPE, kw
    assert fwd(attn(k=0x1001)) == ALIGN and fwd(attn(cu_seqlens=0x1002, nseq=1)) == ALIGN
    assert fwd(attn(), o=None) == INVALID and fwd(attn(), lse=None) == INVALID
    assert fwd(attn(T=0, q=None), o=None, lse=None) == 0

    def bwd(d, ws=None, n=0, gq=X):
        return L.nf4_attention_bwd(d, X, 256, 64, X, X, 256, 64, gq, 256, 64, X, 128, 64, X, 128, 64, ws, n, None)

    assert bwd(attn()) == WORKSPACE and bwd(attn(), X, 8) == WORKSPACE and bwd(attn(), gq=None) == INVALID
    assert bwd(attn(T=0)) == 0


def test_adamw_refusals(L):
    def step(n=10, count=1, dtype=0, bits=8, levels=X, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, **kw):
        tab = (_lib.nf4_adamw_tensor * 1)()
        for f in ("param", "grad", "m", "v", "m_absmax", "v_absmax"):
            setattr(tab[0], f, 0x1000)
        tab[0].n = n
        for k, v in kw.items():
            setattr(tab[0], k, v)
        return L.nf4_adamw_step(tab, count, dtype, bits, levels, levels, lr, b1, b2, eps, wd, t, None, None)

    for kw in (dict(count=-1), dict(dtype=3), dict(bits=4), dict(levels=None), dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0),
               dict(b2=-0.1), dict(eps=-1.0), dict(wd=-1.0), dict(t=0), dict(n=-1), dict(param=None), dict(grad=None), dict(m=None),
               dict(v=None), dict(m_absmax=None), dict(v_absmax=None)):
        assert step(**kw) == INVALID, kw
    assert step(param=0x1002) == ALIGN and step(bits=32, m=0x1001) == ALIGN
    assert L.nf4_adamw_step(None, 1, 0, 32, None, None, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None) == INVALID
    assert L.nf4_adamw_state_values(None, X, X, X, X, X, 5, X, X, None) == INVALID
    assert L.nf4_adamw_state_values(X, X, X, X, X, X, -1, X, X, None) == INVALID
    assert L.nf4_adamw_state_values(None, None, None, None, None, None, 0, None, None, None) == 0


def test_no_cpu_path():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: block_ops.attention_fwd(x, x, x), lambda: block_ops.norm_residual_fwd(x[:, 0], w_pre=torch.ones(64)),
                 lambda: block_ops.adamw_state([x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_unsigned_map():
    """256 ascending levels from an exact 0 to an exact 1, with twice the signed map's fractions in each decade."""
    u, s = codebooks.dynamic_code8_unsigned().double(), codebooks.dynamic_code8().double()
    assert u.numel() == 256 and (u[1:] > u[:-1]).all() and u[0] == 0 and u[-1] == 1
    for e in range(7):
        lo, hi = 10.0 ** (e - 7), 10.0 ** (e - 6)
        assert ((u > lo) & (u < hi)).sum() == 2 ** (e + 1) and ((s > lo) & (s < hi)).sum() == 2 ** e
