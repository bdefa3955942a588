"""64-bit definitions of the training-block operators, with the magnitudes that their
rounding-error bounds need.  Independent of the library: plain torch in float64."""
import math

import torch

# Largest relative error of one rounding to each type.
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# Largest error of a rounding to a subnormal: half the smallest spacing.
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def bounds_of(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def attention(q, k, v, cu, scale, go=None):
    """(outputs, magnitudes): o, lse and with go the gradients gq, gk, gv in float64.  A magnitude is the sum of the
    absolute values of the terms whose rounding the output sees: for o the probabilities times the values; for the
    gradients the probabilities or score gradients times their operand, with the score gradients' own error from a
    rounded o."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    q, k, v = q.double(), k.double(), v.double()
    go = None if go is None else go.double()
    out = {"o": torch.zeros_like(q), "lse": torch.full((Hq, T), -math.inf, dtype=torch.float64, device=q.device)}
    mag = {"o": torch.zeros_like(q)}
    if go is not None:
        for name, x in (("gq", q), ("gk", k), ("gv", v)):
            out[name], mag[name] = torch.zeros_like(x), torch.zeros_like(x)
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        if n <= 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
        for h in range(Hq):
            qs, ks, vs = q[a:b, h], k[a:b, h // G], v[a:b, h // G]
            s = (qs @ ks.T * scale).masked_fill(hidden, -math.inf)
            out["lse"][h, a:b] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            o = p @ vs
            out["o"][a:b, h], mag["o"][a:b, h] = o, p @ vs.abs()
            if go is None:
                continue
            g = go[a:b, h]
            dp = g @ vs.T
            delta = (g * o).sum(1, keepdim=True)
            ds = p * (dp - delta) * scale
            ds_mag = ds.abs() + p * (g.abs() * o.abs()).sum(1, keepdim=True) * abs(scale)
            out["gq"][a:b, h], mag["gq"][a:b, h] = ds @ ks, ds_mag @ ks.abs()
            out["gk"][a:b, h // G] += ds.T @ qs
            mag["gk"][a:b, h // G] += ds_mag.T @ qs.abs()
            out["gv"][a:b, h // G] += p.T @ g
            mag["gv"][a:b, h // G] += p.T @ g.abs()
    return out, mag


def attention_bound(name, ref, mag, dtype, smax):
    """Error bound of an attention output: one rounding of the result, one of each probability (or score gradient)
    to the operand type, and the fp32 arithmetic: products summed over the head, and exponentials of scores up to
    smax in size, each with a relative error of a few units of 2^-24 per unit of score."""
    u = UNIT[dtype] if dtype != torch.float32 else 0.0
    fp32 = (64 + 8 * smax) * 2.0 ** -24
    return (1.1 * u + fp32) * (ref.abs() + mag) + TINY[dtype] + 1e-30


def norm_residual(y, r, w_post, gate, scale, w_pre, eps, gz=None, gh=None):
    """(outputs, magnitudes) of the gated residual norm in float64; with gz / gh the gradients too."""
    def d(x):
        return None if x is None else x.double()
    y, r, w_post, gate, w_pre, gz, gh = map(d, (y, r, w_post, gate, w_pre, gz, gh))
    g = 1.0 if gate is None else gate
    rstd_y = (y.square().mean(1, keepdim=True) + eps).rsqrt() if w_post is not None else torch.ones_like(y[:, :1])
    yhat = y * rstd_y
    n = yhat * w_post if w_post is not None else y
    res = torch.zeros_like(y) if r is None else r
    z = res + scale * g * n
    zmag = res.abs() + (scale * g * n).abs()
    rstd_z = (z.square().mean(1, keepdim=True) + eps).rsqrt()
    zhat, zhat_mag = z * rstd_z, zmag * rstd_z
    out, mag = {"z": z}, {"z": zmag}
    if w_pre is not None:
        out["h"], mag["h"] = zhat * w_pre, zhat_mag * w_pre.abs()
    if gz is None and gh is None:
        return out, mag
    dz = torch.zeros_like(y) if gz is None else gz
    dz_mag = dz.abs()
    if gh is not None:
        a = gh * w_pre
        dz = dz + rstd_z * (a - zhat * (zhat * a).mean(1, keepdim=True))
        dz_mag = dz_mag + rstd_z * (a.abs() + zhat_mag * (zhat_mag * a.abs()).mean(1, keepdim=True))
        out["gw_pre"], mag["gw_pre"] = (gh * zhat).sum(0), (gh.abs() * zhat_mag).sum(0)
    elif w_pre is not None:
        out["gw_pre"], mag["gw_pre"] = torch.zeros_like(w_pre), torch.zeros_like(w_pre)
    if r is not None:
        out["gr"], mag["gr"] = dz, dz_mag
    u, u_mag = scale * g * dz, (scale * g * torch.ones_like(y)).abs() * dz_mag
    if w_post is not None:
        b, b_mag = u * w_post, u_mag * w_post.abs()
        out["gy"] = rstd_y * (b - yhat * (yhat * b).mean(1, keepdim=True))
        mag["gy"] = rstd_y * (b_mag + yhat.abs() * (yhat.abs() * b_mag).mean(1, keepdim=True))
        out["gw_post"], mag["gw_post"] = (u * yhat).sum(0), (u_mag * yhat.abs()).sum(0)
    else:
        out["gy"], mag["gy"] = u, u_mag
    if gate is not None:
        gg, gg_mag = scale * dz * n, abs(scale) * dz_mag * n.abs()
        out["ggate"], mag["ggate"] = (gg.sum(0), gg_mag.sum(0)) if gate.dim() == 1 else (gg, gg_mag)
    return out, mag


def norm_bound(ref, mag, dtype, T, H, summed):
    """One rounding of the result to its type (fp32 for sums over tokens), and fp32 arithmetic: a dozen operations a
    term, sums of H terms in trees and short runs, and for the vectors a sum over T tokens."""
    steps = 64 + H // 256 + (T if summed else 0)
    return (1.05 * UNIT[torch.float32 if summed else dtype]) * ref.abs() + steps * 2.0 ** -24 * mag + (0.0 if summed else TINY[dtype]) + 1e-30


def encode8(x, levels):
    """Codes and scales of x [blocks, 256] fp32: the nearest level of fp32(x / max|x|), ties to the lower index."""
    top = x.abs().amax(1)
    r = x / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    mid = (levels[:-1].double() + levels[1:].double()) / 2
    return torch.bucketize(r.double(), mid).to(torch.uint8), top


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd):
    """One step: (new parameter in float64 from these fp32 moments, m, v), the moments by separately rounded fp32
    operations."""
    g = g.float()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t
    pd = p.double() * (1 - lr * wd) - lr / c1 * (m.double() / (v.double().sqrt() / math.sqrt(c2) + eps))
    return pd, m, v
