"""64-bit definitions of paged attention and of the router, with the magnitudes that their rounding-error bounds need.
Independent of the library: plain torch in float64."""
import math

import torch

from tests.block_refs import TINY, UNIT

ULP = 2.0 ** -24  # largest relative error of one fp32 rounding


def slots_of(table_row, length, page):
    pos = torch.arange(length, device=table_row.device)
    return table_row.long()[pos // page], pos % page


def paged_attention(q, kp, vp, table, lengths, scale):
    """(o, lse, mag, smag) in float64: mag is the sum of p |v|, smag the largest scale * sum |q| |k| of a row."""
    n, Hq, D = q.shape
    G = Hq // kp.shape[2]
    o = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    mag, lse = o.clone(), torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    smag = torch.zeros(n, Hq, dtype=torch.float64, device=q.device)
    for i, m in enumerate(lengths):
        if m <= 0:
            continue
        at = slots_of(table[i], m, kp.shape[1])
        k, v = (p[at].double().repeat_interleave(G, 1) for p in (kp, vp))
        qi = q[i].double()
        s = torch.einsum("hd,lhd->hl", qi, k) * scale
        smag[i] = (torch.einsum("hd,lhd->hl", qi.abs(), k.abs()) * abs(scale)).amax(1)
        p = torch.softmax(s, 1)
        lse[i] = torch.logsumexp(s, 1)
        o[i], mag[i] = torch.einsum("hl,lhd->hd", p, v), torch.einsum("hl,lhd->hd", p, v.abs())
    return o, lse, mag, smag


def paged_bounds(o, lse, mag, smag, lengths, D, dtype):
    """Error bounds of (o, lse).  A score is a sum of D products in fp32 (tensor cores may cut a bit: 2 ULP an addition),
    scaled and rounded; a weight's relative error is its score's error plus those of the exponential and of the moves of
    the maximum.  Sums over the tokens run over runs of at most a sixteenth of them and short trees.  On the tensor cores
    a weight is held as two values of the operand's type: their rest is a square of the unit (fp16 times 2, in whose
    subnormal range a tiny weight's second part ends: 2^-24 of the row's largest)."""
    n = torch.tensor(lengths, dtype=torch.float64, device=o.device)[:, None]
    score = (2 * D + 16) * ULP * smag
    sums = (n / 8 + 128) * ULP
    u = UNIT[dtype] if dtype != torch.float32 else 0.0
    weight = score * 2 + sums + (2 * u * u + (2 * ULP * n if dtype == torch.float16 else 0.0))
    bo = 1.02 * UNIT[dtype] * o.abs() + (weight[..., None] * 1.02) * mag + TINY[dtype] + 1e-30
    bl = score + sums + 4 * ULP * lse.abs().nan_to_num(posinf=0.0)
    return bo, bl


def scores(x, kind):
    return torch.sigmoid(x) if kind == "sigmoid" else torch.softmax(x, 1)


def choose(x, k, kind, bias, groups, top_groups, group_top):
    """The chosen experts [T, k] ascending, in float64; x of no NaN."""
    x = x.double()
    T, E = x.shape
    hidden = x == -math.inf
    c = x
    if bias is not None or group_top == 2:
        s = scores(x, kind).nan_to_num(nan=0.0)  # a row of -inf has no scores
        sums = (s + (0.0 if bias is None else bias.double())).masked_fill(hidden, -math.inf)
    if bias is not None:
        c = sums
    if groups > 1:
        by = (sums if group_top == 2 else c).view(T, groups, -1).sort(dim=2, descending=True).values
        worth = by[:, :, 0]
        if group_top == 2 and by.shape[2] > 1:
            worth = worth + torch.where(by[:, :, 1] == -math.inf, 0.0, by[:, :, 1])
        best = worth.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=x.device).scatter_(1, best, True).repeat_interleave(E // groups, 1)
        # experts that are not kept come after those of -inf that are
        order = torch.where(kept, c.clamp(min=-1e300), -math.inf)
    else:
        order = c
    return order.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(dim=1).values


def weights(x, experts, kind, renormalise, scale):
    """float64 weights [T, k] (differentiable in x)."""
    if renormalise:
        a = (torch.nn.functional.logsigmoid(x) if kind == "sigmoid" else x).gather(1, experts)
        top = a.detach().amax(1, keepdim=True)
        e = torch.where(top == -math.inf, 0.0, (a - torch.where(top == -math.inf, 0.0, top)).exp())
        total = e.sum(1, keepdim=True)
        return scale * e / torch.where(total == 0, 1.0, total)
    return scale * scores(x, kind).nan_to_num(nan=0.0).gather(1, experts)


def tables(experts, w, E):
    """(offsets, row_token, token_rows, row_weight) of routes with -1 for none, by plain loops over sorted pairs."""
    T, k = experts.shape
    e, wl = experts.cpu().tolist(), w.cpu().tolist()
    pairs = sorted((e[t][j], t, j) for t in range(T) for j in range(k) if e[t][j] >= 0)
    row_token, row_weight = [-1] * (T * k), [0.0] * (T * k)
    token_rows, offsets = [[-1] * k for _ in range(T)], [0] * (E + 1)
    for r, (x, t, j) in enumerate(pairs):
        row_token[r], row_weight[r], token_rows[t][j] = t, wl[t][j], r
        offsets[x + 1] += 1
    for x in range(E):
        offsets[x + 1] += offsets[x]
    dev = experts.device
    return (torch.tensor(offsets, dtype=torch.int32, device=dev), torch.tensor(row_token, dtype=torch.int32, device=dev),
            torch.tensor(token_rows, dtype=torch.int32, device=dev), torch.tensor(row_weight, dtype=torch.float32, device=dev))
