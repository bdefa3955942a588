"""Cases of the operators around a mixture-of-experts block that decodes and trains over frozen
4-bit weights: the paged key-value cache (new tokens written into it, one query token a sequence
attending over it) and the router (choice of experts, their weights, the tables that sort the
tokens by expert, and the gradient of the logits).

``listed()`` gives the fixed cases, ``draw(rng)`` more of the same ranges.  ``run`` computes an
operator in its plain form (elementary torch operations in fp32, in fp64 where the choice between
two experts hangs on it, rounded once at the end), or, with ``own`` set, through the package's
public calls.  ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases --

def listed():
    llama = {"Hq": 32, "Hk": 8, "D": 128, "dtype": "bf16", "order": "token"}
    softmax = {"op": "route", "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "pad": 0}
    return [
        # one user, a short chat turn: latency of one decoding step
        dict(llama, name="decode_one_short", op="decode", n=1, low=37, high=37, idle=0, page=16),
        # one user with a document of 131072 tokens in the cache
        dict(llama, name="decode_one_long", op="decode", n=1, low=131072, high=131072, idle=0, page=64),
        # a server's batch: 64 slots, fresh conversations beside long ones, three slots idle
        dict(llama, name="decode_batch_ragged", op="decode", n=64, low=1, high=16384, idle=3, page=16),
        # many short conversations, 40 query heads over 8, fp16 compute
        dict(name="decode_batch_short", op="decode", n=200, low=64, high=1024, idle=0, Hq=40, Hk=8, D=128, dtype="f16", page=32,
             order="token"),
        # unshared heads of 64, pages that hold a head's tokens together
        dict(name="decode_heads64", op="decode", n=24, low=500, high=3000, idle=0, Hq=32, Hk=32, D=64, dtype="bf16", page=128,
             order="head"),
        # fp32 checks of a small model: odd group, width and page
        dict(name="decode_f32_odd", op="decode", n=7, low=1, high=2000, idle=1, Hq=12, Hk=4, D=80, dtype="f32", page=24, order="token"),
        # a packed batch of prompts enters the cache: long, middling, one-token and empty ones, some with a cached beginning
        dict(llama, name="append_prompts_8192", op="append", lens="3001,129,0,1,2048,777,64,1500,672", before="0,300,17,4000,0,0,5,1,64", page=16),
        # one chunk of a long prompt, fp16, pages that hold a head's tokens together
        dict(name="append_chunk", op="append", lens="513", before="4099", Hq=40, Hk=8, D=128, dtype="f16", page=64, order="head"),
        # one token through the router of 64 experts: latency of decoding
        dict(softmax, name="route_one_token", T=1, E=64, k=8, dtype="f32", train=False),
        # a 512-token training micro-batch over 64 experts, eight a token
        dict(softmax, name="route_train_512", T=512, E=64, k=8, dtype="f32", train=True),
        # a large training batch over 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="route_train_groups_8192", op="route", T=8192, E=256, k=8, dtype="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, pad=0, train=True),
        # an odd batch with padding at its end, an odd number of experts, 16-bit logits (with ties among them)
        dict(softmax, name="route_odd", T=4099, E=60, k=4, dtype="bf16", renorm=True, pad=131, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_SLOTS = 64 * 16384 * 8 * 128  # of the largest listed batch: sequences x longest x heads x width


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "route", "route"])
    while op != "route":
        Hk = rng.choice([1, 2, 4, 8, 8, 32])
        G = rng.choice([1, 2, 3, 4, 5, 8, 12]) if Hk < 32 else 1
        case = {"op": op, "Hq": Hk * G, "Hk": Hk, "D": rng.choice([64, 80, 96, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "page": rng.choice([16, 16, 24, 32, 64, 128]), "order": rng.choice(["token", "token", "head"])}
        if op == "decode":
            n, high = _log(rng, 1, 256), _log(rng, 1, 131072)
            case.update(n=n, low=_log(rng, 1, high), high=high, idle=rng.choice([0, 0, n // 8]))
            if n * high * Hk * case["D"] * BYTES[case["dtype"]] <= 2 * MOST_SLOTS:
                return case
        else:
            total, n = _log(rng, 1, 8192), _log(rng, 1, 16)
            cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            before = [rng.choice([0, 0, _log(rng, 1, 4099)]) for _ in lens]
            case.update(lens=",".join(map(str, lens)), before=",".join(map(str, before)))
            if total * Hk * case["D"] * BYTES[case["dtype"]] <= 2 * 8192 * 8 * 128:
                return case
    groups = rng.choice([1, 1, 4, 8])
    E = groups * _log(rng, 4, 256 // groups)
    top_groups = rng.randint(1, groups)
    k = min(rng.randint(1, 10), top_groups * (E // groups))  # a renormalised single expert has weight 1 and no gradient
    T = _log(rng, 1, 8192)
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "score": rng.choice(["softmax", "sigmoid"]),
            "bias": rng.random() < 0.4, "groups": groups, "top_groups": top_groups, "group_top": rng.choice([1, 2]),
            "renorm": rng.random() < 0.5 and k > 1, "pad": rng.choice([0, 0, T // 10]), "train": rng.random() < 0.6}


def _ints(text):
    return [int(n) for n in text.split(",")]


def _lengths(case):
    """Tokens of each sequence in the cache, those of this call among them."""
    if case["op"] == "append":
        return [a + b for a, b in zip(_ints(case["lens"]), _ints(case["before"]))]
    rng = random.Random(1000003 * case["n"] + case["high"])
    n = case["n"] - case["idle"]
    lens = [rng.randint(case["low"], case["high"]) for _ in range(n)]
    if n:
        lens[rng.randrange(n)] = case["high"]
    return lens + [0] * case["idle"]


def _new(case):
    """Tokens of each sequence that this call brings."""
    return _ints(case["lens"]) if case["op"] == "append" else [min(1, n) for n in _lengths(case)]


def work(case):
    if case["op"] == "route":
        T, E, k, e = case["T"], case["E"], case["k"], BYTES[case["dtype"]]
        live = T - case["pad"]
        # logits in; experts, weights, both row tables and the rows' weights out
        moved, flops = live * E * e + 5 * 4 * T * k + 4 * (E + 1), 4 * live * E
        if case["train"]:  # also the rows' gradients in and the logits' out; the logits again are the same input
            moved, flops = moved + 4 * live * k + T * E * e, flops + 4 * live * E
        return {"bytes": moved, "flops": flops}
    e, row = BYTES[case["dtype"]], case["Hk"] * case["D"]
    new, held = sum(_new(case)), sum(_lengths(case))
    if case["op"] == "append":
        return {"bytes": 4 * new * row * e, "flops": 0}
    q = case["n"] * case["Hq"]
    # the new tokens in and into the cache, the cache read once, queries in, outputs and row statistics out
    return {"bytes": (2 * held + 2 * new) * row * e + 2 * q * case["D"] * e + 4 * q, "flops": 4 * held * case["Hq"] * case["D"]}


# -------------------------------------------------------------------------- inputs --

SCALE = 2.5  # of the routing weights with renormalisation


def _cache(case, normal, g):
    """Pages with leftovers in every slot, a shuffled page table, and the lengths."""
    page, Hk, D, dt = case["page"], case["Hk"], case["D"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    need = [-(-n // page) for n in lens]
    total = sum(need)
    shape = (total + 3, page, Hk, D) if case["order"] == "token" else (total + 3, Hk, page, D)
    pages = []
    for mean in (0.0, 0.25):
        x = torch.empty(shape, dtype=dt, device="cuda")
        for part in x.split(max(1, (1 << 26) // (page * Hk * D))):
            part.copy_(normal(*part.shape) + mean)
        pages.append(x if case["order"] == "token" else x.transpose(1, 2))
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)[:total]
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(table.shape[1], device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[held] = order
    return pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dt = DTYPES[case["dtype"]]
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        live = T - case["pad"]
        s.update(logits=(1.5 * normal(T, E)).to(dt), bias=0.1 * normal(E) if case["bias"] else None, live=None,
                 grow=normal(T * case["k"]) if case["train"] else None, scale=SCALE if case["renorm"] else 1.0)
        if case["pad"]:
            s["live"] = torch.arange(T, device="cuda") < live
        return s
    new = _new(case)
    T, Hk, D = sum(new), case["Hk"], case["D"]
    (s["kp"], s["vp"]), s["table"], s["lengths"] = _cache(case, normal, g)
    if case["op"] == "append":
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        s.update(k=normal(T, Hk, D).to(dt), v=(normal(T, Hk, D) + 0.25).to(dt))
    else:  # a row for every slot, idle ones too
        n = case["n"]
        q = normal(n, case["Hq"], D)
        q[..., : D // 16] *= 2
        s.update(q=q.to(dt), k=normal(n, Hk, D).to(dt), v=(normal(n, Hk, D) + 0.25).to(dt), cu=None)
    return s


# --------------------------------------------------------------------- plain forms --

def _plain_append(s):
    """New row r of sequence i goes to position length_i - new_i + r."""
    lengths, table, page = s["lengths"].long(), s["table"].long(), s["page"]
    if s["cu"] is None:
        seq = torch.nonzero(lengths > 0).flatten()
        row, pos = seq, lengths[seq] - 1
    else:
        cu = s["cu"].long()
        row = torch.arange(s["k"].shape[0], device=cu.device)
        seq = (row[:, None] >= cu[None, 1:]).sum(1)
        pos = lengths[seq] - cu[seq + 1] + row
    at = table[seq, pos // page]
    s["kp"][at, pos % page] = s["k"][row]
    s["vp"][at, pos % page] = s["v"][row]
    return {"k_pages": s["kp"], "v_pages": s["vp"]}


def _plain_decode(s):
    out = _plain_append(s)
    n, Hk, D = s["n"], s["Hk"], s["D"]
    at = s["table"].clamp(min=0).long()
    k, v = (p[at].reshape(n, -1, Hk, D).float() for p in (s["kp"], s["vp"]))
    hidden = (torch.arange(k.shape[1], device=k.device)[None, :] >= s["lengths"][:, None])[:, None, None, :]
    q = s["q"].float().view(n, Hk, -1, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5).masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill_(hidden.transpose(1, 3), 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    return dict(out, o=o.reshape(n, s["Hq"], D).to(s["q"].dtype), lse=(top + total.log()).reshape(n, s["Hq"]))


def _plain_scores(x, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + (-x).exp())
    e = (x - x.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    x, T, E, k = s["logits"].float(), s["T"], s["E"], s["k"]
    score = _plain_scores(x, s["score"])
    choice = x
    if s["bias"] is not None or (s["groups"] > 1 and s["group_top"] == 2):  # sums: a border may lie between two of them
        wide = _plain_scores(x.double(), s["score"])
        wide = wide if s["bias"] is None else wide + s["bias"].double()
        choice = x if s["bias"] is None else wide
    if s["groups"] > 1:
        by = (wide if s["group_top"] == 2 else choice).view(T, s["groups"], -1)
        worth = by.sort(dim=2, descending=True).values[:, :, : s["group_top"]].sum(2)
        best = worth.sort(dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        kept = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, best, True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // s["groups"], 1), -math.inf)
    experts = choice.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
    weights = score.gather(1, experts)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    share = weights
    weights = weights * s["scale"]
    live = torch.ones(T, dtype=torch.bool, device=x.device) if s["live"] is None else s["live"]
    experts, weights = experts.masked_fill(~live[:, None], -1), weights * live[:, None]
    # rows sorted by expert, by token within an expert; those of padding are none
    key = torch.where(experts < 0, E, experts).flatten()
    by_row = key.sort(stable=True)
    order, used = by_row.indices, by_row.values < E
    token_rows = torch.empty_like(order)
    token_rows[order] = torch.where(used, torch.arange(T * k, device=x.device), -1)
    offsets = torch.searchsorted(by_row.values, torch.arange(E + 1, device=x.device))
    out = {"experts": experts.int(), "weights": weights, "offsets": offsets.int(), "row_token": torch.where(used, order // k, -1).int(),
           "token_rows": token_rows.view(T, k).int(), "row_weight": weights.flatten()[order]}
    if s["grow"] is None:
        return out
    at = token_rows.view(T, k)
    gw = torch.where(at < 0, 0.0, s["grow"][at.clamp(min=0)])
    held = experts.clamp(min=0)
    mean = (gw * share).sum(1, keepdim=True)
    if s["renorm"]:
        gx = s["scale"] * share * (gw - mean)
        if s["score"] == "sigmoid":
            gx = gx * (1.0 - score.gather(1, held))
        gx = torch.zeros_like(x).scatter_(1, held, gx)
    elif s["score"] == "sigmoid":
        gx = torch.zeros_like(x).scatter_(1, held, s["scale"] * gw * share * (1.0 - share))
    else:
        gx = s["scale"] * score * (torch.zeros_like(x).scatter_(1, held, gw) - mean)
    return dict(out, glogits=(gx * live[:, None]).to(s["logits"].dtype))


def run(s):
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "route": _plain_route}[s["op"]](s)
    import bit_nf4_quantized_linear_gb300 as nf4
    if s["op"] == "route":
        how = dict(score=s["score"], renormalise=s["renorm"], scale=s["scale"])
        r = nf4.route_experts(s["logits"], s["k"], bias=s["bias"], groups=s["groups"], top_groups=s["top_groups"],
                              group_top=s["group_top"], live=s["live"], **how)
        out = {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "row_token": r.row_token, "token_rows": r.token_rows,
               "row_weight": r.row_weight}
        if s["grow"] is None:
            return out
        return dict(out, glogits=nf4.route_experts_bwd(s["logits"], r, grad_row_weight=s["grow"], **how))
    nf4.paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lengths"], s["cu"])
    out = {"k_pages": s["kp"], "v_pages": s["vp"]}
    if s["op"] == "append":
        return out
    o, lse = nf4.paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["lengths"])
    return dict(out, o=o, lse=lse)


# ------------------------------------------------------------------ 64-bit definitions --

def _exact_cache(s, case):
    """The pages after the call, and each sequence's slots in order."""
    kp, vp = s["kp"].double(), s["vp"].double()
    lens, new, page = _lengths(case), _new(case), case["page"]
    slots, first = [], 0
    for i, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n, device="cuda")
        slots.append((s["table"][i].long()[pos // page], pos % page))
        rows = slice(first, first + m) if case["op"] == "append" else slice(i, i + m)
        last = tuple(x[n - m:] for x in slots[-1])
        kp[last], vp[last] = s["k"][rows].double(), s["v"][rows].double()
        first += m
    return kp, vp, slots


def _exact_decode(s, case):
    kp, vp, slots = _exact_cache(s, case)
    G = s["Hq"] // s["Hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, at in enumerate(slots):
        if at[0].numel():
            k, v = (x[at].repeat_interleave(G, 1) for x in (kp, vp))
            score = torch.einsum("hd,lhd->hl", s["q"][i].double(), k) / math.sqrt(s["D"])
            lse[i] = torch.logsumexp(score, 1)
            o[i] = torch.einsum("hl,lhd->hd", torch.softmax(score, 1), v)
    return {"k_pages": kp, "v_pages": vp, "o": o, "lse": lse}


def _places(c):
    """The rank of each value in its row: how many are larger, or equal and before it."""
    before = torch.ones(c.shape[1], c.shape[1], dtype=torch.bool, device=c.device).triu(1)
    rank = [((b[:, :, None] > b[:, None, :]) | ((b[:, :, None] == b[:, None, :]) & before)).sum(1) for b in c.split(512)]
    return torch.cat(rank)


def _exact_route(s):
    T, E, k = s["T"], s["E"], s["k"]
    with torch.enable_grad():
        x = s["logits"].double().requires_grad_()
        score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
        with torch.no_grad():
            c = score if s["bias"] is None else score + s["bias"].double()
            if s["groups"] > 1:
                in_group = c.view(T, s["groups"], -1)
                worth = in_group.topk(min(s["group_top"], in_group.shape[2]), 2).values.sum(2)
                lost = _places(worth) >= s["top_groups"]
                order = (x.detach() if s["bias"] is None else c).masked_fill(lost.repeat_interleave(E // s["groups"], 1), -math.inf)
            else:
                order = x.detach() if s["bias"] is None else c
            chosen = _places(order) < k
            if s["live"] is not None:
                chosen &= s["live"][:, None]
        w = score * chosen
        if s["renorm"]:
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total > 0, total, torch.ones_like(total))
        w = s["scale"] * w
        # the pairs by expert and then by token are the true places of the transposed table
        by_row = chosen.T.nonzero()
        row_weight = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        row_weight[: by_row.shape[0]] = w.detach()[by_row[:, 1], by_row[:, 0]]
        row_token = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        row_token[: by_row.shape[0]] = by_row[:, 1].int()
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = chosen.sum(0).cumsum(0)
        place = torch.zeros(T, E, dtype=torch.int64, device="cuda")
        place[by_row[:, 1], by_row[:, 0]] = torch.arange(by_row.shape[0], device="cuda")
        by_token = chosen.nonzero()
        experts = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        token_rows, weights = experts.clone(), torch.zeros(T, k, dtype=torch.float64, device="cuda")
        rows = chosen.any(1)
        experts[rows] = by_token[:, 1].int().view(-1, k)
        token_rows[rows] = place[chosen].int().view(-1, k)
        weights[rows] = w.detach()[chosen].view(-1, k)
        out = {"experts": experts, "weights": weights, "offsets": offsets, "row_token": row_token, "token_rows": token_rows,
               "row_weight": row_weight}
        if s["grow"] is None:
            return out
        gw = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        gw[by_row[:, 1], by_row[:, 0]] = s["grow"][: by_row.shape[0]].double()
        return dict(out, glogits=torch.autograd.grad((w * gw).sum(), x)[0])


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["op"] == "route":
            return _exact_route(s)
        if case["op"] == "append":
            return dict(zip(("k_pages", "v_pages"), _exact_cache(s, case)))
        return _exact_decode(s, case)
