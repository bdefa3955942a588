"""Cases of the training-block operators: causal attention over packed sequences, the
gated residual norm around a block, and the AdamW step over many tensors.

``listed()`` gives the fixed cases, ``draw(rng)`` more of the same ranges.  ``run`` computes an
operator in its plain form (elementary torch operations in fp32, rounded once at the end), or,
with ``own`` set, through the package's public calls.  ``exact`` restates the definitions in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 256  # values that share one scale of the 8-bit optimiser states


# --------------------------------------------------------------------------- cases --

def listed():
    llama = {"op": "attention", "Hq": 32, "Hk": 8, "D": 128, "dtype": "bf16"}
    return [
        # a short user turn in evaluation: latency of one forward
        dict(llama, name="attn_short_prompt", lens="77", train=False),
        # a training micro-batch of 512 tokens: three packed samples of uneven length
        dict(llama, name="attn_train_512", lens="301,1,210", train=True),
        # a full packed training batch: long, middling, one-token and empty samples
        dict(llama, name="attn_train_packed_8192", lens="3001,129,0,1,2048,777,64,1500,672", train=True),
        # a long document in evaluation, 40 query heads over 8, fp16 compute
        dict(name="attn_long_prompt", op="attention", Hq=40, Hk=8, D=128, dtype="f16", lens="12289", train=False),
        # unshared heads of 64 in training, one even sample and one odd
        dict(name="attn_train_heads64", op="attention", Hq=32, Hk=32, D=64, dtype="bf16", lens="2048,2047", train=True),
        # one token through the norms of a block: latency
        dict(name="norm_one_token", op="norm", T=1, H=4096, dtype="bf16", gate="channel", train=False),
        # a 512-token training micro-batch at hidden 4096, gain per channel on the branch
        dict(name="norm_train_512", op="norm", T=512, H=4096, dtype="bf16", gate="channel", train=True),
        # a large training batch at hidden 5120, gate per token and channel
        dict(name="norm_train_8192", op="norm", T=8192, H=5120, dtype="bf16", gate="token", train=True),
        # widths and counts that fit no vector, fp16
        dict(name="norm_train_odd", op="norm", T=1023, H=2047, dtype="f16", gate="channel", train=True),
        # rank-16 adapters of one layer's seven projections, fp32 with fp32 states
        dict(name="adamw_adapters_f32", op="adamw", set="adapters", layers=1, rank=16, dtype="f32", bits=32),
        # rank-16 adapters of eight layers with 8-bit states
        dict(name="adamw_adapters_8bit", op="adamw", set="adapters", layers=8, rank=16, dtype="bf16", bits=8),
        # dense matrices trained in full with 8-bit states: three projections, a gain and an odd vector
        dict(name="adamw_dense_8bit", op="adamw", set="dense", N=14336, K=4096, odd=1000003, dtype="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "norm", "adamw"])
    while op == "attention":
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
        D = rng.choice([64, 80, 96, 128, 128])
        total, n, train = _log(rng, 16, 12000), _log(rng, 1, 16), rng.random() < 0.6
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        case = {"op": "attention", "Hq": Hq, "Hk": Hk, "D": D, "dtype": rng.choice(["bf16", "bf16", "f16"]),
                "lens": ",".join(map(str, lens)), "train": train}
        if work(case)["flops"] <= 1.5e12:  # the longest listed prompt
            return case
    if op == "norm":
        T, H = _log(rng, 1, 8192), _log(rng, 256, 5120)
        if rng.random() < 0.6:
            H = -(-H // 64) * 64
        return {"op": "norm", "T": T, "H": H, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "gate": rng.choice(["none", "channel", "token"]), "train": rng.random() < 0.7}
    dtype = rng.choice(["bf16", "f32", "f16"])
    if rng.random() < 0.6:
        return {"op": "adamw", "set": "adapters", "layers": rng.randint(1, 12), "rank": _log(rng, 4, 64),
                "dtype": dtype, "bits": rng.choice([8, 32])}
    return {"op": "adamw", "set": "dense", "N": _log(rng, 256, 8192), "K": _log(rng, 256, 4096),
            "odd": _log(rng, 1, 1000003), "dtype": dtype, "bits": rng.choice([8, 32])}


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _shapes(case):
    """The trained tensors of an optimiser case."""
    if case["set"] == "dense":
        N, K = case["N"], case["K"]
        return [(N, K), (K, N), (K, K), (K,), (case["odd"],)]
    r = case["rank"]
    proj = [(4096, 4096), (4096, 1024), (4096, 1024), (4096, 4096), (4096, 14336), (4096, 14336), (14336, 4096)]
    return [s for _ in range(case["layers"]) for k, n in proj for s in ((r, k), (n, r))]


def work(case):
    if case["op"] == "attention":
        lens, Hq, Hk, D = _lens(case), case["Hq"], case["Hk"], case["D"]
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        q, kv = 2 * T * Hq * D, 2 * T * Hk * D
        if not case["train"]:
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * pairs * Hq * D}
        # forward: two products; backward: five (scores, their gradient, and three gradients)
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * pairs * Hq * D}
    if case["op"] == "norm":
        T, H, e = case["T"], case["H"], BYTES[case["dtype"]]
        act, vec = T * H * e, 4 * H
        tok = act if case["gate"] == "token" else 0
        ch = vec if case["gate"] == "channel" else 0
        if not case["train"]:
            return {"bytes": 4 * act + tok + ch + 2 * vec, "flops": 12 * T * H}
        # also the gradients of both outputs in, those of y, residual, gate and gains out
        return {"bytes": 8 * act + 2 * tok + 2 * ch + 4 * vec, "flops": 40 * T * H}
    n = sum(math.prod(s) for s in _shapes(case))
    e = BYTES[case["dtype"]]
    # parameter read and written, gradient read, both states read and written; 8-bit states also read out as values
    state = 16 * n if case["bits"] == 32 else 4 * n + 8 * n + 16 * (n // BLOCK)
    return {"bytes": 3 * e * n + state, "flops": 16 * n}


# -------------------------------------------------------------------------- inputs --

HYPER = dict(lr=2e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
EPS, SCALE = 1e-6, 0.5  # of the norms, and of the residual branch


def signed_levels():
    """The 256 levels of the signed 8-bit dynamic map in 64 bits: seven decades, 2**e fractions in decade e."""
    mags = []
    for e in range(7):
        edges = torch.linspace(0.1, 1.0, 2 ** e + 1, dtype=torch.float64)
        mags.append((edges[:-1] + edges[1:]) / 2 * 10.0 ** (e - 6))
    m = torch.cat(mags)
    return torch.sort(torch.cat([m, -m, torch.tensor([0.0, 1.0], dtype=torch.float64)])).values


def unsigned_levels():
    """The 256 levels of the unsigned map: the sign bit buys twice the fractions in each decade."""
    mags = []
    for e in range(7):
        edges = torch.linspace(0.1, 1.0, 2 ** (e + 1) + 1, dtype=torch.float64)
        mags.append((edges[:-1] + edges[1:]) / 2 * 10.0 ** (e - 6))
    return torch.sort(torch.cat([*mags, torch.tensor([0.0, 1.0], dtype=torch.float64)])).values


def _levels(dtype, device):
    """Both maps, at the fp32 values that the states hold."""
    return [f().to(torch.float32).to(dtype).to(device) for f in (signed_levels, unsigned_levels)]


def _encode(x, levels):
    """Codes and scales of x [blocks, 256]: the nearest level of x / max|x|, ties to the lower index."""
    top = x.abs().amax(dim=1)
    r = x / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    mid = (levels[:-1].double() + levels[1:].double()) / 2
    return torch.bucketize(r.double(), mid), top


def _padded(case):
    return [-(-math.prod(s) // BLOCK) * BLOCK for s in _shapes(case)]


def _views(flat, case):
    out, at = [], 0
    for s, n in zip(_shapes(case), _padded(case)):
        out.append(flat[at:at + math.prod(s)].view(s))
        at += n
    return out


def _adamw_inputs(case, seed):
    """Parameters, gradients and states some hundred steps into training, each tensor starting a block of one flat buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, dt = sum(_padded(case)), DTYPES[case["dtype"]]

    def normal():
        return torch.randn(n, generator=g, device="cuda")

    size = 1e-3 * torch.exp(0.5 * torch.randn(n // BLOCK, 1, generator=g, device="cuda")).expand(-1, BLOCK).reshape(-1)
    p, gr = 0.02 * normal(), size * normal()
    m, v = 0.3 * size * normal(), size.square() * (0.2 + normal().square())
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for t in _views(live, case):
        t.fill_(True)
    return [x * live for x in (p, gr, m, v)], dt


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "attention":
        dt, lens = DTYPES[case["dtype"]], _lens(case)
        T, Hq, Hk, D = sum(lens), case["Hq"], case["Hk"], case["D"]
        # normalised queries and keys, a few strong directions among them; values with a mean
        q, k = normal(T, Hq, D), normal(T, Hk, D)
        q[..., : D // 16] *= 2
        k[..., : D // 16] *= 2
        v = normal(T, Hk, D) + 0.25 * normal(1, Hk, D)
        s.update(q=q.to(dt), k=k.to(dt), v=v.to(dt), go=normal(T, Hq, D).to(dt) if case["train"] else None, lens=lens,
                 cu=torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda"))
    elif case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        # a residual stream with a few large channels
        loud = 1 + 20 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s.update(y=(0.7 * normal(T, H)).to(dt), r=(1.5 * loud * normal(T, H)).to(dt),
                 w_post=1 + 0.2 * normal(H), w_pre=1 + 0.2 * normal(H), gate=None,
                 gz=(0.1 * normal(T, H)).to(dt) if case["train"] else None, gh=normal(T, H).to(dt) if case["train"] else None)
        if case["gate"] == "channel":
            s["gate"] = 0.5 + 0.2 * normal(H)
        elif case["gate"] == "token":
            s["gate"] = torch.sigmoid(normal(T, H)).to(dt)
    else:
        (p, gr, m, v), dt = _adamw_inputs(case, seed)
        s.update(flat_p=p.to(dt), flat_g=gr.to(dt), step=100)
        s.update(p=_views(s["flat_p"], case), g=_views(s["flat_g"], case))
        if case["bits"] == 32:
            s.update(m=m, v=v)
        else:
            for key, x, lev in zip("mv", (m, v), _levels(torch.float32, "cuda")):
                codes, top = _encode(x.view(-1, BLOCK), lev)
                s[key], s[key + "_top"], s[key + "_lev"] = codes.to(torch.uint8).view(-1), top, lev
        if own:
            import bit_nf4_quantized_linear_gb300 as nf4
            state = nf4.adamw_state(s["p"], bits=case["bits"])
            state.step = s["step"]
            state.exp_avg.copy_(s["m"])
            state.exp_avg_sq.copy_(s["v"])
            if case["bits"] == 8:
                state.exp_avg_absmax.copy_(s["m_top"])
                state.exp_avg_sq_absmax.copy_(s["v_top"])
            s["state"] = state
    return s


# --------------------------------------------------------------------- plain forms --

def _attention(s):
    q, k, v, go, dt = s["q"], s["k"], s["v"], s["go"], s["q"].dtype
    G, scale = s["Hq"] // s["Hk"], s["D"] ** -0.5
    outs = [torch.zeros_like(x) for x in ((q, q, k, v) if go is not None else (q,))]
    at = 0
    for n in s["lens"]:  # the packed sequences
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        qf = q[rows].float().transpose(0, 1).reshape(s["Hk"], G, n, -1)
        kf, vf = (x[rows].float().transpose(0, 1).unsqueeze(1) for x in (k, v))
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1)
        p = (qf @ kf.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        p = p.div_(p.sum(-1, keepdim=True))
        outs[0][rows] = (p @ vf).reshape(s["Hq"], n, -1).transpose(0, 1).to(dt)
        if go is None:
            continue
        gf = go[rows].float().transpose(0, 1).reshape(s["Hk"], G, n, -1)
        outs[3][rows] = (p.transpose(-1, -2) @ gf).sum(1).transpose(0, 1).to(dt)
        dp = gf @ vf.transpose(-1, -2)
        ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        outs[1][rows] = (ds @ kf).reshape(s["Hq"], n, -1).transpose(0, 1).to(dt)
        outs[2][rows] = (ds.transpose(-1, -2) @ qf).sum(1).transpose(0, 1).to(dt)
    return dict(zip(("o", "gq", "gk", "gv"), outs))


def _norm(s):
    dt, y, r = s["y"].dtype, s["y"].float(), s["r"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    rstd_y = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    yhat = y * rstd_y
    n = yhat * s["w_post"]
    z = r + SCALE * gate * n
    rstd_z = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
    zhat = z * rstd_z
    out = {"z": z.to(dt), "h": (zhat * s["w_pre"]).to(dt)}
    if s["gh"] is None:
        return out
    gz, gh = s["gz"].float(), s["gh"].float()
    a = gh * s["w_pre"]
    dz = gz + rstd_z * (a - zhat * (zhat * a).mean(-1, keepdim=True))
    u = SCALE * gate * dz
    b = u * s["w_post"]
    out.update(gr=dz.to(dt), gy=(rstd_y * (b - yhat * (yhat * b).mean(-1, keepdim=True))).to(dt),
               gw_pre=(gh * zhat).sum(0), gw_post=(u * yhat).sum(0))
    if s["gate"] is not None:
        gg = SCALE * dz * n
        out["ggate"] = gg.sum(0) if s["gate"].dim() == 1 else gg.to(dt)
    return out


def _adamw(s):
    b1, b2 = HYPER["betas"]
    s["step"] += 1
    c1, c2 = 1 - b1 ** s["step"], 1 - b2 ** s["step"]
    p, g = s["flat_p"].float(), s["flat_g"].float()
    m, v = s["m"], s["v"]
    if s["bits"] == 8:
        m, v = ((s[x + "_lev"][s[x].int()].view(-1, BLOCK) * s[x + "_top"][:, None]).view(-1) for x in "mv")
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    p = p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - (HYPER["lr"] / c1) * (m / (v.sqrt() / math.sqrt(c2) + HYPER["eps"]))
    s["flat_p"].copy_(p)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["flat_p"], "m": s["m"], "v": s["v"]}
    out = {"p": s["flat_p"]}
    for key, x in zip("mv", (m, v)):
        codes, top = _encode(x.view(-1, BLOCK), s[key + "_lev"])
        s[key].copy_(codes.view(-1))
        s[key + "_top"].copy_(top)
        out[key] = (s[key + "_lev"][codes] * top[:, None]).view(-1)
    return out


def run(s):
    if not own:
        return {"attention": _attention, "norm": _norm, "adamw": _adamw}[s["op"]](s)
    import bit_nf4_quantized_linear_gb300 as nf4
    if s["op"] == "attention":
        o, lse = nf4.attention_fwd(s["q"], s["k"], s["v"], s["cu"])
        if s["go"] is None:
            return {"o": o}
        gq, gk, gv = nf4.attention_bwd(s["go"], s["q"], s["k"], s["v"], o, lse, s["cu"])
        return {"o": o, "gq": gq, "gk": gk, "gv": gv}
    if s["op"] == "norm":
        z, h, stats = nf4.norm_residual_fwd(s["y"], s["r"], w_post=s["w_post"], gate=s["gate"], scale=SCALE,
                                            w_pre=s["w_pre"], eps=EPS)
        if s["gh"] is None:
            return {"z": z, "h": h}
        gy, gr, gw_post, ggate, gw_pre = nf4.norm_residual_bwd(
            s["gz"], s["gh"], s["y"], s["r"], stats, w_post=s["w_post"], gate=s["gate"], scale=SCALE, w_pre=s["w_pre"])
        out = {"z": z, "h": h, "gr": gr, "gy": gy, "gw_pre": gw_pre, "gw_post": gw_post}
        return out if ggate is None else dict(out, ggate=ggate)
    nf4.adamw_step(s["p"], s["g"], s["state"], **HYPER)
    if s["bits"] == 32:
        return {"p": s["flat_p"], "m": s["state"].exp_avg, "v": s["state"].exp_avg_sq}
    m, v = nf4.adamw_state_values(s["state"])
    return {"p": s["flat_p"], "m": m, "v": v}


# ------------------------------------------------------------------ 64-bit definitions --

def _exact_attention(s):
    T, Hq, Hk, D = s["q"].shape[0], s["Hq"], s["Hk"], s["D"]
    q, k, v = (s[x].double() for x in "qkv")
    o = torch.zeros_like(q)
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    first = 0
    for n in s["lens"]:
        last = first + n
        for h in range(Hq if n else 0):
            qh, kh, vh = q[first:last, h], k[first:last, h // (Hq // Hk)], v[first:last, h // (Hq // Hk)]
            for a in range(0, n, 2048):  # query rows a .. b - 1 see keys 0 .. b - 1 at most
                b = min(n, a + 2048)
                seen = torch.arange(b, device=q.device)[None, :] <= torch.arange(a, b, device=q.device)[:, None]
                score = torch.where(seen, qh[a:b] @ kh[:b].T / math.sqrt(D), torch.full((), -math.inf, dtype=torch.float64, device=q.device))
                w = torch.softmax(score, dim=1)
                o[first + a:first + b, h] = w @ vh[:b]
                if s["go"] is None:
                    continue
                d = s["go"][first + a:first + b, h].double()
                dw = d @ vh[:b].T
                dscore = w * (dw - torch.sum(w * dw, dim=1, keepdim=True)) / math.sqrt(D)
                gq[first + a:first + b, h] = dscore @ kh[:b]
                gk[first:first + b, h // (Hq // Hk)] += dscore.T @ qh[a:b]
                gv[first:first + b, h // (Hq // Hk)] += w.T @ d
        first = last
    return {"o": o} if s["go"] is None else {"o": o, "gq": gq, "gk": gk, "gv": gv}


def _exact_norm(s):
    def norm(x, w):
        return x / torch.sqrt(torch.mean(x ** 2, dim=1, keepdim=True) + EPS) * w

    with torch.enable_grad():
        y, r, w_post, w_pre = (s[x].double().requires_grad_() for x in ("y", "r", "w_post", "w_pre"))
        gate = None if s["gate"] is None else s["gate"].double().requires_grad_()
        branch = norm(y, w_post)
        z = r + SCALE * (branch if gate is None else gate * branch)
        h = norm(z, w_pre)
        out = {"z": z.detach(), "h": h.detach()}
        if s["gh"] is None:
            return out
        names, leaves = ["gr", "gy", "gw_pre", "gw_post"], [r, y, w_pre, w_post]
        if gate is not None:
            names, leaves = names + ["ggate"], leaves + [gate]
        grads = torch.autograd.grad([z, h], leaves, [s["gz"].double(), s["gh"].double()])
    return dict(out, **dict(zip(names, grads)))


def _exact_adamw(s):
    b1, b2 = HYPER["betas"]
    t = s["step"] + 1
    levels = _levels(torch.float64, "cuda")
    p, g = s["flat_p"].double(), s["flat_g"].double()
    mom = []
    for key, lev in zip("mv", levels):
        x = s[key]
        mom.append(x.double() if s["bits"] == 32 else (lev[x.long()].view(-1, BLOCK) * s[key + "_top"].double()[:, None]).flatten())
    m, v = b1 * mom[0] + (1 - b1) * g, b2 * mom[1] + (1 - b2) * g ** 2
    p = p - HYPER["lr"] * HYPER["weight_decay"] * p - HYPER["lr"] * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"])
    if s["bits"] == 32:
        return {"p": p, "m": m, "v": v}
    out = {"p": p}
    for key, x, lev in zip("mv", (m, v), levels):
        x = x.view(-1, BLOCK)
        codes, top = _encode(x, lev)
        out[key] = (lev[codes] * top[:, None]).flatten()
    return out


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        return {"attention": _exact_attention, "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](s)
