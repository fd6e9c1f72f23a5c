"""Operators of the decoder block's second half that serve its norms and its router in training as well.

Four calls next to dwdp_add_rmsnorm, dwdp_route_scored and dwdp_quantize_rows:

  norm       norms after and before a block, with the block's gate and the residual's scale:
               n = x / sqrt(mean(x^2) + eps) * post,  h = a residual + c gate n,
               y = h / sqrt(mean(h^2) + eps) * pre
             and, where asked for, y as E4M3 rows for the expert layer and x and h as E4M3 rows with one scale
             each, which is all that the backward pass needs of them          (dwdp_sandwich_norm)
  norm_grad  its gradients (x, residual, both weights, each group's gate) from bf16 rows or from the rows
             kept in 8 bits                                                   (dwdp_sandwich_norm_grad)
  balance    per sequence b of T_b tokens: how often each expert was chosen, the experts' mean share of the
             scores P, and the losses E / (k T_b) sum_e counts_e P_e and mean(logsumexp(z)^2)
                                                                              (dwdp_balance_loss)
  router_grad  the logits' gradient from those losses and from the weights of the chosen experts
                                                                              (dwdp_route_scored_grad)

`run` computes them in elementary torch operations, or, where `own` is true, with the calls of this library.
`exact` computes them again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    r1 = {"E": 256, "k": 8, "score": "sigmoid", "renorm": True, "scale": 2.5}
    small = {"E": 64, "k": 6, "score": "softmax", "renorm": False, "scale": 1.0}
    return [
        # one decoded token: latency; the expert layer takes E4M3 rows
        {"name": "norm_1", "op": "norm", "rows": 1, "H": 7168, "groups": 0, "codes": True, "kept": False, "pad": 0},
        # 11 ragged prompts with a gate each, x a slice of a wider projection's rows, rows kept for the backward pass
        {"name": "norm_1003", "op": "norm", "rows": 1003, "H": 2048, "groups": 11, "codes": False, "kept": True,
         "pad": 576},
        # the repository's 8192-token layer in training: 16 sequences
        {"name": "norm_8192", "op": "norm", "rows": 8192, "H": 7168, "groups": 16, "codes": False, "kept": True,
         "pad": 0},
        # the backward pass of a small batch, from bf16 rows, one learned gate for all
        {"name": "norm_grad_256", "op": "norm_grad", "rows": 256, "H": 7168, "groups": 1, "kept": False, "pad": 0},
        # ragged sequences, a gate each, rows kept in 8 bits
        {"name": "norm_grad_1003", "op": "norm_grad", "rows": 1003, "H": 2048, "groups": 11, "kept": True, "pad": 0},
        # a smaller model's batch, bf16 rows inside wider ones, no gate
        {"name": "norm_grad_16384", "op": "norm_grad", "rows": 16384, "H": 2048, "groups": 0, "kept": False,
         "pad": 64},
        # the 8192-token layer, rows kept in 8 bits
        {"name": "norm_grad_8192", "op": "norm_grad", "rows": 8192, "H": 7168, "groups": 16, "kept": True, "pad": 0},
        # the losses of the 256-token layer's router
        dict(r1, name="balance_256", op="balance", T=256, seqs=1, z=False),
        # a smaller router, ragged sequences
        dict(small, name="balance_1003", op="balance", T=1003, seqs=11, z=True),
        # a training batch of 16 sequences of the R1 models' router
        dict(r1, name="balance_65536", op="balance", T=65536, seqs=16, z=True),
        # the logits' gradients of the same two
        dict(small, name="router_grad_1003", op="router_grad", T=1003, seqs=11, z=True, half=True),
        dict(r1, name="router_grad_65536", op="router_grad", T=65536, seqs=16, z=False, half=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "router_grad"])
    if op in ("norm", "norm_grad"):
        rows = _log_int(rng, 1, 8192)
        case = {"op": op, "rows": rows, "H": 8 * _log_int(rng, 32, 896),
                "groups": rng.choice([0, 1, min(rows, rng.randint(2, 40))]), "kept": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 64, 576])}
        if op == "norm":
            case["codes"] = rng.random() < 0.4
        elif case["kept"]:
            case["pad"] = 0
        return case
    T = _log_int(rng, 1, 65536)
    E = rng.choice([4 * _log_int(rng, 2, 64), _log_int(rng, 8, 255)])
    case = {"op": op, "T": T, "E": E, "k": rng.randint(1, min(10, E)), "score": rng.choice(["softmax", "sigmoid"]),
            "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
            "seqs": rng.randint(1, min(T, 48)), "z": rng.random() < 0.5}
    if op == "router_grad":
        case["half"] = rng.random() < 0.4
    return case


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _offsets(host, n, parts):
    """n rows cut into `parts` runs of random lengths of at least one."""
    cuts = np.sort(host.permutation(n - 1)[:parts - 1] + 1)
    return torch.from_numpy(np.concatenate([[0], cuts, [n]]).astype(np.int32)).cuda()


def _rows8(v):
    """fp32 rows as E4M3 codes and one scale a row."""
    amax = v.abs().amax(dim=1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), scale


def _wide(v, pad):
    """v as the first columns of rows `pad` elements longer."""
    if not pad:
        return v
    buf = torch.full((v.shape[0], v.shape[1] + pad), 7.0, dtype=v.dtype, device=v.device)
    buf[:, :v.shape[1]] = v
    return buf[:, :v.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = np.random.Generator(np.random.PCG64(int(seed)))
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        rows, H, G = case["rows"], case["H"], case["groups"]
        # a residual stream: a few channels far larger than the others
        spread = torch.exp(0.7 * _randn(g, H))
        x = (0.3 * _randn(g, rows, H)).to(BF16)
        residual = (_randn(g, rows, H) * spread).to(BF16)
        s["post"] = (1.0 + 0.2 * _randn(g, H)).to(BF16)
        s["pre"] = (1.0 + 0.2 * _randn(g, H)).to(BF16)
        s["gate"] = (0.5 + 0.3 * _randn(g, G, H)).to(BF16) if G else None
        s["offsets"] = _offsets(host, rows, G) if G > 1 else None
        s["a"], s["c"] = 0.9, 1.25
        if case["op"] == "norm":
            s["x"], s["residual"] = _wide(x, case["pad"]), residual
        else:
            # what the forward pass left: its input and its residual stream, as they are or in 8 bits
            xf = x.float()
            rx = torch.rsqrt(xf.square().mean(dim=1) + EPS)
            h = s["c"] * (xf * rx[:, None] * s["post"].float())
            if G:
                h = h * s["gate"].float()[_group_of(s["offsets"], rows)]
            h = h + s["a"] * residual.float()
            s["rstd"] = torch.stack([rx, torch.rsqrt(h.square().mean(dim=1) + EPS)], dim=1).contiguous()
            if case["kept"]:
                s["x"], s["x_scale"] = _rows8(xf)
                s["h"], s["h_scale"] = _rows8(h)
            else:
                s["x"], s["x_scale"], s["h"], s["h_scale"] = _wide(x, case["pad"]), None, h.to(BF16), None
            s["dout"] = _randn(g, rows, H).to(BF16)
            s["dres"] = _randn(g, rows, H).to(BF16)
    else:
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        # some experts are liked more than others
        s["z"] = 1.2 * _randn(g, T, E) + 0.5 * _randn(g, E)
        s["offsets"] = _offsets(host, T, S)
        # chosen with a bias on the scores, listed in ascending order as the router does
        choice = s["z"] + 0.3 * _randn(g, E)
        s["ids"] = torch.sort(torch.topk(choice, k, dim=1)[1], dim=1)[0].to(torch.int32)
        if case["op"] == "router_grad":
            of = _group_of(s["offsets"], T)
            flat = (of[:, None] * E + s["ids"]).reshape(-1)
            s["counts"] = torch.bincount(flat, minlength=S * E).view(S, E).to(torch.int32)
            s["dw"] = _randn(g, T, k) / T
            s["dbalance"] = (0.5 + torch.rand(S, generator=g, device="cuda")) * (0.1 / S)
            s["dz"] = (0.5 + torch.rand(S, generator=g, device="cuda")) * (0.01 / S) if case["z"] else None
    if own:
        s["own"] = _handles(s)
    return s


def _handles(s):
    """What a program that calls the library keeps: its objects, workspaces and output buffers."""
    from moe_expert_grouped_split_gb300 import binding as B
    case = s["case"]
    f32, cuda = torch.float32, "cuda"
    h = {}
    if case["op"] in ("norm", "norm_grad"):
        rows, H, G = case["rows"], case["H"], case["groups"]
        h["norm"] = B.SandwichNorm(H, rows, pre_weight=s["pre"], post_weight=s["post"], block_scale=s["c"],
                                   residual_scale=s["a"], eps=EPS, max_groups=G)
        bf = lambda: torch.empty((rows, H), dtype=BF16, device=cuda)  # noqa: E731
        e4 = lambda: torch.empty((rows, H), dtype=F8, device=cuda)  # noqa: E731
        one = lambda *n: torch.empty(n, dtype=f32, device=cuda)  # noqa: E731
        if case["op"] == "norm":
            h["o"] = {"out": bf(), "residual_out": bf()}
            if case["codes"]:
                h["o"].update(codes=e4(), row_scale=one(rows))
            if case["kept"]:
                h["o"].update(x_codes=e4(), x_scale=one(rows), h_codes=e4(), h_scale=one(rows), rstd=one(rows, 2))
        else:
            h["o"] = {"dx": bf(), "dresidual": bf(), "dpost_weight": one(H), "dpre_weight": one(H)}
            if G:
                h["o"]["dgate"] = one(G, H)
    else:
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        h["rt"] = B.Runtime(64, 64, E, k, 0, T, 1, 0, min_ws_bytes=B.dwdp_balance_workspace_bytes(T, E, S))
        h["scoring"] = B.scoring(score=B.SCORE_SIGMOID if case["score"] == "sigmoid" else B.SCORE_SOFTMAX,
                                 renormalize=case["renorm"], scale=case["scale"])
        if case["op"] == "balance":
            h["out"] = B.BalanceBuffers(S, E, z=case["z"])
        else:
            h["dlogits"] = torch.empty((T, E), dtype=BF16 if case["half"] else f32, device=cuda)
    return h


def run(state):
    f = {"norm": (_norm, _own_norm), "norm_grad": (_norm_grad, _own_norm_grad), "balance": (_balance, _own_balance),
         "router_grad": (_router_grad, _own_router_grad)}[state["case"]["op"]]
    return f[1](state) if own else f[0](state)


# ------------------------------------------------------- the plain forms --
def _group_of(offsets, rows):
    """The run of each row, whole numbers in 64 bits."""
    if offsets is None:
        return torch.zeros(rows, dtype=torch.int64, device="cuda")
    at = torch.arange(rows, device=offsets.device)
    return (at[:, None] >= offsets[None, 1:-1]).sum(dim=1)


def _gate(s, rows):
    if s["gate"] is None:
        return 1.0
    return s["gate"].float()[_group_of(s["offsets"], rows)]


def _norm(s):
    c = s["case"]
    x = s["x"].float()
    rx = torch.rsqrt(x.square().mean(dim=1) + EPS)
    h = s["a"] * s["residual"].float() + s["c"] * _gate(s, c["rows"]) * (x * rx[:, None] * s["post"].float())
    rh = torch.rsqrt(h.square().mean(dim=1) + EPS)
    y = h * rh[:, None] * s["pre"].float()
    r = {"out": y.to(BF16), "residual_out": h.to(BF16)}
    if c["codes"]:
        r["codes"], r["row_scale"] = _rows8(y)
    if c["kept"]:
        r["x_codes"], r["x_scale"] = _rows8(x)
        r["h_codes"], r["h_scale"] = _rows8(h)
        r["rstd"] = torch.stack([rx, rh], dim=1)
    return r


def _values(codes, scale):
    return codes.float() if scale is None else codes.float() * scale[:, None]


def _norm_grad(s):
    rows, G = s["case"]["rows"], s["case"]["groups"]
    rx, rh = s["rstd"][:, :1], s["rstd"][:, 1:]
    post, pre, dout = s["post"].float(), s["pre"].float(), s["dout"].float()
    xhat = _values(s["x"], s["x_scale"]) * rx
    hhat = _values(s["h"], s["h_scale"]) * rh
    gy = dout * pre
    dh = s["dres"].float() + rh * (gy - hhat * (gy * hhat).mean(dim=1, keepdim=True))
    dn = s["c"] * _gate(s, rows) * dh
    gn = dn * post
    r = {"dx": (rx * (gn - xhat * (gn * xhat).mean(dim=1, keepdim=True))).to(BF16), "dresidual": (s["a"] * dh).to(BF16),
         "dpost_weight": (dn * xhat).sum(dim=0), "dpre_weight": (dout * hhat).sum(dim=0)}
    if G:
        mine = (_group_of(s["offsets"], rows)[None, :] == torch.arange(G, device=dh.device)[:, None]).float()
        r["dgate"] = mine @ (s["c"] * dh * (xhat * post))
    return r


def _shares(z, score):
    """(scores, each token's scores over their sum)"""
    if score == "sigmoid":
        v = 1.0 / (1.0 + torch.exp(-z))
        return v, v / v.sum(dim=1, keepdim=True)
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    return p, p


def _log_sum_exp(z):
    m = z.amax(dim=1)
    return m + torch.log(torch.exp(z - m[:, None]).sum(dim=1))


def _balance(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    p = _shares(s["z"], c["score"])[1]
    of = _group_of(s["offsets"], T)
    lengths = (s["offsets"][1:] - s["offsets"][:-1]).float()
    mine = (of[None, :] == torch.arange(S, device=of.device)[:, None]).float()
    mean_p = (mine @ p) / lengths[:, None]
    # whole numbers below 2^24: their fp32 sums are exact
    chosen = torch.zeros_like(p).scatter_(1, s["ids"].long(), 1.0)
    counts = mine @ chosen
    r = {"counts": counts.to(torch.int32), "mean_p": mean_p,
         "balance": E / (k * lengths) * (counts * mean_p).sum(dim=1)}
    if c["z"]:
        r["z"] = (mine @ _log_sum_exp(s["z"]).square()[:, None])[:, 0] / lengths
    return r


def _router_grad(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z, ids = s["z"], s["ids"].long()
    v, p = _shares(z, c["score"])
    of = _group_of(s["offsets"], T)
    lengths = (s["offsets"][1:] - s["offsets"][:-1]).float()
    # the losses: d loss / d p of every expert, then through the shares
    per_seq = E * s["counts"].float() / (k * lengths[:, None]) * (s["dbalance"] / lengths)[:, None]
    G = per_seq[of]
    if c["score"] == "sigmoid":
        total = v.sum(dim=1, keepdim=True)
        dz = v * (1.0 - v) / total * (G - (p * G).sum(dim=1, keepdim=True))
    else:
        dz = p * (G - (p * G).sum(dim=1, keepdim=True))
    if s["dz"] is not None:
        soft = _shares(z, "softmax")[0]
        dz = dz + (s["dz"] / lengths)[of][:, None] * 2.0 * _log_sum_exp(z)[:, None] * soft
    # the chosen experts' weights
    mine, dw = v.gather(1, ids), s["dw"] * c["scale"]
    if c["renorm"]:
        q = mine / mine.sum(dim=1, keepdim=True)
        d = q * (dw - (q * dw).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1.0 - mine)
        dz = dz.scatter_add(1, ids, d)
    elif c["score"] == "sigmoid":
        dz = dz.scatter_add(1, ids, dw * mine * (1.0 - mine))
    else:
        dz = dz.scatter_add(1, ids, dw * mine) - v * (dw * mine).sum(dim=1, keepdim=True)
    return dz.to(BF16) if c["half"] else dz


# ----------------------------------------------------- the library's calls --
def _own_norm(s):
    h = s["own"]
    h["norm"].forward(s["x"], residual=s["residual"], gate=s["gate"], row_offsets=s["offsets"], **h["o"])
    return h["o"]


def _own_norm_grad(s):
    h = s["own"]
    h["norm"].grad(s["x"], s["h"], s["rstd"], s["dout"], s["dres"], gate=s["gate"], row_offsets=s["offsets"],
                   x_scale=s["x_scale"], h_scale=s["h_scale"], **h["o"])
    return h["o"]


def _own_balance(s):
    h = s["own"]
    b = h["out"]
    h["rt"].balance_loss(s["z"], s["ids"], h["scoring"], b, seq_offsets=s["offsets"])
    r = {"counts": b.counts, "mean_p": b.mean_p, "balance": b.balance}
    if b.z is not None:
        r["z"] = b.z
    return r


def _own_router_grad(s):
    h = s["own"]
    h["rt"].route_scored_grad(s["z"], s["ids"], h["scoring"], h["dlogits"], dtopk_w=s["dw"], counts=s["counts"],
                              dbalance=s["dbalance"], dz=s["dz"], seq_offsets=s["offsets"])
    return h["dlogits"]


# ---------------------------------------------------------------- the work --
def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["H"]
        per = 8 + (1 if case["codes"] else 0) + (2 if case["kept"] else 0)
        small = 2 * case["H"] * (2 + case["groups"]) + case["rows"] * (4 * case["codes"] + 16 * case["kept"])
        return {"bytes": n * per + small, "flops": 12 * n}
    if case["op"] == "norm_grad":
        n = case["rows"] * case["H"]
        per = 8 + (2 if case["kept"] else 4)
        small = case["H"] * (2 * (2 + case["groups"]) + 4 * (2 + case["groups"])) + case["rows"] * (8 + 8 * case["kept"])
        return {"bytes": n * per + small, "flops": 25 * n}
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    if case["op"] == "balance":
        return {"bytes": 4 * T * (E + k) + 8 * S * E + 8 * S, "flops": 8 * T * E}
    return {"bytes": T * E * (4 + (2 if case["half"] else 4)) + 8 * T * k + 4 * S * E + 8 * S, "flops": 16 * T * E}


# ------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "balance": _exact_balance,
            "router_grad": _exact_router_grad}[case["op"]](s)


def _runs(offsets, n):
    at = [0, n] if offsets is None else offsets.tolist()
    return list(zip(at[:-1], at[1:]))


def _exact_norm(s):
    c = s["case"]
    H = c["H"]
    x = s["x"].double()
    n = s["post"].double() * x / torch.sqrt((x ** 2).sum(1, keepdim=True) / H + EPS)
    if s["gate"] is not None:
        for i, (lo, hi) in enumerate(_runs(s["offsets"], c["rows"])):
            n[lo:hi] *= s["gate"][i].double()
    h = s["c"] * n + s["a"] * s["residual"].double()
    rms = torch.sqrt((h ** 2).sum(1, keepdim=True) / H + EPS)
    y = s["pre"].double() * h / rms
    r = {"out": y, "residual_out": h}

    def rows8(name, scale_name, v):
        r[scale_name] = v.abs().max(dim=1)[0] / E4M3_MAX
        r[name] = v / r[scale_name][:, None]

    if c["codes"]:
        rows8("codes", "row_scale", y)
    if c["kept"]:
        rows8("x_codes", "x_scale", x)
        rows8("h_codes", "h_scale", h)
        r["rstd"] = torch.cat([1 / torch.sqrt((x ** 2).sum(1, keepdim=True) / H + EPS), 1 / rms], dim=1)
    return r


def _exact_norm_grad(s):
    c = s["case"]
    rows, H, G = c["rows"], c["H"], c["groups"]
    post, pre = s["post"].double(), s["pre"].double()
    dev = post.device
    dx, dres = (torch.empty((rows, H), dtype=torch.float64, device=dev) for _ in range(2))
    dpost, dpre = torch.zeros(H, dtype=torch.float64, device=dev), torch.zeros(H, dtype=torch.float64, device=dev)
    dgate = torch.zeros((max(G, 1), H), dtype=torch.float64, device=dev)

    def through(v, r, dy, w):
        """Back through v r w, r = 1 / sqrt(mean(v^2) + eps): (the input's gradient, the weight's)."""
        by = dy * w
        inner = torch.einsum("rc,rc->r", by, v)[:, None] * r ** 3 / H
        return by * r - v * inner, torch.einsum("rc,rc->c", dy, v * r)

    for i, (lo, hi) in enumerate(_runs(s["offsets"], rows)):
        at = slice(lo, hi)
        x, h = (s[n][at].double() * (s[n + "_scale"][at].double()[:, None] if s[n + "_scale"] is not None else 1.0)
                for n in "xh")
        rx, rh = s["rstd"][at].double().split(1, dim=1)
        back, dw = through(h, rh, s["dout"][at].double(), pre)
        dpre += dw
        dh = back + s["dres"][at].double()
        dres[at] = s["a"] * dh
        g = s["gate"][i].double() if G else torch.ones(H, dtype=torch.float64, device=dev)
        dgate[i] = s["c"] * torch.einsum("rc,rc->c", dh, x * rx) * post
        dx[at], dw = through(x, rx, s["c"] * dh * g, post)
        dpost += dw
    r = {"dx": dx, "dresidual": dres, "dpost_weight": dpost, "dpre_weight": dpre}
    if G:
        r["dgate"] = dgate
    return r


def _exact_shares(z, score):
    if score == "softmax":
        return torch.softmax(z, dim=1)
    v = torch.sigmoid(z)
    return v / v.sum(dim=1, keepdim=True)


def _exact_balance(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    counts, mean_p, balance, zs = [], [], [], []
    for lo, hi in _runs(s["offsets"], c["T"]):
        z = s["z"][lo:hi].double()
        counts.append(torch.bincount(s["ids"][lo:hi].reshape(-1).long(), minlength=E))
        mean_p.append(_exact_shares(z, c["score"]).mean(dim=0))
        balance.append((counts[-1].double() / ((hi - lo) * k) * E * mean_p[-1]).sum())
        zs.append(torch.logsumexp(z, dim=1).square().mean())
    r = {"counts": torch.stack(counts), "mean_p": torch.stack(mean_p), "balance": torch.stack(balance)}
    if c["z"]:
        r["z"] = torch.stack(zs)
    return r


def _exact_router_grad(s):
    # the losses and weights themselves, and torch's derivative of them
    c = s["case"]
    E, k = c["E"], c["k"]
    out = torch.empty((c["T"], E), dtype=torch.float64, device=s["z"].device)
    for b, (lo, hi) in enumerate(_runs(s["offsets"], c["T"])):
        z = s["z"][lo:hi].double().requires_grad_(True)
        f = s["counts"][b].double() / ((hi - lo) * k) * E
        loss = float(s["dbalance"][b]) * (f * _exact_shares(z, c["score"]).mean(dim=0)).sum()
        if s["dz"] is not None:
            loss = loss + float(s["dz"][b]) * torch.logsumexp(z, dim=1).square().mean()
        v = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)
        w = torch.take_along_dim(v, s["ids"][lo:hi].long(), dim=1)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        loss = loss + c["scale"] * (w * s["dw"][lo:hi].double()).sum()
        out[lo:hi] = torch.autograd.grad(loss, z)[0]
    return out
