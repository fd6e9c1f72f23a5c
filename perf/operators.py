"""The operators around the expert layer, as cases that can be timed and checked.

Three operators of a decoder block's second half, next to dwdp_moe_layer:

  lora   low-rank adapters of many requests beside the shared projection that
         produced `base`:  out[t] = base[t] + s_a (x[t] A_a^T) B_a^T, a = the
         token's adapter, -1 = none                      (dwdp_lora_add)
  norm   h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight as bf16 and,
         where asked for, as E4M3 codes with one scale per row
                                                         (dwdp_add_rmsnorm)
  route  softmax or sigmoid scores of x W_r^T, a bias that only steers the
         choice, groups of experts, top-k, renormalised weights, and the
         (token, slot) pairs grouped by expert           (dwdp_route_scored)

`run` computes them in elementary torch operations, or, where `own` is true,
with the calls of this library.  `exact` computes them again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    r1 = {"op": "route", "H": 7168, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4,
          "group_top2": True, "renorm": True, "scale": 2.5}
    return [
        # one decoded token: latency
        {"name": "norm_1", "op": "norm", "rows": 1, "H": 7168, "residual": True, "codes": True, "pad": 0},
        # a decode batch of the repository's 256-token layer
        {"name": "norm_256", "op": "norm", "rows": 256, "H": 7168, "residual": True, "codes": True, "pad": 0},
        # a latent inside a wider projection's rows (a row stride), ragged count, no residual, no codes
        {"name": "norm_1003_strided", "op": "norm", "rows": 1003, "H": 1536, "residual": False, "codes": False,
         "pad": 576},
        # a prefill of the repository's 8192-token layer
        {"name": "norm_8192", "op": "norm", "rows": 8192, "H": 7168, "residual": True, "codes": True, "pad": 0},
        # routing of one decoded token
        dict(r1, name="route_1", T=1),
        # the 256-token layer
        dict(r1, name="route_256", T=256),
        # a smaller router: softmax, no groups, no bias, weights as they are
        {"name": "route_1003_softmax", "op": "route", "T": 1003, "H": 2048, "E": 64, "k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top2": False, "renorm": False, "scale": 1.0},
        # the 8192-token layer
        dict(r1, name="route_8192", T=8192),
        # one decoded token of one tenant
        {"name": "lora_1", "op": "lora", "T": 1, "K": 7168, "N": 7168, "R": 16, "adapters": 8, "requests": 1,
         "bare": 0, "pad": 0},
        # a decode batch: 64 tokens of 64 tenants
        {"name": "lora_64_tenants", "op": "lora", "T": 64, "K": 7168, "N": 7168, "R": 16, "adapters": 64,
         "requests": 64, "bare": 0, "pad": 0},
        # a mixed batch of ragged prompts, some without an adapter, into a slice of a fused projection's rows
        {"name": "lora_517_rank64", "op": "lora", "T": 517, "K": 2048, "N": 1536, "R": 64, "adapters": 16,
         "requests": 11, "bare": 3, "pad": 512},
        # a prefill batch of 16 prompts
        {"name": "lora_8192", "op": "lora", "T": 8192, "K": 7168, "N": 7168, "R": 16, "adapters": 16, "requests": 16,
         "bare": 0, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "lora"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "H": 8 * _log_int(rng, 64, 896),
                "residual": rng.random() < 0.7, "codes": rng.random() < 0.5, "pad": rng.choice([0, 0, 64, 576])}
    if op == "route":
        groups = rng.choice([1, 2, 4, 8])
        E = groups * 4 * _log_int(rng, max(4, 16 // groups), 64 // groups)
        top = 1 if groups == 1 else rng.randint(max(1, groups // 2), groups)
        return {"op": op, "T": _log_int(rng, 1, 8192), "H": 64 * _log_int(rng, 8, 112), "E": E,
                "k": min(rng.randint(1, 10), top * (E // groups)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.6, "groups": groups, "top_groups": top, "group_top2": rng.random() < 0.5,
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    T = _log_int(rng, 1, 8192)
    requests = T if T <= 64 and rng.random() < 0.7 else rng.randint(1, min(T, 24))
    return {"op": op, "T": T, "K": 8 * _log_int(rng, 64, 896), "N": 8 * _log_int(rng, 64, 896),
            "R": rng.choice([8, 16, 16, 32, 64]) if T <= 2048 else rng.choice([8, 16]),
            "adapters": rng.randint(1, 16 if T > 64 else 64),
            "requests": requests, "bare": rng.choice([0, 0, 1, requests // 4]), "pad": rng.choice([0, 0, 512])}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _grid(v, step, most):
    """v rounded to whole multiples of step, at most `most` of them: exact in bf16 for most < 256."""
    return (v / step).round().clamp(-most, most).mul(step).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = np.random.Generator(np.random.PCG64(int(seed)))
    s = {"case": case}
    if case["op"] == "norm":
        rows, H = case["rows"], case["H"]
        # a residual stream: a few channels far larger than the others
        spread = torch.exp(0.7 * _randn(g, H))
        wide = torch.empty((rows, H + case["pad"]), dtype=BF16, device="cuda")
        wide[:, :H] = _randn(g, rows, H)
        if case["pad"]:
            wide[:, H:] = 7.0
        s["x"] = wide[:, :H]
        s["residual"] = (_randn(g, rows, H) * spread).to(BF16) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(g, H)).to(BF16)
    elif case["op"] == "route":
        T, H, E = case["T"], case["H"], case["E"]
        # The chosen ids are whole numbers and have to be equal, so the logits
        # have to be: tokens and router weights lie on grids on which every
        # order of summation gives the same fp32 logit (tokens ~ N(0, 1) in
        # steps of 1/16, weights ~ N(0, 1/H) in steps of 1/32 to 1/64 of their
        # deviation, so a logit ~ N(0, 1) is a multiple of about 2^-16).
        s["x"] = _grid(_randn(g, T, H), 1.0 / 16.0, 127)
        std = 1.0 / math.sqrt(H)
        s["w"] = _grid(_randn(g, E, H) * std, 2.0 ** math.floor(math.log2(std / 32.0)), 255)
        s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
    else:
        T, K, N, R, n = case["T"], case["K"], case["N"], case["R"], case["adapters"]
        s["x"] = _randn(g, T, K).to(BF16)
        s["a"] = (_randn(g, n, R, K) / math.sqrt(K)).to(BF16)
        s["b"] = (0.5 * _randn(g, n, N, R) / math.sqrt(R)).to(BF16)
        s["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
        s["base"] = torch.empty((T, N + case["pad"]), dtype=BF16, device="cuda")
        s["base"].copy_(_randn(g, T, N + case["pad"]))
        s["base"] = s["base"][:, :N]
        # requests of random lengths, one after the other; the first `bare` have no adapter
        cuts = np.sort(host.permutation(T - 1)[:case["requests"] - 1] + 1)
        lengths = np.diff(np.concatenate([[0], cuts, [T]]))
        of = np.concatenate([np.full(min(case["bare"], case["requests"]), -1), np.arange(case["requests"]) % n])
        of = host.permutation(of[:case["requests"]])
        s["ids"] = torch.from_numpy(np.repeat(of, lengths).astype(np.int32)).cuda()
    if own:
        s["own"] = _handles(case)
    return s


def _handles(case):
    """What a program that calls the library keeps: its context, workspace and output buffers."""
    from moe_expert_grouped_split_gb300 import binding as B
    h = {"B": B}
    if case["op"] == "norm":
        rows, H = case["rows"], case["H"]
        h["out"] = torch.empty((rows, H), dtype=BF16, device="cuda")
        h["residual"] = torch.empty((rows, H), dtype=BF16, device="cuda") if case["residual"] else None
        h["codes"] = torch.empty((rows, H), dtype=torch.float8_e4m3fn, device="cuda") if case["codes"] else None
        h["row_scale"] = torch.empty(rows, dtype=torch.float32, device="cuda") if case["codes"] else None
    elif case["op"] == "route":
        h["rt"] = B.Runtime(case["H"], 64, case["E"], case["k"], 0, case["T"], 1, 0)
        h["rb"] = B.RouteBuffers(case["T"], case["E"], case["k"])
        h["scoring"] = B.scoring(score=B.SCORE_SIGMOID if case["score"] == "sigmoid" else B.SCORE_SOFTMAX,
                                 n_groups=case["groups"], top_groups=case["top_groups"],
                                 group_score=B.GROUP_TOP2 if case["group_top2"] else B.GROUP_MAX,
                                 renormalize=case["renorm"], scale=case["scale"])
    else:
        h["rt"] = B.Runtime(64, 64, 1, 1, 0, case["T"], 1, 0,
                            min_ws_bytes=B.dwdp_lora_workspace_bytes(case["T"], case["K"], case["N"], case["R"]))
        h["out"] = torch.empty((case["T"], case["N"] + case["pad"]), dtype=BF16, device="cuda")[:, :case["N"]]
    return h


def run(state):
    f = {"norm": (_norm, _own_norm), "route": (_route, _own_route), "lora": (_lora, _own_lora)}[state["case"]["op"]]
    return f[1](state) if own else f[0](state)


# ------------------------------------------------------- the plain forms --
def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    r = {"out": y.to(BF16)}
    if s["residual"] is not None:
        r["residual"] = h.to(BF16)
    if s["case"]["codes"]:
        amax = y.abs().amax(dim=1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        r["codes"] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        r["row_scale"] = scale
    return r


def _route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    # exact in 32 bits on the inputs' grid; what follows it decides between
    # values next to each other, in 64 bits
    z = (s["x"].float() @ s["w"].float().t()).double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True)[0]
        group = best[:, :, :2].sum(dim=2) if c["group_top2"] and E // G > 1 else best[:, :, 0]
        kept = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        allowed = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        choice = torch.where(allowed[:, :, None].expand(T, G, E // G).reshape(T, E), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    ids = torch.sort(ids, dim=1)[0]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    flat = ids.reshape(-1)
    perm = torch.sort(flat, stable=True)[1]
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=z.device)
    counts = (flat[:, None] == torch.arange(E, device=z.device)).sum(dim=0)
    offsets = torch.cat([torch.zeros(1, dtype=counts.dtype, device=z.device), counts.cumsum(0)])
    i32 = torch.int32
    return {"topk_ids": ids.to(i32), "topk_w": (w * c["scale"]).float(), "counts": counts.to(i32),
            "offsets": offsets.to(i32), "perm": perm.to(i32), "inv_perm": inv.to(i32)}


def _lora(s):
    a, b, ids = s["a"].float(), s["b"].float(), s["ids"]
    n, R, K = a.shape
    # every adapter's product, then each token's own kept: no loop over adapters
    v = (s["x"].float() @ a.reshape(n * R, K).t()).view(-1, n, R)
    mine = torch.where(ids[:, None] == torch.arange(n, device=ids.device), s["scale"], 0.0)
    v = (v * mine[:, :, None]).reshape(-1, n * R)
    return (s["base"].float() + v @ b.permute(0, 2, 1).reshape(n * R, -1)).to(BF16)


# ----------------------------------------------------- the library's calls --
def _own_norm(s):
    h = s["own"]
    x = s["x"]
    h["B"].dwdp_add_rmsnorm(x, x.shape[0], x.shape[1], s["weight"], EPS, h["out"], residual=s["residual"],
                            residual_out=h["residual"], codes=h["codes"], row_scale=h["row_scale"],
                            x_stride=x.stride(0))
    r = {"out": h["out"]}
    if h["residual"] is not None:
        r["residual"] = h["residual"]
    if h["codes"] is not None:
        r["codes"], r["row_scale"] = h["codes"], h["row_scale"]
    return r


def _own_route(s):
    h = s["own"]
    rb = h["rb"]
    h["rt"].route_scored(s["x"], s["w"], s["bias"], h["scoring"], rb)
    return {"topk_ids": rb.topk_ids, "topk_w": rb.topk_w, "counts": rb.counts, "offsets": rb.offsets,
            "perm": rb.perm, "inv_perm": rb.inv_perm}


def _own_lora(s):
    h = s["own"]
    h["rt"].lora_add(s["x"], s["a"], s["b"], s["scale"], s["ids"], s["base"], h["out"])
    return h["out"]


# ---------------------------------------------------------------- the work --
def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["H"]
        b = n * (2 + 2 + (4 if case["residual"] else 0) + (1 if case["codes"] else 0))
        return {"bytes": b + 2 * case["H"] + (4 * case["rows"] if case["codes"] else 0), "flops": 4 * n}
    if case["op"] == "route":
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        return {"bytes": 2 * H * (T + E) + 16 * T * k + 8 * E + (4 * E if case["bias"] else 0),
                "flops": 2 * T * H * E}
    T, K, N, R = case["T"], case["K"], case["N"], case["R"]
    with_adapter = case["requests"] - min(case["bare"], case["requests"])
    used = min(with_adapter, case["adapters"])
    rows = T * with_adapter / case["requests"]  # on average: the lengths are drawn
    return {"bytes": 2 * rows * K + 4 * T * N + 2 * used * R * (K + N) + 4 * T, "flops": 2 * rows * R * (K + N)}


# ------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm": _exact_norm, "route": _exact_route, "lora": _exact_lora}[case["op"]](s)


def _exact_norm(s):
    d = lambda t: t.cpu().double().numpy()  # noqa: E731
    h = d(s["x"]) + (d(s["residual"]) if s["residual"] is not None else 0.0)
    y = h / np.sqrt(np.mean(h * h, axis=1) + EPS)[:, None] * d(s["weight"])
    r = {"out": y}
    if s["residual"] is not None:
        r["residual"] = h
    if s["case"]["codes"]:
        r["row_scale"] = np.abs(y).max(axis=1) / E4M3_MAX
        r["codes"] = y / r["row_scale"][:, None]
    return r


def _exact_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = (s["x"].double() @ s["w"].double().t()).cpu().numpy()
    if c["score"] == "sigmoid":
        score = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    else:
        m = z.max(axis=1, keepdims=True)
        score = np.exp(z - (m + np.log(np.exp(z - m).sum(axis=1, keepdims=True))))
    choice = score + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    if G > 1:
        by = choice.reshape(T, G, E // G)
        first = by.max(axis=2)
        if c["group_top2"] and E // G > 1:
            first = first + np.partition(by, -2, axis=2)[:, :, -2]
        lost = np.argsort(-first, axis=1, kind="stable")[:, c["top_groups"]:]
        by = by.copy()
        np.put_along_axis(by, lost[:, :, None].repeat(E // G, axis=2), -np.inf, axis=1)
        choice = by.reshape(T, E)
    ids = np.sort(np.argsort(-choice, axis=1, kind="stable")[:, :k], axis=1)
    w = np.take_along_axis(score, ids, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    counts = np.bincount(ids.reshape(-1), minlength=E)
    perm = np.argsort(ids.reshape(-1), kind="stable")
    return {"topk_ids": ids, "topk_w": w * c["scale"], "counts": counts,
            "offsets": np.concatenate([[0], np.cumsum(counts)]), "perm": perm, "inv_perm": np.argsort(perm)}


def _exact_lora(s):
    out = s["base"].double()
    for i in range(s["a"].shape[0]):  # adapter by adapter, on its own tokens
        at = torch.nonzero(s["ids"] == i)[:, 0]
        v = s["x"][at].double() @ s["a"][i].double().t()
        out[at] += float(s["scale"][i]) * (v @ s["b"][i].double().t())
    return out
