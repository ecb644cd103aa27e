"""Cases for the operators around the seam: embedding rows into the residual
streams and their gradient, the norms around a block with its gate and residual
scale and their gradient, and the routing of tokens to experts and its gradient.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, where ``own`` is set, through the
framework's entry points.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
WORKSPACE_BYTES = 64 << 20  # one zeroed workspace, large enough for every case here


def listed():
    return [
        # a decode step of 64 sequences: each token's row into the four streams that the first seam reads
        {"name": "embed_decode", "op": "embed", "T": 64, "V": 131072, "H": 5120, "streams": 4, "dtype": "bf16",
         "ids": "int64", "shards": 1},
        # the prefill of the seam's largest workload
        {"name": "embed_prefill", "op": "embed", "T": 16384, "V": 131072, "H": 5120, "streams": 4, "dtype": "bf16",
         "ids": "int64", "shards": 1},
        # a small model's training step; one residual stream, odd token count, gradient in the table's type
        {"name": "embed_grad_small", "op": "embed_grad", "T": 1003, "V": 32000, "H": 512, "streams": 1,
         "dtype": "bf16", "grad": "bf16", "ids": "int32", "shards": 1},
        # a training step of the seam's largest workload: four streams summed, whole gradient table in 32 bits
        {"name": "embed_grad_large", "op": "embed_grad", "T": 16384, "V": 131072, "H": 5120, "streams": 4,
         "dtype": "bf16", "grad": "fp32", "ids": "int64", "shards": 1},
        # a decode step of four tokens
        {"name": "block_norm_decode", "op": "block_norm", "T": 4, "H": 5120, "dtype": "bf16", "gate": "token",
         "post": True, "pre": True},
        # prefill or a training step at full size
        {"name": "block_norm_prefill", "op": "block_norm", "T": 16384, "H": 5120, "dtype": "bf16", "gate": "channel",
         "post": True, "pre": True},
        # a small model trained in 32 bits, odd token count, no norm after the block
        {"name": "block_norm_grad_small", "op": "block_norm_grad", "T": 1023, "H": 1024, "dtype": "fp32",
         "gate": "token", "post": False, "pre": True},
        # the training step at full size with every part
        {"name": "block_norm_grad_large", "op": "block_norm_grad", "T": 16384, "H": 5120, "dtype": "bf16",
         "gate": "channel", "post": True, "pre": True},
        # a decode step of 64 tokens over 256 experts in 8 groups
        {"name": "route_decode", "op": "route", "T": 64, "E": 256, "groups": 8, "top_groups": 4, "k": 8,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32", "masked": False},
        # a large prefill batch, the same router
        {"name": "route_prefill", "op": "route", "T": 131072, "E": 256, "groups": 8, "top_groups": 4, "k": 8,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32", "masked": False},
        # a small softmax router without renormalisation: every logit has a gradient
        {"name": "route_grad_softmax", "op": "route_grad", "T": 4159, "E": 64, "groups": 1, "top_groups": 1, "k": 6,
         "score": "softmax", "bias": False, "renorm": False, "dtype": "bf16", "masked": False},
        # the gradient of the large sigmoid router
        {"name": "route_grad_large", "op": "route_grad", "T": 131072, "E": 256, "groups": 8, "top_groups": 4, "k": 8,
         "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32", "masked": False},
    ]


def _log_int(rng, lo, hi):
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n in (384, 3072) else n


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "block_norm", "block_norm_grad", "route", "route_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("route", "route_grad"):
        groups, per = rng.choice([(1, 8), (1, 60), (1, 64), (4, 16), (8, 20), (8, 32), (1, 128), (4, 96), (1, 512)])
        E = groups * per
        top_groups = rng.randint(1, groups)
        renorm = rng.random() < 0.6
        k = rng.randint(2 if renorm else 1, min(10, top_groups * per))  # one renormalised weight is a constant
        score = rng.choice(["sigmoid", "softmax"])
        return {"op": op, "T": _log_int(rng, 1, 131072 * 256 // max(E, 256)), "E": E, "groups": groups,
                "top_groups": top_groups, "k": k, "score": score,
                # a bias with softmax scores is left to the tests: sums in another order can swap near ties
                "bias": score == "sigmoid" and rng.random() < 0.7, "renorm": renorm,
                "dtype": rng.choice(["fp32", "fp32", "bf16"]), "masked": rng.random() < 0.3}
    H = 8 * _log_int(rng, 8, 1024)
    most = 16384 * 5120 * 2 // (H * SIZES[dtype])
    if op in ("block_norm", "block_norm_grad"):
        post = rng.random() < 0.7
        return {"op": op, "T": _log_int(rng, 1, min(65536, most)), "H": H, "dtype": dtype,
                "gate": rng.choice(["none", "channel", "token"]), "post": post, "pre": rng.random() < 0.9}
    streams = rng.choice([1, 1, 2, 4])
    V = min(_log_int(rng, 1000, 131072), 131072 * 5120 // H)
    c = {"op": op, "T": _log_int(rng, 1, min(65536, most)), "V": V, "H": H, "streams": streams, "dtype": dtype,
         "ids": rng.choice(["int32", "int64"])}
    c["shards"] = rng.choice([1, 1, 1, 8]) if c["T"] >= 64 else 1  # a shard of the vocabulary; some tokens are in it
    if op == "embed_grad":
        c["grad"] = rng.choice([dtype, "fp32"])
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(case, g):
    """Token ids with the skew of text: the rank is log-uniform over the vocabulary, ranks shuffled."""
    n = case["V"] * case["shards"]
    rank = (torch.rand(case["T"], device="cuda", generator=g, dtype=torch.float64) * math.log(n + 1)).exp().long() - 1
    ids = torch.randperm(n, device="cuda", generator=g)[rank.clamp_(0, n - 1)]
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64), (case["shards"] // 2) * case["V"]


def prepare(case, seed):
    g = _gen(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32)

    s = {"case": case, "ws": torch.zeros(WORKSPACE_BYTES, device="cuda", dtype=torch.uint8)}
    op = case["op"]
    if op in ("embed", "embed_grad"):
        T, V, H, S, dt = case["T"], case["V"], case["H"], case["streams"], DTYPES[case["dtype"]]
        s["ids"], s["first"] = _ids(case, g)
        s["scale"] = math.sqrt(H) if op == "embed" else 0.5
        if op == "embed":
            s["table"] = torch.empty(V, H, device="cuda", dtype=dt).normal_(0, 0.02, generator=g)
            s["out"] = torch.empty(T, S, H, device="cuda", dtype=dt)
        else:
            s["dout"] = torch.empty(T, S, H, device="cuda", dtype=dt).normal_(0, 1, generator=g)
            s["dtable"] = torch.empty(V, H, device="cuda", dtype=DTYPES[case["grad"]])
    elif op in ("block_norm", "block_norm_grad"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        s["y"], s["r"] = (3 * normal(T, H)).to(dt), (2 * normal(T, H)).to(dt)
        s["gamma_post"] = (1 + 0.1 * normal(H)).to(dt) if case["post"] else None
        s["gamma_pre"] = (1 + 0.1 * normal(H)).to(dt) if case["pre"] else None
        s["gate"] = {"none": None, "channel": (0.5 + 0.1 * normal(H)).to(dt),
                     "token": 2 * torch.sigmoid(normal(T))}[case["gate"]]
        s["scale"], s["eps"] = 0.75, 1e-6
        f32 = dict(device="cuda", dtype=torch.float32)
        s["rstd_post"] = torch.empty(T, **f32) if case["post"] else None
        s["rstd_pre"] = torch.empty(T, **f32) if case["pre"] else None
        if op == "block_norm":
            s["r_out"] = torch.empty(T, H, device="cuda", dtype=dt)
            s["norm"] = torch.empty(T, H, device="cuda", dtype=dt) if case["pre"] else None
        else:  # what the forward pass left, and the gradients that come back
            out = _block_norm(s)
            s["r_out"], s["rstd_post"], s["rstd_pre"] = out["r_out"], out.get("rstd_post"), out.get("rstd_pre")
            s["dr_out"] = normal(T, H).to(dt)
            s["dnorm"] = normal(T, H).to(dt) if case["pre"] else None
            s["dy"], s["dr"] = (torch.empty(T, H, device="cuda", dtype=dt) for _ in range(2))
            s["dgamma_post"] = torch.empty(H, **f32) if case["post"] else None
            s["dgamma_pre"] = torch.empty(H, **f32) if case["pre"] else None
            s["dgate"] = {"none": None, "channel": torch.empty(H, **f32), "token": torch.empty(T, **f32)}[case["gate"]]
    else:
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = (1.5 * normal(T, E)).to(DTYPES[case["dtype"]])
        if case["masked"]:  # experts out of service, for every token; a few tokens have no expert left
            s["logits"][:, 2:][:, torch.rand(E - 2, device="cuda", generator=g) < 0.3] = -math.inf
            s["logits"][1:][torch.rand(T - 1, device="cuda", generator=g) < 0.01] = -math.inf
        s["bias"] = 0.1 * normal(E) if case["bias"] else None
        s["scale"] = 2.5
        s["indices"] = torch.empty(T, k, device="cuda", dtype=torch.int32)
        s["weights"] = torch.empty(T, k, device="cuda", dtype=torch.float32)
        s["counts"] = torch.empty(E, device="cuda", dtype=torch.int32)
        if op == "route_grad":
            s["indices"] = _route(s)["indices"]
            s["dweights"] = normal(T, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ------------------------------------------------------------- plain forms --
def _embed(s):
    row = s["ids"].long() - s["first"]
    here = (row >= 0) & (row < s["case"]["V"])
    x = s["table"][torch.where(here, row, 0)].float() * s["scale"]
    x = torch.where(here[:, None], x, 0.0).to(s["table"].dtype)
    return {"out": x[:, None, :].repeat(1, s["case"]["streams"], 1)}


def _embed_grad(s):
    V, H = s["case"]["V"], s["case"]["H"]
    row = s["ids"].long() - s["first"]
    here = (row >= 0) & (row < V)
    d = s["dout"].float().sum(1) * s["scale"]
    d = torch.where(here[:, None], d, 0.0)
    acc = torch.zeros(V, H, device="cuda", dtype=torch.float32).index_add_(0, torch.where(here, row, 0), d)
    return {"dtable": acc.to(DTYPES[s["case"]["grad"]])}


def _gate(s):
    g = s["gate"]
    return None if g is None else g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _block_norm(s):
    dt, y, r = s["y"].dtype, s["y"].float(), s["r"].float()
    out = {}
    p = y
    if s["gamma_post"] is not None:
        rho = 1 / torch.sqrt((y * y).mean(1) + s["eps"])
        out["rstd_post"] = rho
        p = y * rho[:, None] * s["gamma_post"].float()
    g = _gate(s)
    x = s["scale"] * r + (p if g is None else g * p)
    out["r_out"] = x.to(dt)
    if s["gamma_pre"] is not None:
        rho = 1 / torch.sqrt((x * x).mean(1) + s["eps"])
        out["rstd_pre"] = rho
        out["norm"] = (x * rho[:, None] * s["gamma_pre"].float()).to(dt)
    return out


def _block_norm_grad(s):
    dt, y, x = s["y"].dtype, s["y"].float(), s["r_out"].float()
    out = {}
    G = s["dr_out"].float()
    if s["gamma_pre"] is not None:
        dn, rho = s["dnorm"].float(), s["rstd_pre"][:, None]
        out["dgamma_pre"] = (dn * x * rho).sum(0)
        c = s["gamma_pre"].float() * dn
        G = G + rho * (c - x * rho * rho * (c * x).mean(1, keepdim=True))
    out["dr"] = (s["scale"] * G).to(dt)
    p, rho = y, None
    if s["gamma_post"] is not None:
        rho = s["rstd_post"][:, None]
        p = y * rho * s["gamma_post"].float()
    g = _gate(s)
    dp = G if g is None else g * G
    if g is not None:
        out["dgate"] = (p * G).sum(1 if s["case"]["gate"] == "token" else 0)
    if rho is None:
        out["dy"] = dp.to(dt)
    else:
        out["dgamma_post"] = (dp * y * rho).sum(0)
        c = s["gamma_post"].float() * dp
        out["dy"] = (rho * (c - y * rho * rho * (c * y).mean(1, keepdim=True))).to(dt)
    return out


def _scores(s):
    """Scores of every expert (for softmax also the unnormalised ones, which order the experts the same way)."""
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l)
    ok = l > -math.inf
    if s["case"]["score"] == "sigmoid":
        v = 1 / (1 + torch.exp(-l))
        return ok, v, v
    m = l.max(1, keepdim=True).values
    e = torch.exp(torch.where(l == m, 0.0, l - torch.where(m == -math.inf, 0.0, m)))
    e = torch.where(ok, e, 0.0)
    total = e.sum(1, keepdim=True)
    return ok, torch.where(total > 0, e / total, 0.0), e


def _route(s):
    c = s["case"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    ok, score, order = _scores(s)
    sel = order if s["bias"] is None else score + s["bias"]
    sel = torch.where(ok, sel, -math.inf)
    if n > 1:
        best = sel.view(T, n, E // n).sort(2, descending=True).values
        second = best[:, :, 1] if E // n > 1 else torch.full_like(best[:, :, 0], -math.inf)
        group = best[:, :, 0] + torch.where(second > -math.inf, second, 0.0)
        first = group.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros(T, n, device="cuda", dtype=torch.bool).scatter_(1, first, True)
        sel = torch.where(keep.repeat_interleave(E // n, 1), sel, -math.inf)
    val, idx = sel.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    got = val > -math.inf
    if c["renorm"]:
        w = torch.where(got, order.gather(1, idx), 0.0)
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, s["scale"] * w / total, 0.0)
    else:
        w = torch.where(got, s["scale"] * score.gather(1, idx), 0.0)
    counts = torch.zeros(E, device="cuda", dtype=torch.int32).index_add_(0, idx.reshape(-1), got.reshape(-1).int())
    return {"indices": torch.where(got, idx, -1).int(), "weights": w, "counts": counts}


def _route_grad(s):
    c, scale = s["case"], s["scale"]
    ok, score, order = _scores(s)
    got = s["indices"] >= 0
    idx = torch.where(got, s["indices"], 0).long()
    dw = torch.where(got, s["dweights"], 0.0)
    v = torch.where(got, (order if c["renorm"] else score).gather(1, idx), 0.0)
    if c["renorm"]:
        total = v.sum(1, keepdim=True)
        q = torch.where(total > 0, v / total, 0.0)
        ds = dw - (q * dw).sum(1, keepdim=True)
        d = scale * q * ds if c["score"] == "softmax" else scale * q * ds * (1 - v)
        out = torch.zeros_like(score).scatter_add_(1, idx, d)
    elif c["score"] == "sigmoid":
        out = torch.zeros_like(score).scatter_add_(1, idx, scale * dw * v * (1 - v))
    else:
        up = torch.zeros_like(score).scatter_add_(1, idx, dw)
        out = scale * score * (up - (v * dw).sum(1, keepdim=True))
    return {"dlogits": out.to(s["logits"].dtype)}


PLAIN = {"embed": _embed, "embed_grad": _embed_grad, "block_norm": _block_norm, "block_norm_grad": _block_norm_grad,
         "route": _route, "route_grad": _route_grad}


# ------------------------------------------------------ the framework's own --
def _own(s):
    from mhc_residual_seam_gb300 import binding as B

    c = s["case"]
    op = c["op"]
    if op == "embed":
        B.mhc_embed(s["ids"], s["table"], s["out"], scale=s["scale"], first_id=s["first"])
        return {"out": s["out"]}
    if op == "embed_grad":
        B.mhc_embed_grad(s["ids"], s["dout"], s["dtable"], s["ws"], scale=s["scale"], first_id=s["first"])
        return {"dtable": s["dtable"]}
    if op in ("block_norm", "block_norm_grad"):
        mode = {"none": B.MHC_GATE_NONE, "channel": B.MHC_GATE_CHANNEL, "token": B.MHC_GATE_TOKEN}[c["gate"]]
        if op == "block_norm":
            B.mhc_block_norm(s["y"], s["r"], s["gamma_post"], s["gate"], s["gamma_pre"], s["r_out"], s["norm"],
                             s["rstd_post"], s["rstd_pre"], gate_mode=mode, res_scale=s["scale"], eps=s["eps"])
            names = ("r_out", "norm", "rstd_post", "rstd_pre")
        else:
            B.mhc_block_norm_grad(s["dr_out"], s["dnorm"], s["y"], s["r_out"], s["gamma_post"], s["gate"],
                                  s["gamma_pre"], s["rstd_post"], s["rstd_pre"], s["dy"], s["dr"], s["dgamma_post"],
                                  s["dgate"], s["dgamma_pre"], s["ws"], gate_mode=mode, res_scale=s["scale"])
            names = ("dy", "dr", "dgamma_post", "dgate", "dgamma_pre")
        return {n: s[n] for n in names if s[n] is not None}
    score = B.MHC_SCORE_SIGMOID if c["score"] == "sigmoid" else B.MHC_SCORE_SOFTMAX
    if op == "route":
        B.mhc_route(s["logits"], s["bias"], s["indices"], s["weights"], s["counts"], s["ws"], score=score,
                    groups=c["groups"], top_groups=c["top_groups"], renorm=c["renorm"], scale=s["scale"])
        return {n: s[n] for n in ("indices", "weights", "counts")}
    B.mhc_route_grad(s["dweights"], s["logits"], s["indices"], s["dlogits"], score=score, renorm=c["renorm"],
                     scale=s["scale"])
    return {"dlogits": s["dlogits"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        out = torch.zeros(case["T"], case["streams"], case["H"], device="cuda", dtype=torch.float64)
        row = s["ids"].long() - s["first"]
        t = torch.nonzero((row >= 0) & (row < case["V"]))[:, 0]
        out[t] = (s["table"][row[t]].double() * s["scale"])[:, None, :]
        return {"out": out}
    if op == "embed_grad":
        out = torch.zeros(case["V"], case["H"], device="cuda", dtype=torch.float64)
        row, t = torch.sort(s["ids"].long() - s["first"], stable=True)
        rows, many = torch.unique_consecutive(row, return_counts=True)
        at = 0
        for v, n in zip(rows.tolist(), many.tolist()):
            if 0 <= v < case["V"]:
                out[v] = s["dout"][t[at:at + n]].double().sum((0, 1)) * s["scale"]
            at += n
        return {"dtable": out}
    if op in ("block_norm", "block_norm_grad"):
        return _exact_block(case, {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()})
    return _exact_route(case, s)


def _exact_block(case, s):
    H, y, a, eps = case["H"], s["y"], s["scale"], s["eps"]
    one = torch.ones((), device="cuda", dtype=torch.float64)
    gate = one if s["gate"] is None else s["gate"][:, None] if case["gate"] == "token" else s["gate"]
    if case["op"] == "block_norm":
        out = {}
        if case["post"]:
            out["rstd_post"] = torch.rsqrt(y.square().sum(1) / H + eps)
            y = y * s["gamma_post"] * out["rstd_post"][:, None]
        out["r_out"] = gate * y + a * s["r"]
        if case["pre"]:
            out["rstd_pre"] = torch.rsqrt(out["r_out"].square().sum(1) / H + eps)
            out["norm"] = out["r_out"] * s["gamma_pre"] * out["rstd_pre"][:, None]
        return out
    out = {}

    def back(x, rho, gamma, d):
        """The gradients of sum(d * x / rms(x) * gamma) by x and by gamma."""
        u = x * rho[:, None]
        dg = d * gamma
        return (dg - u * ((dg * u).sum(1) / H)[:, None]) * rho[:, None], (d * u).sum(0)

    G = s["dr_out"]
    if case["pre"]:
        dx, out["dgamma_pre"] = back(s["r_out"], s["rstd_pre"], s["gamma_pre"], s["dnorm"])
        G = G + dx
    out["dr"] = G * a
    if case["post"]:
        out["dy"], out["dgamma_post"] = back(y, s["rstd_post"], s["gamma_post"], G * gate)
        y = y * s["gamma_post"] * s["rstd_post"][:, None]
    else:
        out["dy"] = G * gate
    if case["gate"] != "none":
        out["dgate"] = torch.einsum("th,th->t" if case["gate"] == "token" else "th,th->h", y, G)
    return out


def _exact_route(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, 1))  # a row with no expert left gives no number
    if case["op"] == "route":
        sel = p if s["bias"] is None else p + s["bias"].double()
        sel = sel.masked_fill(l == -math.inf, -math.inf)
        if case["groups"] > 1:
            top = sel.view(T, case["groups"], -1).topk(min(2, E // case["groups"]), 2).values
            score = top[..., 0] + (top[..., 1:].masked_fill(top[..., 1:] == -math.inf, 0).sum(2))
            out = score.argsort(dim=1, descending=True, stable=True)[:, case["top_groups"]:]
            sel.view(T, case["groups"], -1).scatter_(1, out[:, :, None].expand(-1, -1, E // case["groups"]), -math.inf)
        at = sel.argsort(dim=1, descending=True, stable=True)[:, :k]
        w = p.gather(1, at).masked_fill(sel.gather(1, at) == -math.inf, 0)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        return {"indices": None, "weights": w * s["scale"], "counts": None}
    hot = torch.zeros(T, E, device="cuda", dtype=torch.float64)
    dw = torch.zeros(T, E, device="cuda", dtype=torch.float64)
    t, j = torch.nonzero(s["indices"] >= 0, as_tuple=True)
    e = s["indices"][t, j].long()
    hot[t, e] = 1
    dw[t, e] = s["dweights"][t, j].double()
    if case["renorm"]:  # w = scale h p / sum(h p)
        total = (hot * p).sum(1, keepdim=True).clamp_min(1e-300)
        dp = hot * (dw - (dw * p).sum(1, keepdim=True) / total) / total * s["scale"]
    else:
        dp = dw * s["scale"]
    if case["score"] == "sigmoid":
        return {"dlogits": dp * p * (1 - p)}
    return {"dlogits": p * (dp - (dp * p).sum(1, keepdim=True))}


# ------------------------------------------------------------------- work --
def _distinct(case):
    """Expected number of different rows of the table that the ids name."""
    n = case["V"] * case["shards"]
    v = torch.arange(1, n + 1, dtype=torch.float64)
    p = torch.log1p(1 / v) / math.log(n + 1)
    return float((1 - (1 - p) ** case["T"]).sum()) / case["shards"]


def work(case):
    op, T = case["op"], case["T"]
    b = SIZES[case["dtype"]]
    if op in ("embed", "embed_grad"):
        H, S, idb = case["H"], case["streams"], 4 if case["ids"] == "int32" else 8
        if op == "embed":
            return {"bytes": T * idb + _distinct(case) * H * b + T * S * H * b, "flops": T * H}
        here = T / case["shards"]
        return {"bytes": T * idb + here * S * H * b + case["V"] * H * SIZES[case["grad"]], "flops": here * H * (S + 1)}
    if op == "block_norm":
        H = case["H"]
        return {"bytes": T * H * b * (3 + case["pre"]) + T * 4 * (case["post"] + case["pre"] + (case["gate"] == "token")),
                "flops": T * H * 10}
    if op == "block_norm_grad":
        H = case["H"]
        return {"bytes": T * H * b * (5 + case["pre"]) + T * 4 * (case["post"] + case["pre"]) + 12 * H,
                "flops": T * H * 24}
    E, k = case["E"], case["k"]
    if op == "route":
        return {"bytes": T * (E * b + 8 * k) + 4 * E, "flops": T * E * 8}
    whole = case["score"] == "softmax" and not case["renorm"]
    return {"bytes": T * (8 * k + (E if whole else k) * b + E * b), "flops": T * ((E if whole else k) * 8)}
