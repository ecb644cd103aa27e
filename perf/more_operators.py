"""Cases for the operators inside a block: the gated projections of its
feed-forward part and their gradient, low-rank adapters of many requests beside a
shared projection, and dropout before a residual add.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, where ``own`` is set, through the
framework's entry points.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
WORKSPACE_BYTES = 128 << 20  # one zeroed workspace, large enough for every case here
MOST_PRODUCT = 8192 * 5120 * 10240  # T * H * F of the largest gated case


def listed():
    return [
        # a decode step of four sequences: the weights are read once for four tokens
        {"name": "glu_decode", "op": "glu", "T": 4, "H": 5120, "F": 10240, "dtype": "bf16", "act": "silu", "add": False,
         "keep": False},
        # a decode step of 64 sequences whose requests have adapters on the gated projections
        {"name": "glu_decode_adapters", "op": "glu", "T": 64, "H": 5120, "F": 10240, "dtype": "bf16", "act": "silu",
         "add": True, "keep": False},
        # a prompt of odd length in a smaller model, 16-bit floats, another activation
        {"name": "glu_prompt", "op": "glu", "T": 1003, "H": 2048, "F": 5000, "dtype": "fp16", "act": "gelu_tanh",
         "add": False, "keep": False},
        # a training step at the seam's width; the pre-activations are kept for the gradient
        {"name": "glu_train", "op": "glu", "T": 8192, "H": 5120, "F": 10240, "dtype": "bf16", "act": "silu", "add": False,
         "keep": True},
        # a small model's training step, odd sizes
        {"name": "glu_grad_small", "op": "glu_grad", "T": 1003, "H": 512, "F": 1368, "dtype": "bf16", "act": "gelu"},
        # the training step at the seam's width, backward
        {"name": "glu_grad_large", "op": "glu_grad", "T": 8192, "H": 5120, "F": 10240, "dtype": "bf16", "act": "silu"},
        # a decode step of 64 requests over 32 adapters, beside a square projection
        {"name": "lora_decode", "op": "lora", "T": 64, "H": 5120, "N": 5120, "R": 16, "n": 32, "dtype": "bf16",
         "runs": 64, "base": True, "scaled": True},
        # a batch of prompts of a smaller model: what their adapters add to the gated projections, on its own
        {"name": "lora_prompts", "op": "lora", "T": 1003, "H": 2048, "N": 10000, "R": 8, "n": 5, "dtype": "fp16", "runs": 9,
         "base": False, "scaled": False},
        # a large prefill batch: 24 prompts over 8 adapters of rank 64
        {"name": "lora_prefill", "op": "lora", "T": 8192, "H": 5120, "N": 5120, "R": 64, "n": 8, "dtype": "bf16",
         "runs": 24, "base": True, "scaled": True},
        # a small model trained in 32 bits, odd token count
        {"name": "dropout_small", "op": "dropout", "T": 1003, "H": 512, "dtype": "fp32", "residual": True, "p": 0.1},
        # dropout and the residual add of a training step at the seam's largest workload
        {"name": "dropout_train", "op": "dropout", "T": 16384, "H": 5120, "dtype": "bf16", "residual": True, "p": 0.1},
        # its gradient: the same numbers on the gradient that comes back
        {"name": "dropout_grad", "op": "dropout", "T": 16384, "H": 5120, "dtype": "bf16", "residual": False, "p": 0.25},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_grad", "lora", "lora", "dropout"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("glu", "glu_grad"):
        H, F = 8 * _log_int(rng, 8, 640), 8 * _log_int(rng, 8, 1280)
        T = _log_int(rng, 1, min(16384, MOST_PRODUCT // (H * F)))
        c = {"op": op, "T": T, "H": H, "F": F, "dtype": dtype, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"])}
        if op == "glu":
            c["add"], c["keep"] = rng.random() < 0.3, rng.random() < 0.4
        return c
    if op == "lora":
        H, N, T = 8 * _log_int(rng, 8, 640), 8 * _log_int(rng, 8, 1280), _log_int(rng, 1, 8192)
        R = rng.choice([8, 16, 16, 24, 32, 64, 128])
        n = _log_int(rng, 1, min(64, 4096 // R))
        while T * N > 8192 * 5120:
            T //= 2
        return {"op": op, "T": T, "H": H, "N": N, "R": R, "n": n, "dtype": dtype,
                # how many requests the tokens belong to: one each in a decode step, fewer in a prefill
                "runs": T if T <= 256 and rng.random() < 0.6 else _log_int(rng, 1, min(T, 64)),
                "base": rng.random() < 0.7, "scaled": rng.random() < 0.7}
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    H = 8 * _log_int(rng, 8, 1024)
    return {"op": op, "T": _log_int(rng, 1, min(65536, 16384 * 5120 * 2 // (H * SIZES[dtype]))), "H": H, "dtype": dtype,
            "residual": rng.random() < 0.5, "p": rng.choice([0.0, 0.05, 0.1, 0.2, 0.5])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, T, H, op = DTYPES[case["dtype"]], case["T"], case["H"], case["op"]

    def normal(*shape, std=1.0):
        return torch.empty(*shape, device="cuda", dtype=torch.float32).normal_(0, std, generator=g).to(dt)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case, "ws": torch.zeros(WORKSPACE_BYTES, device="cuda", dtype=torch.uint8)}
    if op in ("glu", "glu_grad"):
        F = case["F"]
        s["x"], s["w"] = normal(T, H), normal(2 * F, H, std=H ** -0.5)  # a norm's output; the gate's rows, then the other's
        if op == "glu":
            s["add"] = normal(T, 2 * F, std=0.3) if case["add"] else None
            s["h"], s["gu"] = empty(T, F), empty(T, 2 * F) if case["keep"] else None
        else:  # the pre-activations that the forward pass kept, and the gradient that comes back
            s["gu"] = torch.matmul(s["x"].float(), s["w"].float().t()).to(dt)
            s["dh"] = normal(T, F)
            s["dgu"], s["dx"], s["dw"] = empty(T, 2 * F), empty(T, H), empty(2 * F, H)
    elif op == "lora":
        N, R, n = case["N"], case["R"], case["n"]
        s["x"], s["a"], s["b"] = normal(T, H), normal(n, R, H, std=H ** -0.5), normal(n, N, R, std=R ** -0.5)
        # runs of tokens of one request, of random lengths; about one request in eight has no adapter
        cuts = torch.rand(case["runs"] - 1, device="cuda", generator=g).mul_(T).long().sort().values
        of = torch.randint(0, n, (case["runs"],), device="cuda", generator=g)
        of[1:][torch.rand(case["runs"] - 1, device="cuda", generator=g) < 0.125] = -1
        s["index"] = of[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)].int()
        s["scale"] = 0.5 + torch.rand(n, device="cuda", generator=g) if case["scaled"] else None
        s["base"] = normal(T, N) if case["base"] else None  # what the shared projection gave
        s["out"] = empty(T, N)
    else:
        s["y"], s["r"] = normal(T, H), normal(T, H, std=2.0) if case["residual"] else None
        s["seed"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=g)  # the key, and the call's number
        s["out"] = empty(T, H)
    return s


# ------------------------------------------------------------- plain forms --
GELU_A, GELU_B = 2 * math.sqrt(2 / math.pi), 0.044715


def _act(g, act):
    """The activation and its derivative."""
    if act == "relu":
        up = (g > 0).to(g.dtype)
        return g * up, up
    if act == "gelu":
        phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    q, dq = (g, 1.0) if act == "silu" else (GELU_A * (g + GELU_B * g * g * g), GELU_A * (1 + 3 * GELU_B * g * g))
    v = 1 / (1 + torch.exp(-q))
    return g * v, v + g * v * (1 - v) * dq


def _glu(s):
    c, F, dt = s["case"], s["case"]["F"], s["x"].dtype
    gu = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["add"] is not None:
        gu = gu + s["add"].float()
    out = {"h": (_act(gu[:, :F], c["act"])[0] * gu[:, F:]).to(dt)}
    if c["keep"]:
        out["gu"] = gu.to(dt)
    return out


def _glu_grad(s):
    c, F, dt = s["case"], s["case"]["F"], s["x"].dtype
    g, u, dh = s["gu"][:, :F].float(), s["gu"][:, F:].float(), s["dh"].float()
    a, da = _act(g, c["act"])
    dgu = torch.cat([dh * u * da, dh * a], 1)
    return {"dgu": dgu.to(dt), "dx": torch.matmul(dgu, s["w"].float()).to(dt),
            "dw": torch.matmul(dgu.t(), s["x"].float()).to(dt)}


def _lora(s):
    c = s["case"]
    T, R, n = c["T"], c["R"], c["n"]
    v = torch.matmul(s["x"].float(), s["a"].float().reshape(n * R, -1).t()).view(T, n, R)
    mine = s["index"][:, None] == torch.arange(n, device="cuda")
    v = torch.where(mine[:, :, None], v, 0.0)
    if s["scale"] is not None:
        v = v * s["scale"][:, None]
    y = torch.matmul(v.view(T, n * R), s["b"].float().transpose(1, 2).reshape(n * R, -1))
    if s["base"] is not None:
        y = s["base"].float() + y
    return {"out": y.to(s["x"].dtype)}


PHILOX_M, PHILOX_W = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85)  # multipliers and key steps of Philox 4x32
LOW = 0xFFFFFFFF


def _philox(i, offset, key):
    """Philox 4x32 with ten rounds of the counters (i, offset) under a 64-bit key: [.., 4] words."""
    a, b, c, d = i & LOW, i >> 32, (offset & LOW).expand_as(i), (offset >> 32).expand_as(i)
    k0, k1 = key & LOW, key >> 32
    for r in range(10):
        # the products wrap in 64 signed bits; their upper words are masked after the shift
        p, q = a * PHILOX_M[0], c * PHILOX_M[1]
        a, b, c, d = ((q >> 32) & LOW) ^ b ^ ((k0 + r * PHILOX_W[0]) & LOW), q & LOW, \
            ((p >> 32) & LOW) ^ d ^ ((k1 + r * PHILOX_W[1]) & LOW), p & LOW
    return torch.stack([a, b, c, d], -1)


def _dropout(s):
    c, y = s["case"], s["y"].float()
    w = _philox(torch.arange(y.numel() // 4, device="cuda"), s["seed"][1], s["seed"][0]).view(y.shape)
    out = torch.where(w >= int(c["p"] * 2.0 ** 32 + 0.5), y * (1 / (1 - c["p"])), 0.0)
    if s["r"] is not None:
        out = out + s["r"].float()
    return {"out": out.to(s["y"].dtype)}


PLAIN = {"glu": _glu, "glu_grad": _glu_grad, "lora": _lora, "dropout": _dropout}


# ------------------------------------------------------ the framework's own --
def _own(s):
    from mhc_residual_seam_gb300 import binding as B

    c = s["case"]
    op = c["op"]
    if op in ("glu", "glu_grad"):
        act = {"silu": B.MHC_ACT_SILU, "gelu": B.MHC_ACT_GELU, "gelu_tanh": B.MHC_ACT_GELU_TANH, "relu": B.MHC_ACT_RELU}[c["act"]]
        if op == "glu":
            B.mhc_glu(s["x"], s["w"], s["h"], s["ws"], add=s["add"], gu=s["gu"], act=act)
            return {n: s[n] for n in ("h", "gu") if s[n] is not None}
        B.mhc_glu_grad(s["dh"], s["gu"], s["x"], s["w"], s["dgu"], s["dx"], s["dw"], s["ws"], act=act)
        return {n: s[n] for n in ("dgu", "dx", "dw")}
    if op == "lora":
        B.mhc_lora(s["x"], s["a"], s["b"], s["index"], s["out"], s["ws"], scale=s["scale"], base=s["base"])
        return {"out": s["out"]}
    B.mhc_dropout(s["y"], s["out"], s["seed"], r=s["r"], p=c["p"])
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op in ("glu", "glu_grad"):
        f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
             "gelu_tanh": lambda g: torch.nn.functional.gelu(g, approximate="tanh")}[case["act"]]
        if op == "glu":
            gu = torch.einsum("th,fh->tf", s["x"], s["w"])
            if case["add"]:
                gu += s["add"]
            g, u = gu.chunk(2, 1)
            return {"h": f(g) * u, **({"gu": gu} if case["keep"] else {})}
        gu = s["gu"].requires_grad_()
        g, u = gu.chunk(2, 1)
        (dgu,) = torch.autograd.grad(f(g) * u, gu, s["dh"])
        return {"dgu": dgu, "dx": torch.einsum("tf,fh->th", dgu, s["w"]), "dw": torch.einsum("tf,th->fh", dgu, s["x"])}
    if op == "lora":
        out = s["base"].clone() if case["base"] else torch.zeros(case["T"], case["N"], device="cuda", dtype=torch.float64)
        for e in range(case["n"]):
            t = torch.nonzero(s["index"] == e)[:, 0]
            delta = torch.einsum("tr,nr->tn", torch.einsum("th,rh->tr", s["x"][t], s["a"][e]), s["b"][e])
            out[t] += delta * (s["scale"][e] if case["scaled"] else 1)
        return {"out": out}
    return {"out": _exact_dropout(case, s)}


def _exact_dropout(case, s):
    """Philox again, its 32 x 32-bit products from 16-bit halves."""
    key, offset = (int(v) for v in s["seed"].tolist())
    n = s["y"].numel() // 4
    i = torch.arange(n, device="cuda")
    x = [i % (1 << 32), i // (1 << 32), torch.full_like(i, offset % (1 << 32)), torch.full_like(i, offset // (1 << 32))]
    k = [key % (1 << 32), key // (1 << 32)]

    def times(v, m):
        lo, hi = (v % 65536) * m, (v // 65536) * m  # below 2^48 each
        mid = hi + lo // 65536
        return mid // 65536, (mid % 65536) * 65536 + lo % 65536

    for _ in range(10):
        h0, l0 = times(x[0], 0xD2511F53)
        h1, l1 = times(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k[0], l1, h0 ^ x[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) % (1 << 32), (k[1] + 0xBB67AE85) % (1 << 32)]
    drop = torch.stack([w.double() for w in x], 1).view(s["y"].shape) < math.floor(case["p"] * 2 ** 32 + 0.5)
    out = (s["y"] / (1 - case["p"])).masked_fill(drop, 0)
    return out + s["r"] if case["residual"] else out


# ------------------------------------------------------------------- work --
def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    b = SIZES[case["dtype"]]
    if op == "glu":
        F = case["F"]
        return {"bytes": b * (T * H + 2 * F * H + T * F * (1 + 2 * case["add"] + 2 * case["keep"])), "flops": 4 * T * H * F}
    if op == "glu_grad":
        F = case["F"]
        return {"bytes": b * (T * F * 5 + 2 * T * H + 4 * F * H), "flops": 8 * T * H * F}
    if op == "lora":
        N, R = case["N"], case["R"]
        used = min(case["n"], case["runs"])
        return {"bytes": b * (T * H + used * R * (H + N) + T * N * (1 + case["base"])) + 4 * T,
                "flops": 2 * T * R * (H + N)}
    return {"bytes": T * H * b * (2 + case["residual"]), "flops": T * H * 2}
