"""The operators around the seam, together, as a program uses them.

  python examples/moe_block.py serve   one decode step of a four-stream block: embedding rows into the streams, the
                                       first block's seam, routing on its norm, the experts, the norm and gate of
                                       their output, the next seam
  python examples/moe_block.py train   a small one-stream mixture-of-experts model trained end to end: embedding,
                                       norm, routing, experts, norm + gate + residual + norm, and back

The products (router, experts, head) are plain torch; everything else is this library's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mhc_residual_seam_gb300 import binding as B  # noqa: E402


def experts(x, indices, weights, w_in, w_out):
    """sum_j weights[t, j] * relu(x[t] @ w_in[e]) @ w_out[e] over the chosen experts e."""
    y = torch.zeros_like(x)
    for e in range(w_in.shape[0]):
        t, j = torch.nonzero(indices == e, as_tuple=True)
        y = y.index_add(0, t, (torch.relu(x[t] @ w_in[e]) @ w_out[e] * weights[t, j, None].to(x.dtype)).to(x.dtype))
    return y


# ------------------------------------------------------------------- serve --
def serve(T=8, V=1000, H=1024, E=16, k=4, seed=0):
    """One block of a four-stream model; returns the next block's input and what the routing chose."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf16 = dict(device="cuda", dtype=torch.bfloat16)
    rand = lambda *s, std=1.0: std * torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    table, gamma, gamma_y = rand(V, H, std=0.02).bfloat16(), torch.ones(H, **bf16), torch.ones(H, **bf16)
    fn, bias, alpha = rand(4 * H, 24, std=(4 * H) ** -0.5), torch.zeros(24, device="cuda"), torch.ones(3, device="cuda")
    w_route, balance = rand(H, E, std=H ** -0.5), torch.zeros(E, device="cuda")
    w_in, w_out = rand(E, H, 64, std=H ** -0.5).bfloat16(), rand(E, 64, H, std=0.125).bfloat16()
    packed = torch.empty(B.mhc_packed_fn_bytes(H) // 2, **bf16)
    B.mhc_pack_fn(fn, packed)

    # the residual's four streams start as the token's embedding
    ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    R = torch.empty(T, 4, H, **bf16)
    B.mhc_embed(ids, table, R, scale=H ** 0.5)

    # the first block's seam reads them: layer input, and the gates of the next seam
    first = B.alloc_outputs(T, H, B.MHC_OUT_BF16, "cuda")
    pre = torch.full((T, 4), 0.25, device="cuda")
    B.mhc_seam(R, None, None, None, pre, fn, packed, bias, alpha, gamma, 1e-6, B.MHC_OUT_BF16, None, first["norm"], None,
               None, first["pre_out"], first["post_out"], first["comb_out"], first["workspace"])

    # the layer: route on the norm, run the experts
    logits = first["norm"].float() @ w_route
    indices, weights = torch.empty(T, k, device="cuda", dtype=torch.int32), torch.empty(T, k, device="cuda")
    counts = torch.empty(E, device="cuda", dtype=torch.int32)
    ws = torch.empty(B.mhc_route_workspace_bytes(E), device="cuda", dtype=torch.uint8)
    B.mhc_workspace_init(ws)
    B.mhc_route(logits, balance, indices, weights, counts, ws, groups=4, top_groups=2, scale=2.5)
    y = experts(first["norm"], indices, weights, w_in, w_out)

    # the norm after the block: Y = y / rms(y) * gamma_y (the seam adds it, with the post gates, to the streams)
    Y, rstd = torch.empty(T, H, **bf16), torch.empty(T, device="cuda")
    B.mhc_block_norm(y, None, gamma_y, None, None, Y, None, rstd, None)
    second = B.alloc_outputs(T, H, B.MHC_OUT_BF16, "cuda")
    B.mhc_seam(R, Y, first["post_out"], first["comb_out"], first["pre_out"], fn, packed, bias, alpha, gamma, 1e-6,
               B.MHC_OUT_BF16, second["residual_out"], second["norm"], None, None, second["pre_out"], second["post_out"],
               second["comb_out"], second["workspace"])
    return {"norm": second["norm"], "residual": second["residual_out"], "indices": indices, "weights": weights,
            "counts": counts, "Y": Y, "y": y}


# ------------------------------------------------------------------- train --
class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table):
        out = torch.empty(len(ids), table.shape[1], device="cuda", dtype=table.dtype)
        B.mhc_embed(ids, table, out)
        ctx.save_for_backward(ids)
        ctx.shape = table.shape
        return out

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        V, H = ctx.shape
        grad = torch.empty(V, H, device="cuda", dtype=dout.dtype)
        ws = torch.empty(B.mhc_embed_grad_workspace_bytes(len(ids), V, H), device="cuda", dtype=torch.uint8)
        B.mhc_embed_grad(ids, dout.contiguous(), grad, ws)
        return None, grad


class BlockNorm(torch.autograd.Function):
    """(r', norm) of a block's output y and the residual r, with a channel gate; y None: the first norm."""

    @staticmethod
    def forward(ctx, y, r, gamma_post, gate, gamma_pre):
        T, H = r.shape
        norm = torch.empty_like(r)
        x = r if y is None else torch.empty_like(r)
        rp = None if gamma_post is None else torch.empty(T, device="cuda")
        rq = torch.empty(T, device="cuda")
        ctx.mode = B.MHC_GATE_NONE if gate is None else B.MHC_GATE_CHANNEL
        B.mhc_block_norm(y, r, gamma_post, gate, gamma_pre, None if y is None else x, norm, rp, rq, gate_mode=ctx.mode)
        ctx.save_for_backward(y, x, gamma_post, gate, gamma_pre, rp, rq)
        ctx.set_materialize_grads(False)
        return (norm, None) if y is None else (norm, x)

    @staticmethod
    def backward(ctx, dnorm, dx):
        y, x, gamma_post, gate, gamma_pre, rp, rq = ctx.saved_tensors
        T, H = x.shape
        dr, dy = torch.empty_like(x), None if y is None else torch.empty_like(x)
        f = lambda w: None if w is None else torch.empty(H, device="cuda")  # noqa: E731
        dp, dg, dq = f(gamma_post), f(gate), f(gamma_pre)
        ws = torch.empty(B.mhc_block_norm_grad_workspace_bytes(T, H), device="cuda", dtype=torch.uint8)
        B.mhc_block_norm_grad(None if dx is None else dx.contiguous(), dnorm.contiguous(), y, x, gamma_post, gate, gamma_pre,
                              rp, rq, dy, dr, dp, dg, dq, ws, gate_mode=ctx.mode)
        return dy, dr, dp, dg, dq


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        T, E = logits.shape
        indices, weights = torch.empty(T, k, device="cuda", dtype=torch.int32), torch.empty(T, k, device="cuda")
        B.mhc_route(logits, None, indices, weights, score=B.MHC_SCORE_SOFTMAX)
        ctx.save_for_backward(logits, indices)
        ctx.mark_non_differentiable(indices)
        return weights, indices

    @staticmethod
    def backward(ctx, dweights, _):
        logits, indices = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        B.mhc_route_grad(dweights.contiguous(), logits, indices, dlogits, score=B.MHC_SCORE_SOFTMAX)
        return dlogits, None


def model(p, ids, k=2):
    """Logits over the vocabulary of a one-block model."""
    r = Embed.apply(ids, p["table"])
    n, _ = BlockNorm.apply(None, r, None, None, p["gamma_in"])
    weights, indices = Route.apply(n @ p["w_route"], k)
    y = experts(n, indices, weights, p["w_in"], p["w_out"])
    n, _ = BlockNorm.apply(y, r, p["gamma_post"], p["gate"], p["gamma_pre"])
    return n @ p["head"]


def parameters(V=64, H=128, E=8, F=64, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, std: (std * torch.randn(*s, device="cuda", generator=g)).requires_grad_()  # noqa: E731
    one = lambda: torch.ones(H, device="cuda", requires_grad=True)  # noqa: E731
    return {"table": rand(V, H, std=1.0), "gamma_in": one(), "w_route": rand(H, E, std=H ** -0.5),
            "w_in": rand(E, H, F, std=H ** -0.5), "w_out": rand(E, F, H, std=F ** -0.5), "gamma_post": one(),
            "gate": one(), "gamma_pre": one(), "head": rand(H, V, std=H ** -0.5)}


def train(steps=60, T=512, V=64, seed=0):
    """Learns a fixed permutation of the tokens; returns the losses."""
    p = parameters(V=V, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    target = torch.randperm(V, device="cuda", generator=g)
    optimizer = torch.optim.Adam(list(p.values()), lr=1e-2)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, V, (T,), device="cuda", generator=g)
        loss = torch.nn.functional.cross_entropy(model(p, ids), target[ids])
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    what = sys.argv[1] if len(sys.argv) > 1 else "train"
    if what == "serve":
        out = serve()
        print("experts of token 0:", out["indices"][0].tolist(), "weights:", [round(w, 3) for w in out["weights"][0].tolist()])
        print("tokens per expert:", out["counts"].tolist())
        print("next block's input:", tuple(out["norm"].shape), "rms", round(float(out["norm"].float().square().mean().sqrt()), 3))
    elif what == "train":
        losses = train()
        print("loss", " ".join("%.3f" % x for x in losses[::10] + losses[-1:]))
    else:
        sys.exit("moe_block.py serve | train")
