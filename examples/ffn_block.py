"""The operators inside a block, together with those around it, as a program uses them.

  python examples/ffn_block.py serve   one decode step of a feed-forward block between two seams: the seam's norm, what the
                                       requests' adapters add to the gated projections, the projections, the down projection
                                       and its adapters, the norm of the output, the next seam; captured in a graph
  python examples/ffn_block.py train   a small feed-forward model trained end to end: embedding, norm, gated projections,
                                       down projection, dropout and residual add, norm, and back

The down projection and the head are plain torch products; everything else is this library's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mhc_residual_seam_gb300 import binding as B  # noqa: E402


def workspace(n):
    ws = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    B.mhc_workspace_init(ws)
    return ws


# ------------------------------------------------------------------- serve --
class Block:
    """A feed-forward block of a four-stream model with adapters for `n` kinds of requests, for up to T tokens."""

    def __init__(self, T=8, H=1024, F=2048, n=4, rank=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = dict(device="cuda", dtype=torch.bfloat16)
        rand = lambda *s, std=1.0: (std * torch.randn(*s, device="cuda", generator=g)).bfloat16()  # noqa: E731
        self.T, self.H, self.F = T, H, F
        self.w, self.w_down = rand(2 * F, H, std=H ** -0.5), rand(H, F, std=F ** -0.5)
        self.up_a, self.up_b = rand(n, rank, H, std=H ** -0.5), rand(n, 2 * F, rank, std=rank ** -0.5)
        self.down_a, self.down_b = rand(n, rank, F, std=F ** -0.5), rand(n, H, rank, std=rank ** -0.5)
        self.scale = torch.full((n,), 0.5, device="cuda")
        self.gamma, self.gamma_y = torch.ones(H, **bf16), torch.ones(H, **bf16)
        self.fn = torch.randn(4 * H, 24, device="cuda", generator=g) * (4 * H) ** -0.5
        self.bias, self.alpha = torch.zeros(24, device="cuda"), torch.ones(3, device="cuda")
        self.packed = torch.empty(B.mhc_packed_fn_bytes(H) // 2, **bf16)
        B.mhc_pack_fn(self.fn, self.packed)
        # what a call works in: kept by the program, shared by nothing that runs at the same time
        self.ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
        self.lora_ws = workspace(B.mhc_lora_workspace_bytes(T, rank))
        self.seam = B.alloc_outputs(T, H, B.MHC_OUT_BF16, "cuda")
        self.add, self.h = torch.empty(T, 2 * F, **bf16), torch.empty(T, F, **bf16)
        self.y, self.Y, self.rstd = torch.empty(T, H, **bf16), torch.empty(T, H, **bf16), torch.empty(T, device="cuda")

    def step(self, R, norm, gates, index):
        """The block on the seam's `norm` [T, H] and the next seam on its output; returns that seam's outputs."""
        B.mhc_lora(norm, self.up_a, self.up_b, index, self.add, self.lora_ws, scale=self.scale)
        B.mhc_glu(norm, self.w, self.h, self.ws, add=self.add)
        torch.matmul(self.h, self.w_down.t(), out=self.y)
        B.mhc_lora(self.h, self.down_a, self.down_b, index, self.y, self.lora_ws, scale=self.scale, base=self.y)
        B.mhc_block_norm(self.y, None, self.gamma_y, None, None, self.Y, None, self.rstd, None)
        o = self.seam
        B.mhc_seam(R, self.Y, gates["post"], gates["comb"], gates["pre"], self.fn, self.packed, self.bias, self.alpha, self.gamma,
                   1e-6, B.MHC_OUT_BF16, o["residual_out"], o["norm"], None, None, o["pre_out"], o["post_out"], o["comb_out"],
                   o["workspace"])
        return o

    def outputs(self):
        """What a step writes, one after another."""
        seam = ("norm", "residual_out", "pre_out", "post_out", "comb_out")
        return {"add": self.add, "h": self.h, "y": self.y, "Y": self.Y, **{k: self.seam[k] for k in seam}}


def serve(T=8, H=1024, F=2048, n=4, seed=0):
    """A step of T requests, once as calls and once as a replayed graph."""
    b = Block(T, H, F, n, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    R = torch.randn(T, 4, H, device="cuda", generator=g).bfloat16()
    norm = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    index = torch.randint(-1, n, (T,), device="cuda", generator=g).int()  # -1: a request without an adapter
    gates = {"pre": torch.full((T, 4), 0.25, device="cuda"), "post": torch.ones(T, 4, device="cuda"),
             "comb": torch.full((T, 4, 4), 0.25, device="cuda")}
    b.step(R, norm, gates, index)
    outputs = b.outputs()
    eager = {k: v.clone() for k, v in outputs.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(R, norm, gates, index)  # torch's own products want a first call before a capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.step(R, norm, gates, index)
    torch.cuda.current_stream().wait_stream(side)
    for v in outputs.values():
        v.fill_(float("nan"))  # what a replay does not write is seen
    graph.replay()
    torch.cuda.synchronize()
    for ws in (b.ws, b.lora_ws, b.seam["workspace"]):
        B.mhc_check_status(ws)
    return {"block": b, "x": norm, "index": index, "eager": eager, "replayed": outputs}


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
        grad = torch.empty(*ctx.shape, device="cuda", dtype=dout.dtype)
        ws = torch.empty(B.mhc_embed_grad_workspace_bytes(len(ids), *ctx.shape), device="cuda", dtype=torch.uint8)
        B.mhc_embed_grad(ids, dout.contiguous(), grad, ws)
        return None, grad


class Norm(torch.autograd.Function):
    """r / rms(r) * gamma."""

    @staticmethod
    def forward(ctx, r, gamma):
        norm, rstd = torch.empty_like(r), torch.empty(len(r), device="cuda")
        B.mhc_block_norm(None, r, None, None, gamma, None, norm, None, rstd)
        ctx.save_for_backward(r, gamma, rstd)
        return norm

    @staticmethod
    def backward(ctx, dnorm):
        r, gamma, rstd = ctx.saved_tensors
        T, H = r.shape
        dr, dgamma = torch.empty_like(r), torch.empty(H, device="cuda")
        ws = torch.empty(max(16, B.mhc_block_norm_grad_workspace_bytes(T, H)), device="cuda", dtype=torch.uint8)
        B.mhc_block_norm_grad(None, dnorm.contiguous(), None, r, None, None, gamma, None, rstd, None, dr, None, None, dgamma, ws)
        return dr, dgamma.to(gamma.dtype)


class GLU(torch.autograd.Function):
    """act(x Wg^T) * (x Wu^T)."""

    @staticmethod
    def forward(ctx, x, w, act):
        (T, H), F = x.shape, w.shape[0] // 2
        h, gu = x.new_empty(T, F), x.new_empty(T, 2 * F)
        ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
        B.mhc_glu(x, w, h, ws, gu=gu, act=act)
        ctx.save_for_backward(x, w, gu, ws)
        ctx.act = act
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w, gu, ws = ctx.saved_tensors
        dgu, dx, dw = torch.empty_like(gu), torch.empty_like(x), torch.empty_like(w)
        B.mhc_glu_grad(dh.contiguous(), gu, x, w, dgu, dx, dw, ws, act=ctx.act)
        return dx, dw, None


class DropoutAdd(torch.autograd.Function):
    """r + dropout(y); the gradient by y is the same call on the gradient of the sum."""

    @staticmethod
    def forward(ctx, y, r, seed, p):
        out = torch.empty_like(y)
        B.mhc_dropout(y, out, seed, r=r, p=p)
        ctx.save_for_backward(seed)
        ctx.p = p
        return out

    @staticmethod
    def backward(ctx, dout):
        (seed,) = ctx.saved_tensors
        dout = dout.contiguous()
        dy = torch.empty_like(dout)
        B.mhc_dropout(dout, dy, seed, p=ctx.p)
        return dy, dout, None, None


def model(p, ids, seed, drop=0.1):
    """Logits over the vocabulary of a one-block model."""
    r = Embed.apply(ids, p["table"])
    y = GLU.apply(Norm.apply(r, p["gamma_in"]), p["w"], B.MHC_ACT_SILU) @ p["w_down"].t()
    return (Norm.apply(DropoutAdd.apply(y, r, seed, drop), p["gamma_out"]) @ p["head"]).float()


def parameters(V=64, H=128, F=256, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, std: (std * torch.randn(*s, device="cuda", generator=g)).bfloat16().requires_grad_()  # noqa: E731
    one = lambda: torch.ones(H, device="cuda", dtype=torch.bfloat16, requires_grad=True)  # noqa: E731
    return {"table": rand(V, H, std=1.0), "gamma_in": one(), "w": rand(2 * F, H, std=H ** -0.5), "w_down": rand(H, F, std=F ** -0.5),
            "gamma_out": one(), "head": rand(H, V, std=H ** -0.5)}


def train(steps=60, T=512, V=64, seed=0):
    """Learns a fixed permutation of the tokens; returns the losses."""
    p = parameters(V=V, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    target = torch.randperm(V, device="cuda", generator=g)
    optimizer = torch.optim.Adam(list(p.values()), lr=1e-2)
    losses = []
    for step in range(steps):
        ids = torch.randint(0, V, (T,), device="cuda", generator=g)
        drop_seed = torch.tensor([seed, step], device="cuda")  # the key, and the call's number
        loss = torch.nn.functional.cross_entropy(model(p, ids, drop_seed), target[ids])
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    what = sys.argv[1] if len(sys.argv) > 1 else "train"
    if what == "serve":
        out = serve()
        print("adapters of the requests:", out["index"].tolist())
        print("the replay gives the same:", all(torch.equal(v, out["replayed"][k]) for k, v in out["eager"].items()))
    elif what == "train":
        losses = train()
        print("loss", " ".join("%.3f" % x for x in losses[::10] + losses[-1:]))
    else:
        sys.exit("ffn_block.py serve | train")
