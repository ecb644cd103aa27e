"""Plain 64-bit implementations of the operators around the seam (CPU torch),
and how far a kernel's output may be from them.

Tolerances, derived from the arithmetic: a kernel computes in fp32 (unit
roundoff 2^-24) and rounds once to the output's type, so an element may be off
by half a unit in the last place of the type (``UNIT * |ref|``; for fp16 also
its subnormal step) plus ``n * 2^-24`` times the sum of the absolute values of
the terms it is made of, with n the longest chain of fp32 roundings.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
U32 = 2.0 ** -24
# the longest chain of fp32 roundings of one element of a row operator: a sum of
# squares over 16384 columns (32 per thread, then at most 5 + 32 partial sums),
# twice, with the products around them
CHAIN = 160


def check(got, ref, terms, n=CHAIN, what=""):
    """``got`` (any float type) against ``ref`` (64 bits) made of ``terms`` (sum of absolute values)."""
    g = got.detach().cpu().double()
    tol = UNIT[got.dtype] * ref.abs() * (1 + 2.0 ** -8) + TINY[got.dtype] + n * U32 * terms
    bad = (g - ref).abs() > tol
    bad |= torch.isnan(g) != torch.isnan(ref)
    assert not bool(bad.any()), (what, int(bad.sum()), float(((g - ref).abs() - tol).max()))


# ------------------------------------------------------------- embedding --
def embed(ids, table, scale, first, streams):
    out = torch.zeros(len(ids), streams, table.shape[1], dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i - first < table.shape[0]:
            out[t] = table[i - first].double() * scale
    return out


def embed_grad(ids, dout, V, scale, first=0, padding=None):
    """(gradient, sum of absolute terms, most terms of a row)."""
    H = dout.shape[-1]
    d = dout.double().reshape(len(ids), -1, H)
    g, a = torch.zeros(V, H, dtype=torch.float64), torch.zeros(V, H, dtype=torch.float64)
    n = [0] * V
    for t, i in enumerate(ids.tolist()):
        if 0 <= i - first < V and i != padding:
            g[i - first] += scale * d[t].sum(0)
            a[i - first] += abs(scale) * d[t].abs().sum(0)
            n[i - first] += d.shape[1]
    return g, a, max(n + [0])


# ------------------------------------------------------------ block norms --
def _gate(gate, mode):
    return 1.0 if gate is None else gate.double()[:, None] if mode == "token" else gate.double()


def block_norm(y, r, gamma_post, gate, mode, gamma_pre, scale, eps):
    """{name: value} with the sums of absolute terms under name + "_terms"."""
    out = {}
    r = torch.zeros_like(y, dtype=torch.float64) if r is None else r.double()
    if y is None:
        x, terms = r, r.abs()
    else:
        p = y.double()
        if gamma_post is not None:
            out["rstd_post"] = 1 / torch.sqrt(p.square().mean(1) + eps)
            p = p * out["rstd_post"][:, None] * gamma_post.double()
        g = _gate(gate, mode)
        x, terms = scale * r + g * p, (scale * r).abs() + (g * p).abs()
        out["r_out"], out["r_out_terms"] = x, terms
    if gamma_pre is not None:
        rho = 1 / torch.sqrt(x.square().mean(1) + eps)
        out["rstd_pre"] = rho
        out["norm"] = x * rho[:, None] * gamma_pre.double()
        out["norm_terms"] = terms * rho[:, None] * gamma_pre.double().abs()
        # how far an error of x moves rho, relative: sum |x| terms / sum x^2 >= 1
        out["rho_grow"] = (terms * x.abs()).mean(1) * rho.square() + 1
    return out


def block_norm_grad(dr_out, dnorm, y, r_out, gamma_post, gate, mode, gamma_pre, rstd_post, rstd_pre, scale):
    out = {}

    def put(name, value, terms):
        out[name], out[name + "_terms"] = value, terms

    x = r_out.double() if r_out is not None else None
    shape = (x if x is not None else y).shape
    G = torch.zeros(shape, dtype=torch.float64) if dr_out is None else dr_out.double()
    A = G.abs()
    if gamma_pre is not None:
        rho = rstd_pre.double()[:, None]
        u, dn, w = x * rho, dnorm.double(), gamma_pre.double()
        put("dgamma_pre", (dn * u).sum(0), (dn * u).abs().sum(0))
        c = w * dn
        G = G + rho * (c - u * (c * u).mean(1, keepdim=True))
        A = A + rho * (c.abs() + u.abs() * (c * u).abs().mean(1, keepdim=True))
    put("dr", scale * G, abs(scale) * A)
    if y is None:
        return out
    g, u, w, rho = _gate(gate, mode), y.double(), 1.0, None
    if gamma_post is not None:
        rho, w = rstd_post.double()[:, None], gamma_post.double()
        u = u * rho
    if mode != "none":
        axis = 1 if mode == "token" else 0
        put("dgate", (u * w * G).sum(axis), (u * w).abs().mul(A).sum(axis))
    dp, B = g * G, (g if isinstance(g, float) else g.abs()) * A
    if gamma_post is None:
        put("dy", dp, B)
        return out
    put("dgamma_post", (dp * u).sum(0), (B * u.abs()).sum(0))
    c, C = w * dp, w.abs() * B
    put("dy", rho * (c - u * (c * u).mean(1, keepdim=True)),
        rho * (C + u.abs() * (C * u.abs()).mean(1, keepdim=True)))
    return out


# ---------------------------------------------------------------- routing --
def scores(l, sigmoid):
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l).double()
    if sigmoid:
        return l, 1 / (1 + torch.exp(-l))
    out = torch.zeros_like(l)
    for t in range(l.shape[0]):
        m = l[t].max()
        if m == math.inf:
            e = (l[t] == m).double()
        elif m > -math.inf:
            e = torch.exp(l[t] - m)
        else:
            continue
        out[t] = e / e.sum()
    return l, out


def route(logits, bias, sigmoid, groups, top_groups, k, renorm, scale):
    """(indices, weights, counts, clear): ``clear`` marks the rows where every
    comparison that decides is wider than fp32's rounding, or a true tie."""
    l, p = scores(logits, sigmoid)
    T, E = l.shape
    per = E // groups
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double()
    idx = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=torch.float64)
    counts = torch.zeros(E, dtype=torch.int64)
    clear = torch.ones(T, dtype=torch.bool)

    def ranked(pairs, n):  # (value, index, what the value is made of): best first, ties to the lowest index
        order = sorted(pairs, key=lambda q: (-q[0], q[1]))
        near = any(0 <= x[0] - z[0] < 1e-6 and x[2] != z[2] for x, z in zip(order[:n], order[1:]))  # the first n decide
        return [q[1] for q in order], near

    for t in range(T):
        ok = [e for e in range(E) if l[t, e] > -math.inf]
        sel = {e: (float(p[t, e] + b[e]), e, (float(l[t, e]), float(b[e]))) for e in ok}
        if groups > 1:
            gs = []
            for g in range(groups):
                mine = sorted((sel[e] for e in ok if e // per == g), key=lambda q: -q[0])[:2]
                if mine:
                    gs.append((sum(q[0] for q in mine), g, tuple(q[2] for q in mine)))
            best, near = ranked(gs, top_groups)
            clear[t] &= not near
            sel = {e: v for e, v in sel.items() if e // per in best[:top_groups]}
        order, near = ranked(sel.values(), k)
        clear[t] &= not near
        for j, e in enumerate(order[:k]):
            idx[t, j] = e
            w[t, j] = p[t, e]
            counts[e] += 1
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return idx, scale * w, counts, clear


def route_grad(dweights, logits, indices, sigmoid, renorm, scale):
    """(gradient, sum of absolute terms)."""
    l, p = scores(logits, sigmoid)
    out, terms = torch.zeros_like(p), torch.zeros_like(p)
    for t in range(l.shape[0]):
        sel = [(j, int(e)) for j, e in enumerate(indices[t]) if 0 <= e < l.shape[1]]
        if not sel:
            continue
        e = torch.tensor([q[1] for q in sel])
        dw = dweights[t, [q[0] for q in sel]].double()
        s = p[t, e]
        if renorm:
            if s.sum() == 0:
                continue
            q = s / s.sum()
            ds, da = (dw - (q * dw).sum()) / s.sum(), (dw.abs() + (q * dw).abs().sum()) / s.sum()
        else:
            ds, da = dw, dw.abs()
        if sigmoid:
            out[t, e] += scale * ds * s * (1 - s)
            terms[t, e] += abs(scale) * da * s
        else:
            full, fa = torch.zeros_like(p[t]), torch.zeros_like(p[t])
            full[e], fa[e] = ds, da
            out[t] = scale * p[t] * (full - (full * p[t]).sum())
            terms[t] = abs(scale) * p[t] * (fa + (fa * p[t]).sum())
    return out, terms
