"""Binary64 forms of the query/key norm with RoPE and of window attention, written from the
definitions, with error bounds for the kernels' arithmetic.

Rounding to nearest is off by at most half a unit: 2^-8 of the value for bf16, 2^-24 for
binary32.  The bounds count:
  logits   binary32 dot products of d terms: E = (d + 4) 2^-24 max_j sum_c |q_c k_jc| / sqrt d,
           so p_ij and the row sum are off by at most a factor 1 + 2 E + (n + 64) 2^-24 (n
           visible keys; 64 covers the exponential's few units and the joins);
  P, dS    rounded to bf16 once in the bf16 kernels (2^-8);
  outputs  rounded once to the tensor's type.
"""
from __future__ import annotations

import math

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8


def half_step(dtype):
    return U16 if dtype == torch.bfloat16 else U32


def visible(p, q_first, k_len):
    """bool [B, Nq, Nk] from the definition; q_first, k_len: lists of B."""
    i, j = torch.arange(p.Nq)[:, None], torch.arange(p.Nk)[None, :]
    out = []
    for f0, n in zip(q_first, k_len):
        fq, fk = (f0 + i) // p.frame, j // p.frame
        v = (j < n) & ((fk < p.sinks) | (torch.ones_like(fk, dtype=torch.bool) if p.left < 0 else fk >= fq - p.left))
        if p.right >= 0:
            v = v & (fk <= fq + p.right)
        out.append(v.expand(p.Nq, p.Nk))
    return torch.stack(out)


def attention(Q, K, V, vis, G=None):
    """Values and bounds per output: {"O": (value, bound), "lse": ..., "dQ": ..., ...}."""
    dt = Q.dtype
    low = 0.0 if dt == torch.float32 else U16              # rounding of P and dS
    out_u = half_step(dt)
    q, k, v = Q.double(), K.double(), V.double()
    B, H, Nq, d = q.shape
    g = H // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    vis = vis.to(q.device)[:, None]
    sc = 1.0 / math.sqrt(d)
    s = (q @ k.mT * sc).masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    P = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse))
    O = P @ v
    n = vis.sum(-1, keepdim=True).double()
    E = (d + 4) * U32 * sc * ((q.abs() @ k.abs().mT) * vis).amax(-1, keepdim=True)
    rel = 2 * E + (n + 64) * U32
    A = P @ v.abs()
    bO = out_u * O.abs() + (low + 2 * rel) * 1.02 * A
    out = {"O": (O, bO), "lse": (lse[..., 0], (2 * rel + lse.abs().nan_to_num(0, 0, 0) * 4 * U32 + 4 * U32)[..., 0])}
    if G is None:
        return out
    go = G.double()
    D = (go * O).sum(-1, keepdim=True)
    bD = (go.abs() * (bO + 2 * d * U32 * O.abs())).sum(-1, keepdim=True)
    dP = go @ v.mT
    bdP = (d + 4) * U32 * (go.abs() @ v.abs().mT)
    dS = P * (dP - D)
    # P from the saved lse: its error adds E + the rounding of lse (2^-24 |lse|) once more
    u = low + 3 * rel + 2 * U32 * lse.abs().nan_to_num(0, 0, 0)
    bS = 1.02 * (u * dS.abs() + P * (1 + low) * (bD + bdP))
    nq = Nq * g
    dQ = dS @ k * sc
    out["dQ"] = (dQ, out_u * dQ.abs() + 1.02 * sc * ((bS + (n + 64) * U32 * dS.abs()) @ k.abs()))

    def per_key(x):
        return x.view(B, H // g, g, x.shape[2], d).sum(2)

    dK, dV = per_key(dS.mT @ q) * sc, per_key(P.mT @ go)
    out["dK"] = (dK, out_u * dK.abs() + 1.02 * sc * per_key((bS + (nq + 64) * U32 * dS.abs()).mT @ q.abs()))
    out["dV"] = (dV, out_u * dV.abs() + 1.02 * per_key(((u + (nq + 64) * U32) * P).mT @ go.abs()))
    return out


def check(name, got, value, bound):
    got = got.double()
    assert torch.equal(torch.isinf(got), torch.isinf(value)), name
    assert torch.isfinite(got[~torch.isinf(value)]).all(), name
    fine = torch.isfinite(value)
    off = (got - value).abs()[fine] - bound[fine]
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{name}: {worst:.3e} beyond the bound ({(got - value).abs()[fine].max().item():.3e} off)"


def angles(p, first):
    """float64 cos, sin [B, 1, N, d/2]."""
    pos = torch.tensor(first, dtype=torch.int64)[:, None] + torch.arange(p.N)
    t, rem = pos // (p.Hg * p.Wg), pos % (p.Hg * p.Wg)
    a = [ax[..., None].double() * p.base ** (-2.0 * torch.arange(w // 2, dtype=torch.float64) / max(w, 1))
         for ax, w in ((t, p.d_t), (rem // p.Wg, p.d_h), (rem % p.Wg, p.d_w))]
    a = torch.cat(a, -1)[:, None]
    return torch.cos(a).cuda(), torch.sin(a).cuda()


def rotate(x, cs, sn):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * cs - x1 * sn, x0 * sn + x1 * cs), -1).flatten(-2)


def norm(X, w, cs, sn, eps, G=None):
    """{"Y": (value, bound), "dX": ..., "dw": ...}.  Binary32 steps: the mean of squares is
    off by (d / 8 + 6) 2^-24 relative and r by half that and a step, a rotated value by 8 steps
    of its pair's magnitude (cos and sin within 4 steps), one rounding to the type."""
    out_u = half_step(X.dtype)
    x = X.double()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    u = (d // 8 + 24) * U32

    def pairs(v):
        a = v.abs()
        return (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1)

    Y = rotate(xh * w, cs, sn)
    out = {"Y": (Y, out_u * Y.abs() + 1.02 * u * pairs(xh * w))}
    if G is None:
        return out
    g = rotate(G.double(), cs, -sn)
    bg = u * pairs(G.double())
    gw = g * w
    c = (gw * xh).mean(-1, keepdim=True)
    bc = ((bg * w.abs() + 2 * u * gw.abs()) * xh.abs()).mean(-1, keepdim=True)
    dX = r * (gw - xh * c)
    out["dX"] = (dX, out_u * dX.abs() + 1.02 * r * (bg * w.abs() + 2 * u * gw.abs() + xh.abs() * (bc + 4 * u * c.abs())))
    rows = x.numel() // d
    dw = (g * xh).sum((0, 1, 2))
    # sums: at most 96 terms in a row, then at most 2^11 places, 32 rows and 600 blocks a column
    out["dw"] = (dw, 1.02 * ((bg + 2 * u * g.abs()) * xh.abs() + min(rows, 3000) * U32 * (g * xh).abs()).sum((0, 1, 2)))
    return out
