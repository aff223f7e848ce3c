"""Query/key norm with 3D RoPE, and windowed attention with sinks: the measured cases.

Two operators of a video diffusion transformer's attention layer, each forward and with its
gradients:

* ``norm``: per-head RMS norm of queries and keys, a weight per channel, and 3D RoPE in the
  same pass (the step before attention);
* ``window``: softmax attention of every query over a sliding window of frames (or tokens)
  and a few first frames that stay visible, over whole layers, over a cache for the newest
  frame or token, and in training.

``run`` computes them in elementary torch operations (``own`` false) or by the library's
entry points (``own`` true).
"""
from __future__ import annotations

import functools
import math

import torch

own = False


# ---------------------------------------------------------------------------------- cases
def _norm(name, B, H, Hkv, N, split, Hg, Wg, first, dtype, ragged=False, train=False):
    case = {"op": "norm", "B": B, "H": H, "Hkv": Hkv, "N": N, "d_t": split[0], "d_h": split[1], "d_w": split[2],
            "Hg": Hg, "Wg": Wg, "first": first, "dtype": dtype, "ragged": ragged, "train": train}
    return dict(case, name=name) if name else case


def _window(name, B, H, Hkv, Nq, Nk, d, frame, left, right, sinks, dtype, ragged=False, train=False):
    case = {"op": "window", "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d, "frame": frame, "left": left,
            "right": right, "sinks": sinks, "dtype": dtype, "ragged": ragged, "train": train}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one new token of each of 4 streams at its own far position: latency
        _norm("norm 1 token", 4, 24, 24, 1, (16, 56, 56), 45, 80, 100000, "bf16", ragged=True),
        # a whole layer: 40 heads of a 21 x 30 x 52 grid, q and k
        _norm("norm layer", 1, 40, 40, 32760, (44, 42, 42), 30, 52, 0, "bf16"),
        # 32-bit tensors, an odd token count, grouped key heads, positions from the middle of a frame
        _norm("norm f32 odd", 2, 12, 4, 4097, (16, 24, 24), 30, 45, 731, "f32"),
        # training step of a 13 x 30 x 45 layer: outputs, gradients of q and k and of both weights
        _norm("norm train", 1, 48, 48, 17550, (16, 24, 24), 30, 45, 0, "bf16", train=True),
        # one new token over a cache: 4 frames of 1560 tokens and the first frame
        _window("window 1 token", 1, 40, 40, 1, 32760, 128, 1560, 4, 0, 1, "bf16"),
        # a batch of caches of different lengths, shared key heads, a token window with 4 sink tokens
        _window("window batch", 16, 32, 8, 1, 16384, 128, 1, 4095, 0, 4, "bf16", ragged=True),
        # the newest frame over the cache: causal by frame
        _window("window frame", 1, 40, 40, 1560, 32760, 128, 1560, 6, 0, 1, "bf16"),
        # a whole layer: two frames to either side and the first one
        _window("window layer", 1, 40, 40, 32760, 32760, 128, 1560, 2, 2, 1, "bf16"),
        # 32-bit tensors, a padded batch, odd lengths, a token window
        _window("window f32 odd", 2, 6, 3, 1777, 1777, 64, 1, 300, 0, 5, "f32", ragged=True),
        # training step, frames of 1350 tokens, one to either side and the first one
        _window("window train", 1, 48, 48, 17550, 17550, 64, 1350, 1, 1, 1, "bf16", train=True),
        # training step on a padded batch with shared key heads, a causal token window
        _window("window train odd", 3, 16, 4, 4001, 4001, 128, 1, 1023, 0, 4, "bf16", ragged=True, train=True),
        # 32-bit training step
        _window("window train f32", 1, 8, 8, 1430, 1430, 128, 143, 2, 1, 1, "f32", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    B = rng.choice([1, 1, 2, 3, 5])
    Hkv = rng.choice([1, 3, 4, 8, 12])
    H = Hkv * rng.choice([1, 1, 2, 4])
    train = rng.random() < 0.4
    ragged = rng.random() < 0.4
    if rng.random() < 0.4:
        split = rng.choice([(16, 24, 24), (16, 56, 56), (44, 42, 42), (128, 0, 0), (22, 20, 22)])
        return _norm(None, B, H, Hkv, _log(rng, 1, 30000 // B), split, rng.randint(1, 48), rng.randint(1, 80),
                     _log(rng, 1, 100000), dtype, ragged, train)
    d = rng.choice([64, 128])
    frame = rng.choice([1, 1, _log(rng, 2, 1600)])
    if rng.random() < 0.5 and not train:                     # the newest rows over a cache
        Nk = _log(rng, 16, 40000 // B)
        Nq = min(Nk // 2 if ragged else Nk, _log(rng, 1, 1600))
    else:
        Nk = Nq = _log(rng, 1, (12000 if dtype == "bf16" else 3000) // B)
    reach = max(1, Nk // frame)
    left = min(_log(rng, 1, reach), 6000 // frame + 1)
    right = rng.choice([0, 0, min(left, 2000 // frame + 1)])
    return _window(None, B, H, Hkv, max(1, Nq), Nk, d, frame, left, right, rng.choice([0, 1, 1, 4 if frame < 64 else 1]),
                   dtype, ragged, train)


# ---------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Keys in hand of each batch entry, and the position of its first query."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    k_len = [Nk - (b * Nk) // (2 * B) for b in range(B)] if case["ragged"] else [Nk] * B
    return k_len, [0 if Nq == Nk else n - Nq for n in k_len]


def _firsts(case):
    return [case["first"] + (977 * b if case["ragged"] else 0) for b in range(case["B"])]


def _tensor(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, s = _dtype(case), {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        d = case["d_t"] + case["d_h"] + case["d_w"]
        s["q"] = _tensor(g, (case["B"], case["H"], case["N"], d), dt, 1.7)
        s["k"] = _tensor(g, (case["B"], case["Hkv"], case["N"], d), dt, 0.6)
        s["wq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["wk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["first"] = ints(_firsts(case)) if case["ragged"] else None
        if case["train"]:
            s["gq"], s["gk"] = _tensor(g, s["q"].shape, dt), _tensor(g, s["k"].shape, dt)
        return s
    s["q"] = _tensor(g, (case["B"], case["H"], case["Nq"], case["d"]), dt, 1.5)   # logits of about 1.5 in spread
    s["k"] = _tensor(g, (case["B"], case["Hkv"], case["Nk"], case["d"]), dt)
    s["v"] = _tensor(g, (case["B"], case["Hkv"], case["Nk"], case["d"]), dt)
    k_len, q_first = _lengths(case)
    s["k_len"], s["q_first"] = ints(k_len), ints(q_first)
    if case["train"]:
        s["g"] = _tensor(g, s["q"].shape, dt)
    return s


# ---------------------------------------------------------------------------------- norm + RoPE
def _angles(case, firsts, device):
    """cos and sin [B, 1, N, d/2] of every token's pairs; angles in 64 bits."""
    pos = torch.tensor(firsts, device=device)[:, None] + torch.arange(case["N"], device=device)
    plane = case["Hg"] * case["Wg"]
    axes = (pos // plane, pos % plane // case["Wg"], pos % case["Wg"])
    ang = []
    for p, w in zip(axes, (case["d_t"], case["d_h"], case["d_w"])):
        i = torch.arange(w // 2, device=device, dtype=torch.float64)
        ang.append(p[..., None].double() * 10000.0 ** (-2.0 * i / max(w, 1)))
    a = torch.cat(ang, -1)[:, None]
    return torch.cos(a), torch.sin(a)


def _turn(x, cs, sn):
    """Pairs (2i, 2i+1) of the last axis turned by the angle."""
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * cs - x1 * sn, x0 * sn + x1 * cs), -1).flatten(-2)


def _norm_plain(x, w, cs, sn, gy):
    dt = x.dtype
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xh = x * r
    y = _turn(xh * w, cs, sn).to(dt)
    if gy is None:
        return [y]
    g = _turn(gy.float(), cs, -sn)
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return [y, dx.to(dt), (g * xh).sum((0, 1, 2))]


def _run_norm_plain(s):
    case = s["case"]
    cs, sn = (t.float() for t in _angles(case, _firsts(case), "cuda"))
    return (_norm_plain(s["q"], s["wq"], cs, sn, s.get("gq")) + _norm_plain(s["k"], s["wk"], cs, sn, s.get("gk")))


def _exact_norm(s):
    case = s["case"]
    first = _firsts(case)
    out = []
    for x, w, gy in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        B, H, N, d = x.shape
        y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        dx, dw = torch.empty_like(y), torch.zeros(d, dtype=torch.float64, device=x.device)
        w = w.double()
        for b in range(B):
            cs, sn = (t[b] for t in _angles(case, first, x.device))
            rot = torch.complex(cs, sn)
            for h in range(H):
                a = x[b, h].double()
                n = a / torch.sqrt((a ** 2).sum(-1, keepdim=True) / d + 1e-6)
                y[b, h] = torch.view_as_real(torch.view_as_complex((n * w).view(N, d // 2, 2)) * rot[0]).reshape(N, d)
                if gy is not None:
                    c = torch.view_as_complex(gy[b, h].double().reshape(N, d // 2, 2)) * rot[0].conj()
                    u = torch.view_as_real(c).reshape(N, d)
                    dw += (u * n).sum(0)
                    t = u * w
                    dx[b, h] = (t - n * (t * n).sum(-1, keepdim=True) / d) / torch.sqrt((a ** 2).sum(-1, keepdim=True) / d + 1e-6)
        out += [y] if gy is None else [y, dx, dw]
    return out


# ---------------------------------------------------------------------------------- window attention
def _span(case, p0, p1, n):
    """Keys that some query at a position in [p0, p1] sees: (sink end, window begin, window end)."""
    f = case["frame"]
    hi = min(n, (p1 // f + case["right"] + 1) * f)
    lo = min(max(0, (p0 // f - case["left"]) * f), hi)
    return min(case["sinks"] * f, lo), lo, hi


def _seen(case, pos, key, k_len):
    """Whether the key at `key` is visible from position `pos` (broadcast)."""
    f = case["frame"]
    fp, fk = pos // f, key // f
    return (key < k_len) & (fk <= fp + case["right"]) & ((fk >= fp - case["left"]) | (fk < case["sinks"]))


def _run_window_plain(s):
    """Row blocks against the keys that a block can see, the rest masked; a block's scores take about 1 GB."""
    case, q, k, v, g = s["case"], s["q"].float(), s["k"], s["v"], s.get("g")
    B, H, Nq, d = q.shape
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    k_len, q_first = _lengths(case)
    kl, qf = s["k_len"].view(B, 1, 1, 1, 1), s["q_first"].view(B, 1, 1, 1, 1)
    f = case["frame"]
    width = min(case["Nk"], (case["left"] + case["right"] + case["sinks"] + 1) * f)
    rows = max(1, min(Nq, (1 << 28) // (B * H * width)))
    rows = max(rows - rows % f, 1) if rows > f else rows
    scale = 1.0 / math.sqrt(d)
    q = q.view(B, Hkv, G, Nq, d)
    out = torch.empty_like(q)
    if g is not None:
        g = g.float().view(q.shape)
        dq, dk, dv = torch.empty_like(q), *(torch.zeros_like(t, dtype=torch.float32) for t in (k, v))
    for i0 in range(0, Nq, rows):
        i1 = min(Nq, i0 + rows)
        sink, lo, hi = _span(case, min(q_first) + i0, max(q_first) + i1 - 1, max(k_len))
        key = torch.cat((torch.arange(sink, device="cuda"), torch.arange(lo, hi, device="cuda")))
        kb, vb = (torch.cat((t[:, :, :sink], t[:, :, lo:hi]), 2).float() for t in (k, v))
        pos = qf + torch.arange(i0, i1, device="cuda").view(-1, 1)
        qb = (q[:, :, :, i0:i1] * scale).reshape(B, Hkv, -1, d)
        sc = (qb @ kb.transpose(-1, -2)).view(B, Hkv, G, i1 - i0, -1)
        sc.masked_fill_(~_seen(case, pos, key, kl), -math.inf)
        if key.numel() == 0:
            out[:, :, :, i0:i1] = 0
            if g is not None:
                dq[:, :, :, i0:i1] = 0
            continue
        top = sc.amax(-1, keepdim=True)
        sc = torch.exp(sc - torch.where(torch.isinf(top), 0.0, top))
        z = sc.sum(-1, keepdim=True)
        p = (sc / torch.where(z > 0, z, 1.0)).view(B, Hkv, -1, key.numel())
        del sc
        ob = p @ vb
        out[:, :, :, i0:i1] = ob.view(B, Hkv, G, -1, d)
        if g is not None:
            gb = g[:, :, :, i0:i1].reshape(B, Hkv, -1, d)
            ds = p * (gb @ vb.transpose(-1, -2) - (gb * ob).sum(-1, keepdim=True))
            dq[:, :, :, i0:i1] = (ds @ kb * scale).view(B, Hkv, G, -1, d)
            for acc, part in ((dk, ds.transpose(-1, -2) @ qb), (dv, p.transpose(-1, -2) @ gb)):
                acc[:, :, :sink] += part[:, :, :sink]
                acc[:, :, lo:hi] += part[:, :, sink:]
    dt, whole = s["q"].dtype, (B, H, Nq, d)
    if g is None:
        return [out.view(whole).to(dt)]
    return [out.view(whole).to(dt), dq.view(whole).to(dt), dk.to(dt), dv.to(dt)]


def _exact_window(s):
    case, q, k, v, g = s["case"], s["q"], s["k"], s["v"], s.get("g")
    B, H, Nq, d = q.shape
    G, Nk = H // k.shape[1], k.shape[2]
    k_len, q_first = _lengths(case)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if g is not None:
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v))
    key = torch.arange(Nk, device=q.device)
    step = max(1, (1 << 27) // Nk)
    for b in range(B):
        for h in range(H):
            kh, vh = k[b, h // G].double(), v[b, h // G].double()
            for i in range(0, Nq, step):
                qh = q[b, h, i:i + step].double()
                pos = q_first[b] + i + torch.arange(qh.shape[0], device=q.device)
                fp, fk = (pos // case["frame"])[:, None], (key // case["frame"])[None, :]
                sees = (key < k_len[b])[None, :] & (fk - fp <= case["right"])
                sees = sees & ((fp - fk <= case["left"]) | (fk < case["sinks"]))
                x = torch.where(sees, qh @ kh.T / d ** 0.5, torch.tensor(-1e300, dtype=torch.float64, device=q.device))
                p = torch.where(sees, torch.exp(x - x.max(1, keepdim=True).values), 0.0)
                p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
                o = p @ vh
                out[b, h, i:i + step] = o
                if g is not None:
                    gh = g[b, h, i:i + step].double()
                    dp = gh @ vh.T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) / d ** 0.5
                    dq[b, h, i:i + step] = ds @ kh
                    dk[b, h // G] += ds.T @ qh
                    dv[b, h // G] += p.T @ gh
    return [out] if g is None else [out, dq, dk, dv]


# ---------------------------------------------------------------------------------- the library's calls
@functools.lru_cache(maxsize=64)
def _norm_plan(B, H, Hkv, N, d_t, d_h, d_w, Hg, Wg, first, dtype):
    """What a model keeps for its layers of one shape: the parameters and the workspace's size.  The
    workspace itself comes from torch's allocator for each pass, so that passes on two streams, of
    two threads or in two graphs have one each."""
    from free_sparse_attention_b200 import capi
    p = capi.QkNormParams(B=B, H=H, Hkv=Hkv, N=N, d=d_t + d_h + d_w, d_t=d_t, d_h=d_h, d_w=d_w, Hg=Hg, Wg=Wg,
                          first=first, eps=1e-6, base=10000.0,
                          dtype=capi.SCOPE_BF16 if dtype == "bf16" else capi.SCOPE_F32)
    return capi, p, capi.alloc_qk_norm_workspace(p).numel()


@functools.lru_cache(maxsize=64)
def _window_plan(B, H, Hkv, Nq, Nk, d, frame, left, right, sinks, q_first, dtype):
    from free_sparse_attention_b200 import capi
    p = capi.WindowParams(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, frame=frame, left=left, right=right, sinks=sinks,
                          q_first=q_first, dtype=capi.SCOPE_BF16 if dtype == "bf16" else capi.SCOPE_F32)
    return capi, p, capi.alloc_window_workspace(p).numel()


def _run_norm_own(s):
    c = s["case"]
    capi, p, size = _norm_plan(c["B"], c["H"], c["Hkv"], c["N"], c["d_t"], c["d_h"], c["d_w"], c["Hg"], c["Wg"],
                               c["first"], c["dtype"])
    yq, yk = capi.qk_norm_rope3d(p, s["q"], s["k"], s["wq"], s["wk"], first=s["first"])
    if not c["train"]:
        return [yq, yk]
    ws = s["q"].new_empty(size, dtype=torch.uint8)
    dq, dk, dwq, dwk = capi.qk_norm_rope3d_backward(p, s["q"], s["k"], s["wq"], s["wk"], s["gq"], s["gk"],
                                                    first=s["first"], ws=ws)
    return [yq, dq, dwq, yk, dk, dwk]


def _run_window_own(s):
    c = s["case"]
    capi, p, size = _window_plan(c["B"], c["H"], c["Hkv"], c["Nq"], c["Nk"], c["d"], c["frame"], c["left"], c["right"],
                                 c["sinks"], c["Nk"] - c["Nq"], c["dtype"])
    ws = s["q"].new_empty(size, dtype=torch.uint8)
    at = {"q_first": s["q_first"], "k_len": s["k_len"]} if c["ragged"] else {}
    if not c["train"]:
        return [capi.window_attention(p, s["q"], s["k"], s["v"], ws=ws, **at)]
    o, lse = capi.window_attention(p, s["q"], s["k"], s["v"], ws=ws, lse=True, **at)
    dq, dk, dv = capi.window_attention_backward(p, s["q"], s["k"], s["v"], o, s["g"], lse, ws=ws, **at)
    return [o, dq, dk, dv]


def run(state):
    if own:
        return _run_norm_own(state) if state["case"]["op"] == "norm" else _run_window_own(state)
    return _run_norm_plain(state) if state["case"]["op"] == "norm" else _run_window_plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_window(s)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        d = case["d_t"] + case["d_h"] + case["d_w"]
        n = case["B"] * (case["H"] + case["Hkv"]) * case["N"] * d
        return {"bytes": n * es * (4 if case["train"] else 2), "flops": n * (24 if case["train"] else 8)}
    k_len, q_first = _lengths(case)
    f, pairs, keys = case["frame"], 0, 0
    for n, p0 in zip(k_len, q_first):
        pos = torch.arange(p0, p0 + case["Nq"], dtype=torch.int64)
        hi = ((pos // f + case["right"] + 1) * f).clamp(max=n)
        lo = torch.minimum(((pos // f - case["left"]) * f).clamp(min=0), hi)
        pairs += int((hi - lo + lo.clamp(max=case["sinks"] * f)).sum())
        sink, a, z = _span(case, p0, p0 + case["Nq"] - 1, n)
        keys += sink + z - a
    H, Hkv, d, rows = case["H"], case["Hkv"], case["d"], case["B"] * case["H"] * case["Nq"]
    if case["train"]:   # read q, k, v and dO, write O, dQ and (every row of) dK, dV; 2 + 5 products
        total = 4 * rows * d + 2 * Hkv * keys * d + 2 * case["B"] * Hkv * case["Nk"] * d
        return {"bytes": total * es, "flops": 14 * H * pairs * d}
    return {"bytes": (2 * rows * d + 2 * Hkv * keys * d) * es, "flops": 4 * H * pairs * d}
