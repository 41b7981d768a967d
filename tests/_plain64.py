"""The rotary, packed-prompt and drafted-tree operators from their definitions, in double (torch, CPU or GPU)."""
from __future__ import annotations

import math

import torch


def frequencies(rot, base, scaling=None, factor=1.0, trained=0):
    """(radians per position of every pair, factor on the result)."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "ntk":
        return [(base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if scaling == "yarn":
        # pair index with `turns` full turns over the trained length
        at = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, pos, freq, scale, rot, layout, inverse=False):
    """x [B, H, N, d]; pos [B, N]."""
    y = x.double().clone()
    w = torch.tensor(freq, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, :, None] * w * (-1.0 if inverse else 1.0)
    n = rot // 2
    i = torch.arange(n, device=x.device)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    u, v = x.double()[..., a], x.double()[..., b]
    y[..., a] = scale * (u * torch.cos(ang) - v * torch.sin(ang))
    y[..., b] = scale * (u * torch.sin(ang) + v * torch.cos(ang))
    return y


def attend(q, k, v, visible):
    """q [H, n, d], k, v [Hkv, m, d], visible [n, m] -> O [H, n, d], lse [H, n]; a row that sees nothing: 0, -inf."""
    G = q.shape[0] // k.shape[0]
    kk, vv = k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
    s = q.double() @ kk.transpose(1, 2) / math.sqrt(q.shape[-1])
    s = torch.where(visible, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, p @ vv / z, torch.zeros_like(q, dtype=torch.float64))
    lse = (m + torch.log(z)).squeeze(-1)
    return o, lse


def packed(q, k, v, cu):
    """O [H, T, d], lse [H, T] over the sequences [cu[i], cu[i+1]); zeros elsewhere."""
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        t = torch.arange(b - a, device=q.device)
        o[:, a:b], lse[:, a:b] = attend(q[:, a:b], k[:, a:b], v[:, a:b], t[:, None] >= t[None, :])
    return o, lse


def packed_grad(q, k, v, do, cu):
    """dQ, dK, dV of sum(dO * O) by autograd over the definition above."""
    q, k, v = (x.double().detach().clone().requires_grad_() for x in (q, k, v))
    loss = q.new_zeros(())
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        t = torch.arange(b - a, device=q.device)
        o, _ = attend(q[:, a:b], k[:, a:b], v[:, a:b], t[:, None] >= t[None, :])
        loss = loss + (o * do[:, a:b].double()).sum()
    loss.backward()
    return tuple(torch.zeros_like(x) if x.grad is None else x.grad for x in (q, k, v))


def ancestors(parent):
    """parent: list. visible[t] = the set of drafted tokens t sees, empty for an absent slot."""
    out = []
    for t, p in enumerate(parent):
        if p == -1:
            out.append({t})
        elif p < -1 or p >= t or not out[p]:
            out.append(set())
        else:
            out.append(out[p] | {t})
    return out


def tree(q, k, v, lens, parent):
    """q [B, H, T, d], caches k, v [B, Hkv, N, d], lens [B], parent [B][T] lists."""
    B, H, T, _ = q.shape
    N = k.shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = lens[b]
        if n < 0 or n + T > N:
            continue
        see = ancestors(parent[b])
        vis = torch.zeros((T, n + T), dtype=torch.bool)
        for t in range(T):
            if see[t]:
                vis[t, :n] = True
                vis[t, [n + u for u in see[t]]] = True
        used = vis.any(0).to(q.device)
        kk, vv = k[b, :, :n + T].clone(), v[b, :, :n + T].clone()
        kk[:, ~used] = 0  # rows nobody sees may hold anything
        vv[:, ~used] = 0
        o[b], lse[b] = attend(q[b], kk, vv, vis.to(q.device))
    return o, lse
