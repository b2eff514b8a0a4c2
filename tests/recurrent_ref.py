"""Plain 64-bit references of the recurrent-state operators on the CPU,
written from their definitions, token by token; and of each the same formula
over absolute values, the scale that rounding errors are bounded against."""
from __future__ import annotations

import torch

F64 = torch.float64


def heads(x, H):
    """[.., h, D] as fp64 [tokens, H, D] on the CPU, shared heads repeated."""
    x = x.detach().cpu().double()
    x = x.reshape(-1, *x.shape[-2:])
    return x.repeat_interleave(H // x.shape[1], dim=1)


def linattn(q, k, v, decay, scale, offsets, S0, absolute=False):
    """o [tokens, H, V] and final states [units, H, K, V] of S = d S + k v^T,
    o = scale S^T q. absolute: of the absolute values (S0 too)."""
    H = decay.shape[0]
    d = torch.exp(decay.detach().cpu().double())[:, None, None]
    q, k, v = heads(q, H), heads(k, H), heads(v, H)
    n = len(offsets) - 1
    S0 = torch.zeros(n, H, k.shape[-1], v.shape[-1], dtype=F64) if S0 is None else S0.detach().cpu().double()
    if absolute:
        q, k, v, S0, scale = q.abs(), k.abs(), v.abs(), S0.abs(), abs(scale)
    o = torch.zeros(q.shape[0], H, v.shape[-1], dtype=F64)
    final = torch.zeros_like(S0)
    for u in range(n):
        S = S0[u]
        for t in range(offsets[u], offsets[u + 1]):
            S = d * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t][:, None, :] @ S).squeeze(1)
        final[u] = S
    return o, final


def linattn_grads(q, k, v, decay, scale, offsets, S0, dout, dht, absolute=False):
    """dq, dk, dv (per head, [tokens, H, D]) and dh0, by the recurrences of the
    states and of their gradients."""
    H = decay.shape[0]
    d = torch.exp(decay.detach().cpu().double())[:, None, None]
    q, k, v, do = heads(q, H), heads(k, H), heads(v, H), heads(dout, H)
    n = len(offsets) - 1
    zero = torch.zeros(n, H, k.shape[-1], v.shape[-1], dtype=F64)
    S0 = zero if S0 is None else S0.detach().cpu().double()
    dht = zero if dht is None else dht.detach().cpu().double()
    if absolute:
        q, k, v, do, S0, dht, scale = q.abs(), k.abs(), v.abs(), do.abs(), S0.abs(), dht.abs(), abs(scale)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dh0 = torch.zeros_like(zero)
    for u in range(n):
        S, D = S0[u], dht[u]
        for t in range(offsets[u], offsets[u + 1]):
            S = d * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (S @ do[t][:, :, None]).squeeze(-1)
        for t in reversed(range(offsets[u], offsets[u + 1])):
            D = D + scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = (D @ v[t][:, :, None]).squeeze(-1)
            dv[t] = (k[t][:, None, :] @ D).squeeze(1)
            D = d * D
        dh0[u] = D
    return dq, dk, dv, dh0


def shared(x, h):
    """Sums the heads of [tokens, H, D] that share one of h."""
    return x.view(x.shape[0], h, x.shape[1] // h, x.shape[2]).sum(2)


def linattn_step(q, k, v, decay, scale, S, absolute=False):
    """One token of rows [N, h, D] on states [N, H, K, V]: o, new states."""
    H = S.shape[1]
    d = torch.exp(decay.detach().cpu().double())[:, None, None]
    q, k, v, S = heads(q, H), heads(k, H), heads(v, H), S.detach().cpu().double()
    if absolute:
        q, k, v, S, scale = q.abs(), k.abs(), v.abs(), S.abs(), abs(scale)
    S = d * S + k[..., :, None] * v[..., None, :]
    return scale * (q[..., None, :] @ S).squeeze(-2), S


def delta_step(q, k, v, g, beta, scale, S, exp2=False, norm=False, sigmoid=False, absolute=False):
    """One token of the gated delta rule: o, new states."""
    H = S.shape[1]
    q, k, v, S = heads(q, H), heads(k, H), heads(v, H), S.detach().cpu().double()
    g, beta = g.detach().cpu().double(), beta.detach().cpu().double()
    if norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    if sigmoid:
        beta = torch.sigmoid(beta)
    decay = torch.exp2(g) if exp2 else torch.exp(g)
    decay = decay[..., None] if g.dim() == 3 else decay[..., None, None]
    if absolute:
        q, k, v, S, beta, scale = q.abs(), k.abs(), v.abs(), S.abs(), beta.abs(), abs(scale)
    S = decay * S
    kS = (k[..., None, :] @ S).squeeze(-2)
    r = v + kS if absolute else v - kS
    S = S + beta[..., None, None] * k[..., :, None] * r[..., None, :]
    return scale * (q[..., None, :] @ S).squeeze(-2), S


def fork(table, parent, spare, n_pages):
    """New table, copies (source, destination) and pages left, on lists."""
    page = lambda p: 0 <= p < n_pages
    n = len(table)
    source = [p if 0 <= p < n and page(table[p]) else -1 for p in parent]
    continued = set(source)
    free = [table[s] for s in range(n) if page(table[s]) and s not in continued] + [p for p in spare if page(p)]
    new, copies, seen = [], [], set()
    for i in range(n):
        p = source[i]
        if p < 0:
            new.append(-1)
        elif p not in seen:
            seen.add(p)
            new.append(table[p])
        elif len(copies) < len(free):
            new.append(free[len(copies)])
            copies.append((table[p], new[-1]))
        else:
            new.append(-1)
    left = free[len(copies):]
    return new, copies, left + [-1] * (n + len(spare) - len(left))


def compact(table, n_pages):
    """New table, moves (source, destination) and the count, on lists."""
    used = sorted({p for p in table if 0 <= p < n_pages})
    count = len(used)
    inuse = set(used)
    holes = [p for p in range(count) if p not in inuse]
    moves = list(zip([p for p in used if p >= count], holes))
    to = dict(moves)
    return [to.get(p, p) if 0 <= p < n_pages else -1 for p in table], moves, count
