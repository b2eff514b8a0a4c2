"""Plain 64-bit references of the operators around the recurrent layers on the
CPU, written from their definitions, token by token; and of each the same
formula over absolute values, the scale that rounding errors are bounded
against."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def f64(x):
    return None if x is None else x.detach().cpu().double()


def flat(x, n):
    """[.., last n axes] with one token axis, fp64 on the CPU."""
    x = f64(x)
    return None if x is None else x.reshape(-1, *x.shape[x.dim() - n:])


def sigmoid(x):
    return 1 / (1 + torch.exp(-x))


# ------------------------------------------------------------------ convolution
def conv(x, weight, bias, silu, offsets, S0, dout=None, dfinal=None, absolute=False):
    """y, final states and, with dout, a dict of the gradients."""
    x, w, b, S0, dout, dfinal = flat(x, 1), f64(weight), f64(bias), f64(S0), flat(dout, 1), f64(dfinal)
    D, W = w.shape
    n = len(offsets) - 1
    if S0 is None:
        S0 = torch.zeros(n, W - 1, D, dtype=F64)
    b = torch.zeros(D, dtype=F64) if b is None else b
    y, final, dx = torch.zeros_like(x), torch.zeros_like(S0), torch.zeros_like(x)
    d0, dw, db = torch.zeros_like(S0), torch.zeros_like(w), torch.zeros(D, dtype=F64)
    size = (lambda t: t.abs()) if absolute else (lambda t: t)
    for u in range(n):
        lo, hi = offsets[u], offsets[u + 1]
        seq = torch.cat([S0[u], x[lo:hi]])
        dseq = torch.zeros_like(seq)
        final[u] = seq[hi - lo:]
        for t in range(hi - lo):
            win = seq[t:t + W]                                  # [W, D]
            z = b + (win * w.t()).sum(0)
            sg = sigmoid(z)
            slope = sg * (1 + z * (1 - sg)) if silu else torch.ones_like(z)
            if absolute:
                z = b.abs() + (win * w.t()).abs().sum(0)
                y[lo + t] = 1.1 * z if silu else z              # |d silu| <= 1.1
            else:
                y[lo + t] = z * sg if silu else z
            if dout is None:
                continue
            # the slope of silu changes by at most 0.5 for each unit of z
            dz = size(dout[lo + t]) * (size(slope) + (0.5 * z if absolute and silu else 0))
            dseq[t:t + W] += dz * size(w.t())
            dw += (dz * size(win)).t()
            db += dz
        if dout is not None:
            if dfinal is not None:
                dseq[hi - lo:] += size(dfinal[u])
            dx[lo:hi], d0[u] = dseq[W - 1:], dseq[:W - 1]
    if dout is None:
        return y, final
    return y, final, {"dx": dx, "dweight": dw, "dbias": db, "dinitial": d0}


def conv_step(x, weight, bias, silu, state):
    """Rows [N,D] on states [N,W-1,D]: y, its scale, new states."""
    offsets = list(range(x.shape[0] + 1))
    y, final = conv(x, weight, bias, silu, offsets, state)
    return y, conv(x, weight, bias, silu, offsets, state, absolute=True)[0], final


# ------------------------------------------------------------------ scan
def scan(u, dt, A, B, C, skip, gate, dt_bias, softplus, offsets, S0, dout=None, dht=None, absolute=False):
    """out, final states and, with dout, a dict of the gradients. absolute: the
    decays and time steps as they are, everything else by absolute value."""
    u, dt, A, gate, dout = flat(u, 1), flat(dt, 1), f64(A), flat(gate, 1), flat(dout, 1)
    B, C, skip, dt_bias, S0, dht = flat(B, 2), flat(C, 2), f64(skip), f64(dt_bias), f64(S0), f64(dht)
    N, D = u.shape
    S, G, n = A.shape[1], B.shape[1], len(offsets) - 1
    raw = dt + (0 if dt_bias is None else dt_bias)
    t_ = torch.nn.functional.softplus(raw, threshold=60) if softplus else raw
    dsoft = sigmoid(raw) if softplus else torch.ones_like(raw)
    decay = torch.exp(t_[..., None] * A)                          # [N, D, S]
    each = lambda x: x.repeat_interleave(D // G, dim=1)
    B, C = each(B), each(C)
    skip = torch.zeros(D, dtype=F64) if skip is None else skip
    sg = None if gate is None else sigmoid(gate)
    open_ = torch.ones_like(u) if gate is None else gate * sg
    slope = None if gate is None else sg * (1 + gate * (1 - sg))
    zero = torch.zeros(n, D, S, dtype=F64)
    S0 = zero if S0 is None else S0
    dht = zero if dht is None else dht
    if absolute:
        u, t_, B, C, skip, S0, dht, open_ = (x.abs() for x in (u, t_, B, C, skip, S0, dht, open_))
        A = A.abs()
        dout = None if dout is None else dout.abs()
        slope = None if slope is None else slope.abs() + 0.1 * gate.abs() + 0.1
    out, final, h = torch.zeros_like(u), torch.zeros_like(S0), torch.zeros(N, D, S, dtype=F64)
    y = torch.zeros_like(u)
    for i in range(n):
        s = S0[i]
        for t in range(offsets[i], offsets[i + 1]):
            s = decay[t] * s + (t_[t] * u[t])[:, None] * B[t]
            h[t] = s
            y[t] = (C[t] * s).sum(-1) + skip * u[t]
        final[i] = s
    out = y * open_
    if dout is None:
        return out, final
    dy = dout * open_
    r = {k: torch.zeros_like(u) for k in ("du", "ddt")}
    dB, dC, dA, dh0 = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A), torch.zeros_like(S0)
    for i in range(n):
        E = dht[i]
        for t in reversed(range(offsets[i], offsets[i + 1])):
            g = dy[t][:, None] * C[t] + E
            before = h[t - 1] if t > offsets[i] else S0[i]
            dC[t], dB[t] = dy[t][:, None] * h[t], (t_[t] * u[t])[:, None] * g
            ddu = (g * B[t]).sum(-1)
            E = decay[t] * g
            w = E * before
            dA += w * t_[t][:, None]
            r["du"][t] = t_[t] * ddu + skip * dy[t]
            r["ddt"][t] = (u[t] * ddu + (w * A).sum(-1)) * dsoft[t]
        dh0[i] = E
    grouped = lambda x: x.view(N, G, D // G, S).sum(2)
    r.update(dA=dA, dB=grouped(dB), dC=grouped(dC), dskip=(dy * u).sum(0), ddt_bias=r["ddt"].sum(0), dh0=dh0)
    if gate is not None:
        r["dgate"] = dout * y * slope
    return out, final, r


# ------------------------------------------------------------------ norms and rotation
def rotary(q, k, freqs, positions, norm, q_weight, k_weight, eps, interleaved, amplitude, dq=None, dk=None):
    """Dict of q, k and, with dq and dk, of the gradients (by autograd of the
    rotation as a product of complex numbers)."""
    out = {}
    lead = q.shape[:-2]
    if positions is None:
        positions = torch.arange(lead[1]).expand(lead)
    pos = f64(positions)
    for name, x, w, d in (("q", q, q_weight, dq), ("k", k, k_weight, dk)):
        x = f64(x).requires_grad_(d is not None)
        w = None if w is None else f64(w).requires_grad_(d is not None)
        y = x
        if norm is not None:
            size = (x * x).mean(-1, keepdim=True) if norm == "rms" else (x * x).sum(-1, keepdim=True)
            y = x / torch.sqrt(size + eps)
        y = y if w is None else y * w
        if freqs is not None:
            R = 2 * freqs.numel()
            angle = pos[..., None, None] * f64(freqs)
            turn = torch.polar(torch.full_like(angle, amplitude), angle)
            pairs = y[..., :R].unflatten(-1, (R // 2, 2)) if interleaved else \
                y[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
            y = torch.cat([z, y[..., R:]], -1)
        out[name] = y.detach()
        if d is not None:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], f64(d))
            out["d" + name] = grads[0]
            if w is not None:
                out["d" + name + "_weight"] = grads[1]
    return out
