"""The 64-bit references of the operators around the recurrent layers: their
gradients against autograd's and against differences."""
import pytest
import torch

import mixer_ref as ref

F64 = torch.float64


def leaf(*shape, seed=0, scale=1.0, shift=0.0):
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * scale + shift
    return x.requires_grad_()


def conv_plain(x, w, b, silu, offs, s0):
    ys, finals = [], []
    for u, (lo, hi) in enumerate(zip(offs, offs[1:])):
        seq = torch.cat([s0[u], x[lo:hi]])
        z = b + sum(seq[j:j + hi - lo] * w[:, j] for j in range(w.shape[1]))
        ys.append(z * torch.sigmoid(z) if silu else z)
        finals.append(seq[hi - lo:])
    return torch.cat(ys), torch.stack(finals)


def scan_plain(u, dt, A, B, C, skip, gate, bias, softplus, offs, s0):
    raw = dt + bias
    t = torch.log1p(torch.exp(raw)) if softplus else raw
    rep = u.shape[1] // B.shape[1]
    outs, finals = [], []
    for i, (lo, hi) in enumerate(zip(offs, offs[1:])):
        h = s0[i]
        for n in range(lo, hi):
            Bn, Cn = B[n].repeat_interleave(rep, 0), C[n].repeat_interleave(rep, 0)
            h = torch.exp(t[n][:, None] * A) * h + (t[n] * u[n])[:, None] * Bn
            outs.append(((h * Cn).sum(-1) + skip * u[n]) * gate[n] * torch.sigmoid(gate[n]))
        finals.append(h)
    return torch.stack(outs), torch.stack(finals)


def check(plain, args, leaves, names, refer):
    out, final = plain(*args)
    dout, dfin = torch.randn_like(out), torch.randn_like(final)
    loss = lambda: sum((a * b).sum() for a, b in zip(plain(*args), (dout, dfin)))
    got = refer(dout, dfin)
    assert torch.allclose(got[0], out, atol=1e-11) and torch.allclose(got[1], final, atol=1e-11)
    grads = torch.autograd.grad(loss(), leaves)
    for name, x, g in zip(names, leaves, grads):
        assert torch.allclose(got[2][name], g, rtol=1e-9, atol=1e-10), name
        d = torch.randn_like(x)
        with torch.no_grad():
            x += 1e-5 * d
            hi = loss()
            x -= 2e-5 * d
            lo = loss()
            x += 1e-5 * d
        assert abs((hi - lo) / 2e-5 - (d * g).sum()) <= 1e-6 * (1 + (d * g).abs().sum()), name


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("W,offs", [(4, [0, 1, 8]), (2, [0, 5]), (3, [0, 2, 3, 9])])
def test_conv_gradients(W, offs, silu):
    n, D = len(offs) - 1, 8
    x, w, b, s0 = leaf(offs[-1], D), leaf(D, W, seed=1), leaf(D, seed=2), leaf(n, W - 1, D, seed=3)
    check(conv_plain, (x, w, b, silu, offs, s0), (x, w, b, s0), ("dx", "dweight", "dbias", "dinitial"),
          lambda dout, dfin: ref.conv(x, w, b, silu, offs, s0, dout, dfin))


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("G,offs", [(1, [0, 1, 6]), (2, [0, 7])])
def test_scan_gradients(G, offs, softplus):
    N, n, D, S = offs[-1], len(offs) - 1, 16, 8
    a = (leaf(N, D), leaf(N, D, seed=1, scale=0.3), leaf(D, S, seed=2, shift=-1.0), leaf(N, G, S, seed=3),
         leaf(N, G, S, seed=4), leaf(D, seed=5), leaf(N, D, seed=6), leaf(D, seed=7, scale=0.3))
    s0 = leaf(n, D, S, seed=8)
    check(scan_plain, (*a, softplus, offs, s0), (*a, s0),
          ("du", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias", "dh0"),
          lambda dout, dfin: ref.scan(*a, softplus, offs, s0, dout, dfin))
