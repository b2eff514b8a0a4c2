"""LinearAttention as an autograd op, on the CPU: the two native calls are
replaced by plain torch ones, what is tested is the op around them."""
import pytest
import torch

from chunked_gated_delta_05_amd import binding as gb

B, T, H, K = 2, 5, 2, 64


def plain(q, k, v, decay, S0, scale):
    S = torch.zeros(B, H, K, K, dtype=q.dtype) if S0 is None else S0
    o = []
    for t in range(T):
        S = torch.exp(decay)[:, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append(scale * (q[:, t, :, None, :] @ S).squeeze(-2))
    return torch.stack(o, 1), S


@pytest.fixture
def inputs(monkeypatch):
    def fwd(q, k, v, decay, scale=None, *, meta=None, initial_state=None, output_final_state=False):
        return plain(q, k, v, decay, initial_state, K ** -0.5 if scale is None else scale)

    def bwd(q, k, v, decay, dout, scale=None, *, meta=None, initial_state=None, dht=None, want_dh0=True):
        with torch.enable_grad():
            x = [t.detach().requires_grad_() for t in (q, k, v)]
            s0 = None if initial_state is None else initial_state.detach().requires_grad_()
            o, fin = plain(*x, decay.detach(), s0, K ** -0.5 if scale is None else scale)
            loss = (o * dout).sum() + (0 if dht is None else (fin * dht).sum())
            g = torch.autograd.grad(loss, x + ([s0] if s0 is not None and want_dh0 else []))
        return dict(zip(("dq", "dk", "dv", "dh0"), (t.detach() for t in g)))   # native outputs carry no graph

    monkeypatch.setattr(gb, "gdn_linattn_fwd", fwd)
    monkeypatch.setattr(gb, "gdn_linattn_bwd", bwd)
    gen = torch.Generator().manual_seed(0)
    x = [torch.randn(B, T, H, K, generator=gen, dtype=torch.float64).requires_grad_() for _ in range(3)]
    return (*x, torch.tensor([-0.1, -0.5], dtype=torch.float64))


def test_first_order_gradients(inputs):
    q, k, v, decay = inputs
    o, fin = gb.LinearAttention.apply(q, k, v, decay)
    want, wfin = plain(q, k, v, decay, None, K ** -0.5)
    w = torch.randn(o.shape, generator=torch.Generator().manual_seed(1), dtype=o.dtype)
    got = torch.autograd.grad((o * w).sum() + fin.square().sum(), (q, k, v))
    for a, b in zip(got, torch.autograd.grad((want * w).sum() + wfin.square().sum(), (q, k, v))):
        torch.testing.assert_close(a, b)


def test_a_second_order_gradient_is_refused(inputs):
    q, k, v, decay = inputs
    o, _ = gb.LinearAttention.apply(q, k, v, decay)
    dk, = torch.autograd.grad(o.square().sum(), k, create_graph=True)   # a gradient penalty
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (o.sum() + dk.square().sum()).backward()


def test_a_gradient_of_decay_is_refused(inputs):
    q, k, v, decay = inputs
    learnt = decay.clone().requires_grad_()
    with torch.no_grad():   # evaluating with a parameter is fine
        o, _ = gb.LinearAttention.apply(q, k, v, learnt)
    assert torch.equal(o, gb.LinearAttention.apply(q, k, v, decay)[0])
    o, _ = gb.LinearAttention.apply(q, k, v, learnt)
    with pytest.raises(NotImplementedError, match="decay"):
        o.sum().backward()
    assert learnt.grad is None
