"""Generation with a small hybrid model (random weights) whose layers keep their
states in the pages of caches:

    python examples/hybrid_decoding.py

* a state space layer: projection, short convolution, selective scan, gate;
* a gated delta rule layer with a short convolution in front of q, k and v;
* a linear-attention layer with normalised, rotated queries and keys.

Packed prompts of different lengths leave their states in pages; single tokens
advance them in place, a batch of beams takes over pages with gdn_pages_fork,
and the last logits are checked against a prompt pass over each history. A
training step through CausalConv, SelectiveScan, QKRotary and LinearAttention
closes it.
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from chunked_gated_delta_05_amd import binding as gb  # noqa: E402

DIM, INNER, STATES, RANK, TAPS = 256, 512, 16, 16, 4
HEADS, WIDTH, VOCAB = 2, 128, 97


class Model:
    """x -> x + scan(x) -> x + delta(x) -> x + linear(x) -> logits, in fp32."""

    def __init__(self, device, seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=gen, device=device) / s[0] ** 0.5
        self.p = dict(
            embed=w(VOCAB, DIM) * VOCAB ** 0.5,
            s_in=w(DIM, 2 * INNER), s_conv=w(INNER, TAPS) * INNER ** 0.5 / 2, s_bias=torch.zeros(INNER, device=device),
            s_x=w(INNER, RANK + 2 * STATES), s_dt=w(RANK, INNER), s_dt_bias=torch.full((INNER,), -3.0, device=device),
            s_A=-torch.arange(1, STATES + 1, device=device).float().repeat(INNER, 1), s_skip=torch.ones(INNER, device=device),
            s_out=w(INNER, DIM),
            d_in=w(DIM, 3 * HEADS * WIDTH), d_conv=w(3 * HEADS * WIDTH, TAPS) * 14, d_gate=w(DIM, HEADS), d_beta=w(DIM, HEADS),
            d_out=w(HEADS * WIDTH, DIM),
            l_in=w(DIM, 3 * HEADS * WIDTH), l_q=torch.ones(WIDTH, device=device), l_k=torch.ones(WIDTH, device=device),
            l_out=w(HEADS * WIDTH, DIM))
        self.decay = -0.5 * 0.4 ** torch.arange(HEADS, device=device).float()
        self.freqs = gb.rotary_frequencies(64, 10000.0, factor=4, scaling="by_turns", original_length=2048, device=device)

    def caches(self, n_pages, device):
        """Pools of one layer each: [1, n_pages, ...] for the page operators."""
        z = lambda *s: torch.zeros(1, n_pages, *s, device=device)
        return dict(s_conv=z(TAPS - 1, INNER), s_scan=z(INNER, STATES), d_conv=z(TAPS - 1, 3 * HEADS * WIDTH),
                    delta=z(HEADS, WIDTH, WIDTH), linear=z(HEADS, WIDTH, WIDTH))

    def scan_inputs(self, x, conv):
        """u, dt, B, C, gate of the scan; conv: what runs the convolution."""
        p = self.p
        u, gate = (F.rms_norm(x, (DIM,)) @ p["s_in"]).split(INNER, -1)
        u = conv(u)
        dt, B, C = (u @ p["s_x"]).split([RANK, STATES, STATES], -1)
        return u, dt @ p["s_dt"], B.unsqueeze(-2), C.unsqueeze(-2), gate

    def heads(self, x):
        return [t.contiguous() for t in x.unflatten(-1, (3, HEADS, WIDTH)).unbind(-3)]

    def delta_inputs(self, x, conv):
        p, y = self.p, F.rms_norm(x, (DIM,))
        q, k, v = self.heads(conv(y @ p["d_in"]))
        return (F.normalize(q, dim=-1), F.normalize(k, dim=-1), v, -0.1 * F.softplus(y @ p["d_gate"]),
                torch.sigmoid(y @ p["d_beta"]))

    def linear_inputs(self, x, positions):
        p = self.p
        q, k, v = self.heads(F.rms_norm(x, (DIM,)) @ p["l_in"])
        q, k = gb.gdn_qk_rotary_fwd(q, k, self.freqs, positions, q_weight=p["l_q"], k_weight=p["l_k"], q_out=q, k_out=k)
        return q, k, v

    def prompts(self, tokens, positions, meta, caches=None, pages=None):
        """Logits of every token of packed prompts; their states go to pages."""
        p, x = self.p, self.p["embed"][tokens]
        to = lambda n: {} if caches is None else dict(final_out=caches[n][0], final_pages=pages)
        u, dt, B, C, gate = self.scan_inputs(x, lambda u: gb.gdn_conv_fwd(
            u, p["s_conv"], p["s_bias"], activation="silu", meta=meta, **to("s_conv"))[0])
        y, _, _ = gb.gdn_scan_fwd(u, dt, p["s_A"], B, C, p["s_skip"], gate, dt_bias=p["s_dt_bias"], dt_softplus=True,
                                  meta=meta, **to("s_scan"))
        x = x + y @ p["s_out"]
        q, k, v, g, beta = self.delta_inputs(x, lambda t: gb.gdn_conv_fwd(
            t, p["d_conv"], activation="silu", meta=meta, **to("d_conv"))[0])
        o, final, _ = gb.gdn_chunk_fwd(q, k, v, g, beta, meta=meta, output_final_state=True)
        if caches is not None:
            gb.gdn_pages_copy(caches["delta"], final[None], pages, torch.arange(len(pages), dtype=torch.int32, device=x.device))
        x = x + o.flatten(-2) @ p["d_out"]
        o, _ = gb.gdn_linattn_fwd(*self.linear_inputs(x, positions), self.decay, meta=meta, **to("linear"))
        return (x + o.flatten(-2) @ p["l_out"]) @ p["embed"].T

    def step(self, tokens, positions, caches, table):
        """Logits of one token for every slot; rows without a page are ignored."""
        p, x = self.p, self.p["embed"][tokens]
        u, dt, B, C, gate = self.scan_inputs(x, lambda u: gb.gdn_conv_step(
            u, p["s_conv"], caches["s_conv"][0], p["s_bias"], activation="silu", pages=table))
        x = x + gb.gdn_scan_step(u, dt, p["s_A"], B, C, caches["s_scan"][0], p["s_skip"], gate, dt_bias=p["s_dt_bias"],
                                 dt_softplus=True, pages=table) @ p["s_out"]
        q, k, v, g, beta = self.delta_inputs(x, lambda t: gb.gdn_conv_step(
            t, p["d_conv"], caches["d_conv"][0], activation="silu", pages=table))
        x = x + gb.gdn_recurrent_step(q, k, v, g, beta, caches["delta"][0], pages=table).flatten(-2) @ p["d_out"]
        o = gb.gdn_linattn_step(*self.linear_inputs(x, positions), self.decay, caches["linear"][0], pages=table)
        return (x + o.flatten(-2) @ p["l_out"]) @ p["embed"].T


def decode(device="cuda", lengths=(37, 1, 150), beams=3, steps=9, seed=0):
    """Largest difference of the last logits from the prompt pass over each
    beam's history, relative to their rms."""
    model = Model(device, seed)
    gen = torch.Generator(device).manual_seed(seed + 1)
    offs = [0]
    for n in lengths:
        offs.append(offs[-1] + n)
    places = lambda ls: torch.cat([torch.arange(n, device=device) for n in ls])
    prompt = torch.randint(0, VOCAB, (offs[-1],), generator=gen, device=device)
    groups, slots = len(lengths), len(lengths) * beams
    n_pages = slots + 2
    caches = model.caches(n_pages, device)
    free = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    logits = model.prompts(prompt, places(lengths), gb.make_meta(offs, offs[-1], device), caches, free[:groups].clone())
    score, token = F.log_softmax(logits[torch.tensor(offs[1:], device=device) - 1], -1).topk(beams)
    table = torch.full((slots,), -1, dtype=torch.int32, device=device)
    table[::beams] = free[:groups]
    spare = free[groups:].clone()
    base = torch.arange(0, slots, beams, device=device)
    parent, at = base[:, None].expand(groups, beams), torch.tensor(lengths, device=device).repeat_interleave(beams)
    history = prompt.new_zeros(slots, 0)
    for _ in range(steps):
        # one plan for the pages of every cache: the tables stay alike
        forks = [gb.gdn_pages_fork(pool, table, parent.flatten().to(torch.int32), spare=spare) for pool in caches.values()]
        table, spare = forks[0][0], forks[0][1][:n_pages]
        history = torch.cat([history[parent.flatten()], token.reshape(slots, 1)], 1)
        logits = model.step(token.flatten(), at, caches, table)
        at = at + 1
        total = score.reshape(slots, 1) + F.log_softmax(logits, -1)
        score, best = total.view(groups, beams * VOCAB).topk(beams)
        parent, token = base[:, None] + best // VOCAB, best % VOCAB
    seqs = [torch.cat([prompt[offs[s // beams]:offs[s // beams + 1]], history[s]]) for s in range(slots)]
    ends = torch.tensor([len(s) for s in seqs]).cumsum(0)
    whole = model.prompts(torch.cat(seqs), places([len(s) for s in seqs]), gb.make_meta([0] + ends.tolist(), int(ends[-1]), device))
    want = whole[ends.to(device) - 1]
    return ((logits - want).abs().max() / want.square().mean().sqrt()).item()


def loss(p, x, target, freqs, decay):
    """A scan and a linear-attention layer through the autograd ops."""
    u, gate = (x @ p["s_in"]).split(INNER, -1)
    u, _ = gb.CausalConv.apply(u, p["s_conv"], p["s_bias"], None, "silu")
    dt, B, C = (u @ p["s_x"]).split([RANK, STATES, STATES], -1)
    y, _ = gb.SelectiveScan.apply(u, dt @ p["s_dt"], p["s_A"], B.unsqueeze(-2), C.unsqueeze(-2), p["s_skip"], gate,
                                  p["s_dt_bias"], None, True)
    x = x + y @ p["s_out"]
    q, k, v = (x @ p["l_in"]).unflatten(-1, (3, HEADS, WIDTH)).unbind(-3)
    q, k = gb.QKRotary.apply(q, k, freqs, None, p["l_q"], p["l_k"])
    o, _ = gb.LinearAttention.apply(q, k, v, decay)
    return F.mse_loss(x + o.flatten(-2) @ p["l_out"], target)


def train(device="cuda", steps=4, seed=0, rate=0.2):
    """Losses of a few gradient steps, and the last gradients."""
    model = Model(device, seed)
    names = [n for n in model.p if n[:2] in ("s_", "l_")]
    gen = torch.Generator(device).manual_seed(seed + 2)
    x, target = (torch.randn(2, 90, DIM, generator=gen, device=device) for _ in range(2))
    losses = []
    for _ in range(steps):
        p = {n: model.p[n].detach().requires_grad_() for n in names}
        value = loss(p, x, target, model.freqs, model.decay)
        grads = dict(zip(names, torch.autograd.grad(value, list(p.values()))))
        with torch.no_grad():
            for n in names:
                model.p[n] = p[n] - rate * grads[n]
        losses.append(value.item())
    return losses, grads, p, (x, target, model.freqs, model.decay)


if __name__ == "__main__":
    print(f"last logits: max|difference|/rms = {decode():.2e} from the prompt pass")
    print("training losses:", ", ".join(f"{v:.4f}" for v in train()[0]))
