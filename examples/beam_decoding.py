"""Beam search with a small recurrent model whose states live in the pages of
one cache: a gated delta rule layer and a linear-attention layer (random
weights), packed prompts of different lengths, then single tokens.

    python examples/beam_decoding.py

Prompts run through gdn_chunk_fwd and gdn_linattn_fwd and leave their states in
pages; each step advances every beam's states with gdn_recurrent_step and
gdn_linattn_step, picks the best continuations and moves the cache along with
gdn_pages_fork; at the end gdn_pages_compact packs the pages in use. The last
step's logits are checked against a prompt pass over each beam's whole history.
A training step of the linear-attention layer (LinearAttention) closes it.
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

HEADS, WIDTH, VOCAB = 4, 128, 211
DIM = HEADS * WIDTH


class Model:
    """x -> x + delta(x) -> x + linear(x) -> logits; layers 0 and 1 of the cache."""

    def __init__(self, device, seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=gen, device=device) / s[0] ** 0.5
        self.embed = w(VOCAB, DIM) * VOCAB ** 0.5
        self.qkv = [w(DIM, 3 * DIM), w(DIM, 3 * DIM)]
        self.gate, self.beta = w(DIM, HEADS), w(DIM, HEADS)
        self.out = [w(DIM, DIM), w(DIM, DIM)]
        self.decay = -0.5 * 0.4 ** torch.arange(HEADS, device=device).float()

    def heads(self, x, layer):
        """q, k, v as strided views of one projection, bf16 [.., HEADS, WIDTH]."""
        x = F.rms_norm(x, (DIM,)) @ self.qkv[layer]
        if layer == 0:   # the delta rule's q and k have unit norm
            q, k, v = x.unflatten(-1, (3, HEADS, WIDTH)).unbind(-3)
            return tuple(t.bfloat16().contiguous() for t in (F.normalize(q, dim=-1), F.normalize(k, dim=-1), v))
        return x.bfloat16().unflatten(-1, (3, HEADS, WIDTH)).unbind(-3)

    def gates(self, x):
        x = F.rms_norm(x, (DIM,))
        return -0.1 * F.softplus(x @ self.gate), torch.sigmoid(x @ self.beta).bfloat16()

    def add(self, x, o, layer):
        return x + o.float().flatten(-2) @ self.out[layer]

    def prompts(self, tokens, meta, cache=None, pages=None):
        """Logits of every token of packed prompts; their states go to pages."""
        x = self.embed[tokens]
        q, k, v = self.heads(x, 0)
        o, final, _ = gb.gdn_chunk_fwd(q, k, v, *self.gates(x), meta=meta, output_final_state=True)
        x = self.add(x, o, 0)
        q, k, v = self.heads(x, 1)
        o, _ = gb.gdn_linattn_fwd(q, k, v, self.decay, meta=meta, final_out=None if cache is None else cache[1],
                                  final_pages=pages)
        if cache is not None:
            gb.gdn_pages_copy(cache[:1], final[None], pages, torch.arange(len(pages), dtype=torch.int32, device=x.device))
        return self.add(x, o, 1) @ self.embed.T

    def step(self, tokens, cache, table):
        """Logits of one token for every slot; rows without a page are ignored."""
        x = self.embed[tokens]
        o = gb.gdn_recurrent_step(*self.heads(x, 0), *self.gates(x), cache[0], pages=table)
        x = self.add(x, o, 0)
        o = gb.gdn_linattn_step(*self.heads(x, 1), self.decay, cache[1], pages=table)
        return self.add(x, o, 1) @ self.embed.T


def decode(device="cuda", lengths=(37, 130, 5), beams=4, steps=12, seed=0):
    """Returns (largest difference of the last logits from the prompt pass
    over each beam's history, relative to their rms; pages in use)."""
    model = Model(device, seed)
    gen = torch.Generator(device).manual_seed(seed + 1)
    offs = [0]
    for n in lengths:
        offs.append(offs[-1] + n)
    prompt = torch.randint(0, VOCAB, (offs[-1],), generator=gen, device=device)
    groups, slots = len(lengths), len(lengths) * beams
    n_pages = slots + 7
    cache = torch.zeros(2, n_pages, HEADS, WIDTH, WIDTH, device=device)
    # one page for each prompt, scattered; the beams' first fork copies them
    free = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    first, spare = free[:groups].clone(), free[groups:].clone()
    logits = model.prompts(prompt, gb.make_meta(offs, offs[-1], device), cache, first)
    logits = logits[torch.tensor(offs[1:], device=device) - 1]
    table = torch.full((slots,), -1, dtype=torch.int32, device=device)
    table[::beams] = first
    base = torch.arange(0, slots, beams, device=device)
    score, token = F.log_softmax(logits, -1).topk(beams)          # [groups, beams]
    parent = base[:, None].expand(groups, beams)
    history = prompt.new_zeros(slots, 0)
    for _ in range(steps):
        table, spare = gb.gdn_pages_fork(cache, table, parent.flatten().to(torch.int32), spare=spare)
        spare = spare[:n_pages]                                    # what was free and not taken, then -1
        history = torch.cat([history[parent.flatten()] if history.shape[1] else history.new_zeros(slots, 0),
                             token.reshape(slots, 1)], 1)
        logits = model.step(token.flatten(), cache, table)
        total = score.reshape(slots, 1) + F.log_softmax(logits, -1)
        score, best = total.view(groups, beams * VOCAB).topk(beams)
        parent, token = base[:, None] + best // VOCAB, best % VOCAB
    table, count = gb.gdn_pages_compact(cache, table)
    # the same logits from whole histories, and once more from the moved pages
    seqs = [torch.cat([prompt[offs[s // beams]:offs[s // beams + 1]], history[s]]) for s in range(slots)]
    ends = torch.tensor([len(s) for s in seqs]).cumsum(0)
    whole = model.prompts(torch.cat(seqs), gb.make_meta([0] + ends.tolist(), int(ends[-1]), device))
    want = whole[ends.to(device) - 1]
    error = ((logits - want).abs().max() / want.square().mean().sqrt()).item()
    again = model.step(token.flatten(), cache, table)
    assert torch.isfinite(again).all() and int(count) == slots and int(table.max()) == slots - 1
    return error, int(count)


def train(device="cuda", steps=4, seed=0):
    """Losses of a few gradient steps of a linear-attention layer."""
    gen = torch.Generator(device).manual_seed(seed)
    x = torch.randn(2, 90, DIM, generator=gen, device=device)
    target = torch.randn(2, 90, HEADS, WIDTH, generator=gen, device=device)
    w = (torch.randn(DIM, 3 * DIM, generator=gen, device=device) / DIM ** 0.5).requires_grad_()
    decay = -0.5 * 0.4 ** torch.arange(HEADS, device=device).float()
    losses = []
    for _ in range(steps):
        q, k, v = (x @ w).unflatten(-1, (3, HEADS, WIDTH)).unbind(-3)
        o, _ = gb.LinearAttention.apply(q, k, v, decay)
        loss = F.mse_loss(o, target)
        grad, = torch.autograd.grad(loss, w)
        with torch.no_grad():
            w -= 0.5 * grad
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    error, pages = decode()
    print(f"last logits: max|difference|/rms = {error:.2e} from the prompt pass; {pages} pages in use")
    print("training losses:", ", ".join(f"{x:.4f}" for x in train()))
