"""examples/beam_decoding.py: prompts, single tokens and the cache's pages run
together. Decoding and the prompt pass round the same activations to bf16 in
different orders (states, o), layer after layer: their logits agree to a few
bf16 roundings (2^-8 each) of values within a few rms, 5e-2 in all; a lost or
swapped state moves them by their own size."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("lengths,beams,steps", [((37, 130, 5), 4, 12), ((1, 64), 3, 5), ((70,), 1, 3)])
def test_decoding_equals_the_prompt_pass(lengths, beams, steps):
    import beam_decoding

    error, pages = beam_decoding.decode(lengths=lengths, beams=beams, steps=steps)
    assert error <= 5e-2 and pages == len(lengths) * beams


def test_training_lowers_the_loss():
    import beam_decoding

    losses = beam_decoding.train()
    assert all(b < a for a, b in zip(losses, losses[1:]))
