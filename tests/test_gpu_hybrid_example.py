"""The example stack runs the operators together: what its steps say of a
generated text, one prefill over the text has to say too.

Both forms round activations to bf16 (2^-8) at the same places but from sums in
another order; with two layers and unit-variance logits a log probability moves by
a few 2^-8 at most: 0.1 with 16-bit inputs.  E4M3 inputs turn such a difference
into a step of 2^-4 of single inputs now and then: 0.3."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("quant,tol", [("none", 0.1), ("row", 0.3)])
def test_steps_and_prefill_agree(libssu, quant, tol):
    import hybrid_stack
    seen, again, made, entropy = hybrid_stack.run(layers=2, new=12, lengths=(37, 140, 5), quant=quant)
    assert seen.shape == again.shape == made.shape == (3, 12)
    assert torch.isfinite(seen).all() and (seen <= 0).all() and (entropy > 0).all()
    assert (seen - again).abs().max() < tol
