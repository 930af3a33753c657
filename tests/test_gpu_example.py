"""The hybrid-layer example: prompts, single tokens on cached states and a
training step through the public functions together.

Bar: both ways round activations to bf16 (2^-9 relative each) at the same dozen
places of two layers, and the prefill's recurrence is held to 5e-3 relative, so
their difference stays below 3e-2 relative."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_single_tokens_continue_prompts_and_training_lowers_the_loss():
    import hybrid_layers
    err, losses = hybrid_layers.main()
    assert err <= 3e-2
    assert losses[-1] < losses[0]
