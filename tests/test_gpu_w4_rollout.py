"""GPU test of the example that runs the 4-bit head, the log probabilities from logits and
their gradient together: the rollout's and the training side's log probabilities are equal
bit for bit, chosen tokens are allowed, and the gradient is that of the loss."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("hidden,vocab", [(256, 5003), (4096, 32768)])
def test_rollout_and_training_agree(hidden, vocab):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w4_rollout
    r = w4_rollout.run(sequences=3, steps=24, hidden=hidden, vocab=vocab, seed=3)
    s = r["stats"]
    assert s["n_valid"] == 72 and s["n_bit_mismatch"] == 0 and s["max_abs"] == 0
    rows = torch.arange(72, device="cuda")
    assert bool(r["keep"][rows, r["tokens"].long()].all())
    assert bool((r["grad_z"][~r["keep"]] == 0).all())
    # every row's gradient sums to 0: the softmax does not change when all logits move
    # together (fp32 sums of `vocab` terms of at most 1/72 in all: far below 1e-6)
    assert float(r["grad_z"].double().sum(1).abs().max()) < 1e-6
    assert bool(torch.isfinite(r["grad_h"]).all()) and float(r["grad_h"].float().norm()) > 0
