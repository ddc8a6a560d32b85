"""The LM head's number of tokens is refused when the head has no such rows: as
a slice it would silently score another vocabulary (no GPU)."""
import pytest
import torch

from gemm_epilogue_fusion_gb300 import chain


@pytest.mark.parametrize("vocab", [0, -3, 305, 1 << 40])
def test_a_vocabulary_that_the_head_does_not_have(vocab):
    bf = torch.bfloat16
    h, W, t = torch.zeros(2, 128, dtype=bf), torch.zeros(304, 128, dtype=bf), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="vocab"):
        chain.head_logprobs(h, torch.zeros(2, 1), W, 1e-5, t, vocab=vocab)
    fwd = {"logits": torch.zeros(2, 304, dtype=bf), "lse": torch.zeros(2), "entropy": torch.zeros(2), "r": torch.zeros(2)}
    with pytest.raises(ValueError, match="vocab"):
        chain.head_logprobs_backward(h, W, torch.ones(128), fwd, t, vocab=vocab)
