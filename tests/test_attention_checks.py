"""Calls of the attention half that are refused before anything is launched or changed, without a GPU."""
import pytest
import torch

import ternary_weight_moe_forward_b200 as tw


class Recorder:
    """Stands for both halves of a layer: records that it was called."""

    def __init__(self, d_model, max_tokens):
        self.d_model, self.max_tokens, self.shape, self.handle, self.calls = d_model, max_tokens, self, 0, 0

    def decode(self, *args):
        self.calls += 1

    prompt = decode


def test_stack_refuses_more_tokens_than_its_layers_take_before_it_starts():
    first, second = Recorder(64, 100), Recorder(64, 8)
    stack = tw.DecoderStack([(first, first), (second, second)])
    resid = torch.zeros(9, 64)
    with pytest.raises(ValueError, match="9 tokens"):
        stack.decode(resid, None, None, None, None)
    with pytest.raises(ValueError, match="9 tokens"):
        stack.prompt(resid, None, None, None, 9)
    assert first.calls == 0 and second.calls == 0
