"""The example of the recurrent-layer operators: its training step descends and its
decode steps continue its prefill."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_training_descends():
    import recurrent_layer as ex
    stack = ex.Stack()
    losses, norms = ex.train(stack)
    assert losses[-1] < 0.7 * losses[0]
    assert all(n > 0 and n < float("inf") for n in norms)


@pytest.mark.gpu
def test_decode_continues_the_prefill():
    """The states are fp32 and the two recurrences round alike; what differs are the
    bf16 products of other shapes (2^-8 of a value each, six of them one after the
    other) and an 8-bit step (2^-4 of a value) where such a difference crosses one."""
    import recurrent_layer as ex
    got, want = ex.serve(ex.Stack())
    assert float((got - want).abs().max() / want.abs().max()) <= 6 * 2.0 ** -8 + 2.0 ** -4


def test_example_imports_without_a_gpu():
    import recurrent_layer as ex
    assert ex.Block and ex.Stack and callable(ex.main)
