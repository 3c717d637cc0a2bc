"""The operators together, as examples/sparse_layer.py runs them: prompts into
the caches and through the expanded attention, decode steps over picked keys."""
import os
import sys

import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("lens,steps", [((70, 1, 2500), 2), ((63, 64, 65, 2047), 3)])
def test_layer(lens, steps):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_layer
    log("layer", lens, steps)
    forms, picks, share = sparse_layer.run(lens, steps, seed=len(lens))
    # The forms differ by roundings to bfloat16 (2^-9 relative each, at random): of the keys, the values, the absorbed
    # queries, the weights twice, both outputs.  The logits, of size 1, move by sqrt(3) of these, the outputs by less
    # than sqrt(16) in all.
    assert forms < 4 * 2 ** -8, forms
    # the same numbers in another order: weights and outputs rounded to bfloat16
    assert picks < 2 ** -7, picks
    for n, s in zip(lens, share):
        assert s == min(1.0, 2048 / (n + steps)), (n, s)
