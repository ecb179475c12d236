"""The operators together: what a served hybrid model computes step by step is what it computes
on the whole sequences at once.

Tolerance: each layer's outputs are rounded to bf16 (2^-8 of a value) on both sides, at three
places of a layer (its input, the operator's output, the product); with 4 layers that is at most
2 * 3 * 4 * 2^-9 (an average rounding is half the largest) = 0.047 of the logits' norm if all of
them added up, and their square root of it, 0.0096, if they are independent; 2^-5 is in between.
"""

import pytest

from examples import hybrid_serving

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,rounds,seed", [(1, 3, 1), (6, 6, 0), (9, 7, 2)])
def test_served_and_whole_agree(batch, rounds, seed):
    tokens, drafted, far = hybrid_serving.serve(batch, rounds, seed)
    assert len(tokens) == batch
    assert far <= 2.0 ** -5
    assert drafted > 0 or batch == 1
