"""The example's training falls and what it serves agrees with a pass over whole sequences."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_ffn_layers(dtype):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, EXAMPLES)
    try:
        import attention_ffn_layers as example
    finally:
        sys.path.remove(EXAMPLES)
    losses, error, live = example.main(["--dtype", dtype])
    assert all(b < a for a, b in zip(losses, losses[4::4])) and losses[-1] < 0.5 * losses[0]
    # Both passes round the same values to the type at some ten places a layer, where they may go to
    # neighbours; each such place moves a logit by at most a few of its units at the end of two layers.
    # In fp32 sums of up to 512 products in other orders come to it: about 512 units more.
    assert error <= (2.0 ** -8 * 20 if dtype == "bf16" else 2.0 ** -24 * 20 * 512)
    # rows 1, 3 and three beams are left; the beams share the pages that they had in full
    n1, n3, beam = 47 + 20, 16 + 20, 90 + 20
    shared = beam // example.PAGE
    pages = lambda n: -(-n // example.PAGE)
    assert live == pages(n1) + pages(n3) + shared + 3
