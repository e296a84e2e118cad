"""The example blocks run the operators together: training lowers the loss,
and tokens served one by one after padded prompts match the sequences run
whole.  The bf16 projections and the scan's bf16 products differ between the
two ways by some roundings of 2^-8 each: 2e-2."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["HeadBlock", "ChannelBlock"])
def test_block_trains_and_serves(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_ssd_forward_gb300 import build
    build.build()
    import blocks
    torch.manual_seed(0)
    block = getattr(blocks, name)()
    losses = blocks.train(block, steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert blocks.serve(block) < 2e-2
