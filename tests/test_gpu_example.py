"""The decoder-block example: the new operators with the MoE layer, served and trained.

The block's activations are rounded to bf16 at about ten places (2^-9 relative
on average each), so its stream is held to 2e-2 of the 64-bit one, and the
norm's gradient, one rounding, to 4e-3.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_decoder_block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ex = _example()
    assert ex.serve(3, verbose=False) < 2e-2
    assert ex.train(verbose=False) < 4e-3
