"""Arguments of the norm and latent-attention entry points at the ends of their ranges, checked on the host.

As in the tests of refusals, argument checks run before the device check: without a GPU a good call gets as far
as MOE_ERR_UNSUPPORTED_ARCH, and with one only the bad calls are made.
"""
import pytest

from tests.test_ops_refusals import APPEND, CFG, DECODE, _accepted, _refused, m


@pytest.mark.parametrize("scale", [2.4e38, 2.99e38, 3.4e38])
def test_scale_past_the_range_of_its_powers_of_two(scale):
    """softmax_scale * log2(e) is infinite there, and a score of 0 would come out as 0 * inf."""
    cfg = m.mla_config(**{**CFG, "softmax_scale": scale})
    _refused(m.moe_mla_workspace_size, cfg)
    _refused(m.moe_mla_decode, cfg, *DECODE.values())
    _refused(m.moe_mla_append, cfg, *APPEND.values())


@pytest.mark.parametrize("scale", [2.35e38, 1.0, 1e-38])
def test_scales_in_range(scale):
    cfg = m.mla_config(**{**CFG, "softmax_scale": scale})
    assert m.moe_mla_workspace_size(cfg) > 0
    _accepted(m.moe_mla_decode, cfg, *DECODE.values())
