"""Arguments of the norm and latent-attention entry points at the ends of their ranges, checked on the host.

As in the tests of refusals, argument checks run before the device check: without a GPU a good call gets as far
as MOE_ERR_UNSUPPORTED_ARCH, and with one only the bad calls are made.
"""
import pytest

from tests.test_ops_refusals import APPEND, CFG, DECODE, NORM, NORM_BWD, _accepted, _refused, m


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


WIDE = [1 << 31, (1 << 32) + 4, (1 << 40) + 256]      # the low 32 bits of the last two are ordinary sizes


@pytest.mark.parametrize("v", WIDE)
def test_sizes_past_32_bits_are_not_cut(v):
    for k in ("T", "d"):
        _refused(m.moe_add_rmsnorm, *{**NORM, k: v}.values())
        _refused(m.moe_add_rmsnorm_backward, *{**NORM_BWD, k: v}.values())
    _refused(m.moe_add_rmsnorm_backward_workspace, v, 256)
    for k in ("n", "ld", "max_pos"):
        _refused(m.moe_mla_append, m.mla_config(**CFG), *{**APPEND, k: v}.values())
    for k in ("batch", "heads", "latent", "rope", "page_size", "num_pages", "max_pages"):
        _refused(lambda: m.mla_config(**{**CFG, k: v}))
