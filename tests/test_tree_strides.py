"""Strides of q that the attention calls take: a row at least, for heads and for sequences, whatever the rows of a sequence."""
import pytest

from tests.test_drafts_refusals import TREE
from tests.test_ops_refusals import A, CFG, _accepted, _refused, m

ROW = 576


@pytest.mark.parametrize("sb,sh,good", [
    (ROW, ROW, True), (ROW, 16 * ROW, True), (4 * 16 * ROW, ROW, True), (3 * ROW, ROW, True), (ROW + 8, ROW + 8, True),
    ((1 << 38) - 8, (1 << 38) - 8, True), (ROW - 8, ROW, False), (ROW, ROW - 8, False), (0, ROW, False), (-ROW, ROW, False),
    (ROW + 4, ROW, False), (ROW, ROW + 4, False), (1 << 38, ROW, False), (ROW, 1 << 38, False)])
def test_strides(sb, sh, good):
    cfg = m.mla_config(**CFG)
    look = _accepted if good else _refused
    look(m.moe_mla_decode_tree, cfg, *{**TREE, "sb": sb, "sh": sh}.values())
    look(m.moe_mla_decode, cfg, A, sb, sh, A, A, A, A, A, A)
