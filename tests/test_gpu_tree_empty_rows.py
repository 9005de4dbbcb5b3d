"""moe_mla_decode_tree: rows that see nothing are zero, with lse = -inf, also where the sequence's cached rows are not finite.

The products run over all cached rows of a sequence, and 0 times NaN or infinity is NaN: such rows are not what the
product gave.
"""
import pytest
import torch

from tests.test_gpu_tree import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def spoil(s, b, j, value):
    """Cached row j of sequence b, all columns or one latent column of it."""
    page = s.att.page_size
    row = s.cache[s.table[b, j // page], j % page]
    if value == "column":
        row[7] = float("nan")
    else:
        row.fill_(value)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), "column"])
@pytest.mark.parametrize("H,latent,page", [(3, 512, 64), (4, 256, 8), (8, 384, 16), (20, 512, 24), (128, 512, 64)])
@pytest.mark.parametrize("long", [1, 40])
def test_rows_that_see_nothing(lib, H, latent, page, value, long):
    """One piece a sequence, and sequences cut into many that the join adds."""
    n = 6
    lens = [100 * long, 6, 130 * long, 4, 77, 1]
    drafts = [2, 6, 0, 4, 5, 1]
    masks = [[(2 << i) - 1 for i in range(n)] for _ in lens]
    masks[1] = [0, 1, 0, 3, 0, 32]                          # no prefix: rows 0, 2 and 4 see nothing
    masks[3] = [0] * n
    masks[5] = [0] * n
    s = Setup(lens, n, H, latent, page=page, drafts=drafts, masks=masks, seed=60)
    clean = [t.clone() for t in s.run()]
    s.check(*clean)
    for b, j in ((0, 50), (0, 99 * long), (1, 5), (2, 70), (3, 0), (4, 76), (5, 0)):
        spoil(s, b, j, value)
    out, lse = s.run()
    for b, m in enumerate(drafts):
        for i in range(n):
            if i >= m or (lens[b] == m and masks[b][i] & ((1 << m) - 1) == 0):
                assert (out[b, i] == 0).all() and (lse[b, i] == -torch.inf).all(), (b, i)
            else:
                assert not torch.equal(out[b, i], clean[0][b, i])         # and the others are told of it
    # what the spoiled rows do not reach: a sequence that holds none
    s.cache.copy_(torch.nan_to_num(s.cache, nan=1.0, posinf=1.0, neginf=1.0))
    spoil(s, 0, 50, value)
    other, olse = s.run()
    assert torch.isfinite(other[2:].float()).all() and torch.isfinite(other[1].float()).all()
