"""The attention calls on the longest sequence that the library takes, whose last tile ends at 2^31 tokens.

The cache has two pages, the block table hundreds of entries that share the first one. All of its rows have scores
600 below the last tokens' (e^-600 is 0 in 64 bits too), so those alone make the output, and it is known exactly.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F = torch.float64
PAGE = 8 * 43 * 113 * 127                                   # 435 of them are 2^31 - 8 tokens
PAGES = 435


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


@pytest.mark.parametrize("latent,H,n", [(128, 4, 5), (256, 24, 3)])   # single CTAs, and 72 rows on pairs
@pytest.mark.parametrize("short", [0, 3, 61])
def test_last_tile(lib, latent, H, n, short):
    from moe_layer_dsv3_gb300.attention import LatentAttention
    rope, scale = 8, 0.0625
    length = PAGE * PAGES - short
    assert length + short == 2 ** 31 - 8
    g = torch.Generator(device="cuda").manual_seed(short + H)
    row = latent + rope
    cache = torch.zeros(2, PAGE, row, dtype=torch.bfloat16, device="cuda")
    cache[:, :, latent] = -96.0                             # with q's 100: a score of -600
    live = 40                                               # the last tokens, the drafted ones among them
    last = torch.randn(live, row, generator=g, device="cuda").to(torch.bfloat16)
    last[:, latent] = 0.0
    end = PAGE - short
    cache[1, end - live:end] = last
    cache[1, end:] = float("nan")
    table = torch.zeros(1, PAGES, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    q = torch.randn(1, n, H, row, generator=g, device="cuda").to(torch.bfloat16)
    q[..., latent] = 100.0
    masks = [(1 << i) | (i & 1) for i in range(n)]          # itself and, every other one, the first
    tree = torch.tensor([masks], dtype=torch.int64, device="cuda")
    att = LatentAttention(1, H, latent, rope, PAGE, 2, PAGES, scale, drafts=n)
    out = att.decode_tree(q, cache, table, lens, tree=tree)
    one = att.decode(q[:, -1], cache, table, lens)
    torch.cuda.synchronize()
    assert att.status() == (0, 0)
    k = last.to(F)
    for i in range(n + 1):
        mask = masks[i] if i < n else (1 << n) - 1          # (the last one, by moe_mla_decode: it sees all)
        got, lse = (out[0, i], att.tree_lse[0, i]) if i < n else (one[0], att.lse[0])
        seen = list(range(live - n)) + [live - n + j for j in range(n) if mask >> j & 1]
        ks = k[torch.tensor(seen, device="cuda")]
        s = q[0, min(i, n - 1)].to(F) @ ks.T * scale
        p = torch.softmax(s, 1)
        o = p @ ks[:, :latent]
        # the roundings of out and P (2^-8 each), and scores summed over latent + rope products, 2^-23 of the magnitudes each
        ds = scale * row * 2.0 ** -23 * (q[0, min(i, n - 1)].to(F).abs() @ ks.abs().T) + s.abs() * 2.0 ** -21
        spread = p @ ks[:, :latent].abs() + o.abs()
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds.amax(1, keepdim=True) + 2.0 ** -21) * spread * 1.01 + 2.0 ** -20 * spread
        assert ((got.to(F) - o).abs() <= tol).all(), i
        ref = torch.logsumexp(s, 1)
        assert ((lse.to(F) - ref).abs() <= ds.amax(1) + 2.0 ** -19 * (1 + ref.abs())).all(), i
