"""moe_mla_decode_tree against the formula in 64 bits.

Tolerances as for moe_mla_decode, a row at a time: out is rounded to bf16 (2^-8);
P is rounded to bf16 and normalised by the sum of the rounded values, so the
error it leaves is sum_j p_j e_j (v_j - out) with |e_j| <= 2^-8; a score is an fp32
sum of latent + rope products, each addition off by 2^-23 of the sum of magnitudes at
most (the tensor core may truncate), which moves p_j by that much. The lse
carries the scores' error alone.
"""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

F = torch.float64
U = 2.0 ** -8


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def random_tree(r, n):
    seen = []
    for i in range(n):
        parent = r.randint(max(-1, i - 3), i - 1)
        seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
    return seen


def words(masks):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64, device="cuda")


class Setup:
    def __init__(self, lens, n, H, latent=512, rope=64, page=64, drafts=None, seed=0, masks=None, qgain=1.0, fill=float("nan")):
        from moe_layer_dsv3_gb300.attention import LatentAttention
        r = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.n, self.H, self.latent, self.rope = list(lens), n, H, latent, rope
        self.drafts = [min(n, x) for x in lens] if drafts is None else list(drafts)
        need = [-(-x // page) for x in lens]
        width, pool = max(1, max(need, default=1)) + 1, sum(need) + 2
        order = list(range(pool))
        r.shuffle(order)
        cache = torch.full((pool, page, latent + rope), fill, dtype=torch.bfloat16, device="cuda")   # what a freed page may hold
        table = torch.full((len(lens), width), -12345, dtype=torch.int32)
        self.rows = []
        at = 0
        for b, k in enumerate(need):
            rows = torch.randn(lens[b], latent + rope, generator=g, device="cuda").to(torch.bfloat16)
            for i in range(k):
                table[b, i] = order[at + i]
                part = rows[i * page:(i + 1) * page]
                cache[order[at + i], :len(part)] = part
            at += k
            self.rows.append(rows)
        self.cache, self.table = cache, table.cuda()
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.drafts_t = torch.tensor(self.drafts, dtype=torch.int32, device="cuda")
        self.masks = [random_tree(r, n) for _ in lens] if masks is None else masks
        self.tree = words(self.masks) if len(lens) else torch.zeros(0, n, dtype=torch.int64, device="cuda")
        self.q = (qgain * torch.randn(len(lens), n, H, latent + rope, generator=g, device="cuda")).to(torch.bfloat16)
        self.scale = (128 + rope) ** -0.5
        self.att = LatentAttention(len(lens), H, latent, rope, page, pool, width, self.scale, drafts=n)
        self.att.tree_out.fill_(7.0)
        self.att.tree_lse.fill_(7.0)

    def run(self, q=None, **kw):
        kw = {"tree": self.tree, "drafts": self.drafts_t, **kw}
        self.att.decode_tree(self.q if q is None else q, self.cache, self.table, self.lens_t, **kw)
        torch.cuda.synchronize()
        assert self.att.status() == (0, 0)
        return self.att.tree_out, self.att.tree_lse

    def check(self, out=None, lse=None):
        if out is None:
            out, lse = self.run()
        for b, (L, m) in enumerate(zip(self.lens, self.drafts)):
            k = self.rows[b].to(F)
            for i in range(self.n):
                seen = list(range(L - m)) + [L - m + j for j in range(m) if self.masks[b][i] >> j & 1] if i < m else []
                if not seen:
                    assert (out[b, i] == 0).all() and (lse[b, i] == -torch.inf).all()
                    continue
                ks = k if len(seen) == L else k[torch.tensor(seen, device="cuda")]
                q = self.q[b, i].to(F)
                s = q @ ks.T * self.scale
                ds = self.scale * (self.latent + self.rope) * 2.0 ** -23 * (q.abs() @ ks.abs().T) + s.abs() * 2.0 ** -21
                p = torch.softmax(s, 1)
                v = ks[:, :self.latent]
                o = p @ v
                # relative error of a p: its own rounding and its score's; the exponential's 2^-21
                rel = U + 2 * ds.amax(1, keepdim=True) + 2.0 ** -21
                spread = p @ v.abs() + o.abs()
                tol = U * o.abs() + rel * spread * 1.01 + 2.0 ** -20 * spread
                bad = (out[b, i].to(F) - o).abs() > tol
                assert not bad.any(), (b, i, ((out[b, i].to(F) - o).abs() / tol).max().item())
                # the mean error is far below the bound of each
                assert (out[b, i].to(F) - o).norm() <= 1.5 * U * o.norm() + 0.5 * U * spread.norm() / max(1.0, len(seen)) ** 0.5
                ref = torch.logsumexp(s, 1)
                assert ((lse[b, i].to(F) - ref).abs() <= ds.amax(1) + 2.0 ** -19 * (1 + ref.abs())).all()


CASES = [
    # lens, n, H, latent, rope, page: rows per sequence n * H around every form's edges
    ([1], 1, 1, 512, 64, 64), ([5, 130, 64], 4, 4, 512, 64, 64), ([200, 3, 65, 63], 3, 5, 512, 64, 24),
    ([70, 129], 8, 2, 512, 64, 64), ([90, 1, 300], 2, 16, 512, 64, 16), ([77, 500], 3, 21, 512, 64, 64),
    ([128, 127], 4, 16, 512, 64, 64), ([129, 257], 5, 13, 512, 64, 8), ([300, 64], 6, 20, 512, 64, 48),
    ([191, 400], 8, 16, 512, 64, 64), ([33, 260], 7, 20, 512, 64, 24), ([150], 3, 128, 512, 64, 64),
    ([300, 70], 2, 128, 512, 64, 128), ([100, 65], 64, 3, 512, 64, 64), ([64, 200], 64, 1, 512, 64, 16),
    ([140, 10], 9, 16, 256, 64, 64), ([140, 300], 5, 40, 256, 32, 24), ([130, 64], 5, 9, 128, 64, 64),
    ([131, 300], 11, 12, 128, 32, 8), ([90, 257], 7, 33, 384, 64, 64), ([66, 64], 3, 17, 384, 8, 16),
    ([2000], 4, 16, 512, 64, 64), ([1500, 40], 16, 8, 512, 64, 64), ([700] * 9 + [3] * 4, 7, 20, 512, 64, 24),
]


@pytest.mark.parametrize("lens,n,H,latent,rope,page", CASES)
def test_trees(lib, lens, n, H, latent, rope, page):
    Setup(lens, n, H, latent, rope, page, seed=sum(lens) + n).check()


@pytest.mark.parametrize("H,latent", [(4, 512), (16, 512), (128, 512), (12, 384)])
def test_fewer_drafts_empty_sequences_and_empty_masks(lib, H, latent):
    n = 6
    lens = [100, 0, 6, 3, 64, 70, 128, 1, 0]
    drafts = [2, 0, 6, 3, 0, 6, 5, 1, 0]
    r = random.Random(1)
    masks = [[r.getrandbits(64) for _ in range(n)] for _ in lens]      # any bits, those past the drafted ones too
    masks[2] = [0] * n                                                 # no prefix and nothing of the tree: rows that see nothing
    masks[5][3] = 0                                                    # the prefix alone
    Setup(lens, n, H, latent, drafts=drafts, masks=masks, seed=2).check()


@pytest.mark.parametrize("n,H,latent", [(5, 8, 512), (5, 20, 512), (3, 24, 384)])
def test_no_mask_is_a_chain(lib, n, H, latent):
    lens = [130, 2, 77, 0]
    chain = [[(2 << i) - 1 for i in range(n)] for _ in lens]
    s = Setup(lens, n, H, latent, masks=chain, drafts=[min(n, x) for x in lens], seed=3)
    s.check(*s.run(tree=None))


def test_all_drafted(lib):
    lens = [5, 70, 0]
    s = Setup(lens, 5, 4, masks=[[(1 << 5) - 1] * 5] * 3, seed=4)
    s.check(*s.run(drafts=None))


@pytest.mark.parametrize("H,latent", [(1, 512), (16, 512), (64, 512), (100, 512), (48, 384), (128, 256)])
def test_one_drafted_token_is_decode(lib, H, latent):
    """The same bytes: the same products in the same order."""
    s = Setup([300, 0, 64, 1, 1000], 1, H, latent, masks=[[1]] * 5, seed=5)
    out, lse = s.run()
    o2 = s.att.decode(s.q[:, 0].contiguous(), s.cache, s.table, s.lens_t)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 0], o2) and torch.equal(lse[:, 0], s.att.lse)


def test_pitched_queries(lib):
    s = Setup([100, 40], 3, 5, seed=6)
    wide = torch.zeros(2, 3 * 5 + 2, s.latent + s.rope + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, :15, :s.latent + s.rope] = s.q.flatten(1, 2)
    q = wide.as_strided((2, 3, 5, s.latent + s.rope), (wide.stride(0), 5 * wide.stride(1), wide.stride(1), 1))
    s.check(*s.run(q=q))


def test_large_scores(lib):
    """References that move in every tile, in rows that mask different tokens."""
    Setup([400, 70], 6, 16, qgain=30.0, seed=7).check()
    Setup([400, 70], 6, 3, qgain=30.0, seed=7).check()


def test_bad_counts_are_clamped_and_told(lib):
    s = Setup([100, 3, 0], 4, 4, drafts=[4, 3, 0], seed=8)
    given = torch.tensor([9, 4, 1], dtype=torch.int32, device="cuda")
    s.att.decode_tree(s.q, s.cache, s.table, s.lens_t, tree=s.tree, drafts=given)
    torch.cuda.synchronize()
    assert s.att.status()[0] == lib.MOE_ERR_BOUNDS
    s.check(s.att.tree_out, s.att.tree_lse)
    given[0] = -1
    s.drafts[0] = 0
    s.att.decode_tree(s.q, s.cache, s.table, s.lens_t, tree=s.tree, drafts=given)
    torch.cuda.synchronize()
    assert s.att.status()[0] == lib.MOE_ERR_BOUNDS
    s.check(s.att.tree_out, s.att.tree_lse)


def test_captured_and_replayed(lib):
    """A graph takes the lengths, counts and masks of the time."""
    s = Setup([200, 90, 64], 5, 16, seed=9)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call = lambda: s.att.decode_tree(s.q, s.cache, s.table, s.lens_t, tree=s.tree, drafts=s.drafts_t, stream=st.cuda_stream)
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st, capture_error_mode="thread_local"):
        call()
    for lens, drafts in (([200, 90, 64], [5, 5, 5]), ([150, 7, 0], [2, 5, 0]), ([5, 90, 63], [5, 0, 1])):
        s.lens, s.drafts = lens, drafts
        s.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        s.drafts_t.copy_(torch.tensor(drafts, dtype=torch.int32))
        s.masks = [random_tree(random.Random(sum(lens)), 5) for _ in lens]
        s.tree.copy_(words(s.masks))
        s.rows = [r[:n] for r, n in zip(s.rows, lens)] if all(len(r) >= n for r, n in zip(s.rows, lens)) else s.rows
        full = s.rows
        g.replay()
        torch.cuda.synchronize()
        s.rows = [r[:n] for r, n in zip(full, lens)]
        s.check(s.att.tree_out, s.att.tree_lse)
        s.rows = Setup([200, 90, 64], 5, 16, seed=9).rows
    assert s.att.status() == (0, 0)


def test_pages_past_32_bits(lib):
    """Drafted tokens whose pages lie past 2^32 bytes and 2^31 elements of the cache."""
    from moe_layer_dsv3_gb300.attention import LatentAttention
    latent, rope, page = 512, 64, 64
    pool = 2 ** 31 // (page * (latent + rope)) + 40        # 4.3 GB
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.empty(pool, page, latent + rope, dtype=torch.bfloat16, device="cuda")
    lens, n, H = [130, 64, 200], 3, 16
    table = torch.full((3, 5), -1, dtype=torch.int32)
    rows = []
    at = pool - 1
    for b, L in enumerate(lens):
        r = torch.randn(L, latent + rope, generator=g, device="cuda").to(torch.bfloat16)
        for i in range(-(-L // page)):
            table[b, i] = at
            part = r[i * page:(i + 1) * page]
            cache[at].fill_(float("nan"))
            cache[at, :len(part)] = part
            at -= 1
        rows.append(r)
    s = Setup.__new__(Setup)
    s.lens, s.n, s.H, s.latent, s.rope, s.scale = lens, n, H, latent, rope, 192 ** -0.5
    s.drafts, s.masks, s.rows = [3, 2, 3], [[1, 3, 5]] * 3, rows
    s.cache, s.table, s.tree = cache, table.cuda(), words(s.masks)
    s.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s.drafts_t = torch.tensor(s.drafts, dtype=torch.int32, device="cuda")
    s.q = torch.randn(3, n, H, latent + rope, generator=g, device="cuda").to(torch.bfloat16)
    s.att = LatentAttention(3, H, latent, rope, page, pool, 5, s.scale, drafts=n)
    s.check()


def test_many_row_groups(lib):
    """The most rows a sequence can have (64 tokens of 128 heads: 64 groups of 128), and groups that are not full."""
    Setup([70, 66], 64, 128, seed=10).check()
    Setup([140], 43, 3, seed=11).check()                   # 129 rows: groups of 65 and 64
    Setup([90, 200], 37, 7, seed=12).check()               # 259 rows: 87, 87 and 85
    Setup([90, 200], 13, 5, latent=384, seed=13).check()   # 65 rows in groups of up to 64


def test_refused_tensors(lib):
    s = Setup([70, 66], 4, 4, seed=14)
    f = s.att.decode_tree
    bad = lambda *a, **k: pytest.raises(lib.MoeError, f, *a, **k)
    ok = (s.q, s.cache, s.table, s.lens_t)
    bad(s.q.float(), *ok[1:])
    bad(s.q[:1], *ok[1:])
    bad(s.q[..., :512], *ok[1:])
    bad(s.q.flatten(1, 2), *ok[1:])
    bad(s.q.transpose(1, 2).contiguous().transpose(1, 2), *ok[1:])         # a token's heads apart, tokens between them
    bad(*ok, tree=s.tree.int())
    bad(*ok, tree=s.tree[:, :3])
    bad(*ok, drafts=s.drafts_t.long())
    bad(*ok, out=torch.empty(2, 4, 4, 512, device="cuda"))
    bad(torch.zeros(2, 5, 4, 576, dtype=torch.bfloat16, device="cuda"), *ok[1:])      # more drafted tokens than the buffers hold
    with pytest.raises(lib.MoeError):
        s.att.decode_tree(torch.zeros(2, 65, 4, 576, dtype=torch.bfloat16, device="cuda"), *ok[1:],
                          out=torch.empty(2, 65, 4, 512, dtype=torch.bfloat16, device="cuda"),
                          lse=torch.empty(2, 65, 4, device="cuda"))


@pytest.mark.parametrize("lens,n,H,latent,page", [
    ([30000], 3, 16, 512, 64), ([26000], 4, 32, 256, 64), ([12000, 3, 9000], 5, 7, 384, 16), ([700 + 13 * i for i in range(40)], 7, 18, 512, 64),
    ([9000 + i for i in range(7)], 2, 100, 512, 128), ([20001], 9, 40, 512, 48)])
def test_long_lists(lib, lens, n, H, latent, page):
    """Sequences cut into long lists of pieces, and many short ones, in one and in several row groups."""
    Setup(lens, n, H, latent, page=page, seed=15).check()
