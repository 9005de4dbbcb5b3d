"""LatentAttention.decode_tree: calls of fewer drafted tokens than its own outputs hold."""
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


@pytest.mark.parametrize("H,latent", [(4, 512), (20, 512), (16, 384)])
def test_fewer_tokens_than_the_buffers(lib, H, latent):
    """Calls of every size in turn on one object: the bytes of a call that brings its outputs, and nothing behind them."""
    from moe_layer_dsv3_gb300.attention import LatentAttention
    lens = [70, 200, 64]
    own = None
    for n in (5, 8, 1, 7):
        s = Setup(lens, n, H, latent, drafts=[n, max(1, n - 1), n], seed=20 + n)
        want, wlse = (t.clone() for t in s.run())
        s.check(want, wlse)
        if own is None:
            c = s.att.cfg
            own = LatentAttention(3, H, latent, s.rope, c.page_size, c.num_pages, c.max_pages, s.scale, drafts=8)
        own.tree_out.fill_(7.0)
        own.tree_lse.fill_(7.0)
        out = own.decode_tree(s.q, s.cache, s.table, s.lens_t, tree=s.tree, drafts=s.drafts_t)
        torch.cuda.synchronize()
        assert own.status() == (0, 0)
        assert out.shape == want.shape and out.data_ptr() == own.tree_out.data_ptr() and torch.equal(out, want)
        flat = own.tree_lse.view(-1)
        assert torch.equal(flat[:wlse.numel()].view(wlse.shape), wlse)
        assert (flat[wlse.numel():] == 7.0).all() and (own.tree_out.view(-1)[want.numel():] == 7.0).all()


def test_more_tokens_than_the_buffers_are_refused(lib):
    s = Setup([70, 66], 4, 4, seed=30)
    q = torch.zeros(2, 5, 4, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(2, 5, 4, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 5, 4, device="cuda")
    for kw in (dict(), dict(out=out), dict(lse=lse)):
        with pytest.raises(lib.MoeError) as e:
            s.att.decode_tree(q, s.cache, s.table, s.lens_t, **kw)
        assert e.value.code == lib.MOE_ERR_INVALID_ARG
    s.att.decode_tree(q, s.cache, s.table, s.lens_t, out=out, lse=lse)      # outputs of the caller's may be larger
    torch.cuda.synchronize()
    assert s.att.status() == (0, 0)


def test_no_sequences(lib):
    from moe_layer_dsv3_gb300.attention import LatentAttention
    att = LatentAttention(0, 4, 512, 64, 64, 1, 1, 0.1, drafts=8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    out = att.decode_tree(torch.zeros(0, 5, 4, 576, dtype=torch.bfloat16, device="cuda"), att.new_cache(), i32(0, 1), i32(0))
    assert out.shape == (0, 5, 4, 512)


@pytest.mark.parametrize("H,latent", [(4, 512), (20, 512), (16, 384)])
def test_sequences_that_share_rows_of_q(lib, H, latent):
    """A batch stride of one head: sequence b's rows are those of the first one, b heads on."""
    lens, n = [70, 200, 64, 3], 3
    s = Setup(lens, n, H, latent, seed=31)
    row = latent + s.rope
    rows = torch.randn(n * H + len(lens) - 1, row, device="cuda").to(torch.bfloat16)
    s.q = rows.as_strided((len(lens), n, H, row), (row, H * row, row, 1))
    s.check()


@pytest.mark.parametrize("H,latent", [(4, 512), (20, 512), (16, 384)])
def test_heads_farther_apart_than_sequences(lib, H, latent):
    """q with the sequences inside: a batch stride of one row, heads a batch apart."""
    lens, n = [70, 200, 64, 3, 1], 3
    s = Setup(lens, n, H, latent, seed=32)
    row, B = latent + s.rope, len(lens)
    inner = s.q.flatten(1, 2).transpose(0, 1).contiguous()                  # [n * H][B][row]
    q = inner.as_strided((B, n, H, row), (row, H * B * row, B * row, 1))
    assert torch.equal(q, s.q)
    s.check(*s.run(q=q))
    one = Setup(lens, 1, H, latent, masks=[[1]] * B, seed=33)
    out, lse = one.run()
    inner = one.q[:, 0].transpose(0, 1).contiguous()
    got = one.att.decode(inner.transpose(0, 1), one.cache, one.table, one.lens_t)
    torch.cuda.synchronize()
    assert torch.equal(got, out[:, 0]) and torch.equal(one.att.lse, lse[:, 0])
