"""moe_mla_append and moe_mla_decode against the formulas in 64 bits.

Tolerances of decode, a row at a time, from its roundings: out is rounded to
bf16 (2^-8); P is rounded to bf16 and normalised by the sum of the rounded
values, so the error it leaves is sum_j p_j e_j (v_j - out) with |e_j| <= 2^-8;
a score is an fp32 sum of latent + rope products, each addition off by 2^-23 of
the partial sum at most (the tensor core may truncate), which moves p_j by that
much. The lse carries the scores' error alone.
"""
import numpy as np
import pytest
import torch

from tests.helpers import np_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


class Setup:
    def __init__(self, lens, H, latent=512, rope=64, page=64, seed=0, spare=2, num_pages=None, fill=float("nan"), qgain=1.0):
        from moe_layer_dsv3_gb300.attention import LatentAttention
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_l, self.H, self.latent, self.rope, self.page = list(lens), H, latent, rope, page
        need = [-(-n // page) for n in lens]
        width = max(1, max(need, default=1)) + 1
        pool = num_pages or sum(need) + spare
        # the pages at the pool's end, shuffled
        perm = pool - 1 - torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed))
        table = torch.full((len(lens), width), -12345, dtype=torch.int32)
        cache = torch.empty(pool, page, latent + rope, dtype=torch.bfloat16, device="cuda")
        if num_pages is None:
            cache.fill_(fill)                  # whatever a freed page may hold
        at = 0
        for b, k in enumerate(need):
            pages = perm[at:at + k]
            table[b, :k] = pages.to(torch.int32)
            rows = torch.randn(lens[b], latent + rope, generator=g, device="cuda").to(torch.bfloat16)
            for i, p in enumerate(pages.tolist()):
                cache[p].fill_(fill)
                part = rows[i * page:(i + 1) * page]
                cache[p, :part.shape[0]] = part
            at += k
        self.cache, self.table = cache, table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.scale = (128 + rope) ** -0.5
        self.q = (qgain * torch.randn(len(lens), H, latent + rope, generator=g, device="cuda")).to(torch.bfloat16)
        self.att = LatentAttention(len(lens), H, latent, rope, page, pool, width, self.scale)

    def run(self, **kw):
        self.att.out.fill_(7.0)
        self.att.lse.fill_(7.0)
        self.att.decode(self.q, self.cache, self.table, self.lens, **kw)
        torch.cuda.synchronize()
        self.att.check_status()
        return self

    def rows(self, b):
        n = self.lens_l[b]
        pages = self.table[b, :-(-n // self.page)].long()
        return self.cache[pages].reshape(-1, self.latent + self.rope)[:n].double()

    def check(self):
        for b, n in enumerate(self.lens_l):
            out, lse = self.att.out[b].double(), self.att.lse[b].double()
            if n == 0:
                assert not out.any() and (lse == -float("inf")).all()
                continue
            k, q = self.rows(b), self.q[b].double()
            s = q @ k.T * self.scale
            ds = (q.abs() @ k.abs().T).amax(1) * self.scale * (self.latent + self.rope) * 2.0 ** -23
            p = torch.softmax(s, 1)
            v = k[:, :self.latent]
            want = p @ v
            spread = torch.stack([p[h] @ (v - want[h]).abs() for h in range(self.H)])
            tol = U * want.abs() + (U + ds[:, None]) * spread + 1e-5 * (p @ v.abs())
            err = (out - want).abs()
            assert (err <= tol).all(), (b, n, (err / tol).max().item())
            wl = torch.logsumexp(s, 1)
            el = (lse - wl).abs()
            assert (el <= ds + 2.0 ** -20 * (1 + wl.abs())).all(), (b, n, (el / (ds + 2.0 ** -20 * (1 + wl.abs()))).max().item())
        return self


CASES = {
    "one_token": dict(lens=[1], H=16),
    "tile_edges": dict(lens=[63, 64, 65, 127, 128, 129, 1], H=16),
    "empty_rows": dict(lens=[0, 70, 0, 1, 0], H=24),
    "all_empty": dict(lens=[0, 0, 0], H=64),
    "one_head": dict(lens=[100, 3], H=1),
    "heads_17": dict(lens=[200, 64], H=17, page=16),
    "heads_33": dict(lens=[130, 64, 190], H=33, page=8),
    "heads_48": dict(lens=[130, 640], H=48, page=24),
    "heads_64": dict(lens=[1000, 5], H=64, page=128),
    "heads_65": dict(lens=[300, 77], H=65, page=40),
    "heads_96": dict(lens=[256, 77, 3], H=96, page=256),
    "heads_128": dict(lens=[500, 1, 64, 1111], H=128),
    "pair_one_token": dict(lens=[1], H=128),
    "pair_tile_edges": dict(lens=[63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 1], H=128),
    "pair_empty_rows": dict(lens=[0, 70, 0, 1, 0], H=100),
    "pair_all_empty": dict(lens=[0, 0, 0], H=128),
    "pair_page_8": dict(lens=[300, 5, 64, 129], H=66, page=8),
    "pair_page_24": dict(lens=[1000, 77, 200], H=127, page=24),
    "pair_many_short": dict(lens=[(11 * i) % 300 for i in range(300)], H=72, page=16),
    "pair_256_rope_8": dict(lens=[400, 66, 1], H=80, latent=256, rope=8, page=192),
    "pair_256_rope_64": dict(lens=[4000, 66, 1], H=128, latent=256, rope=64),
    "pair_large_scores": dict(lens=[3000, 70, 1], H=128, qgain=30.0),
    "pair_two_pieces_each": dict(lens=[130 * 128] * 3, H=128),
    "two_groups_384": dict(lens=[700, 3, 129], H=128, latent=384),
    "two_groups_128": dict(lens=[700, 3, 129], H=90, latent=128, rope=16),
    "latent_128": dict(lens=[333, 64], H=40, latent=128, rope=8),
    "latent_256": dict(lens=[333, 65], H=128, latent=256, rope=32),
    "latent_384": dict(lens=[333, 66], H=64, latent=384, rope=56),
    "one_long": dict(lens=[20000], H=128),
    "long_beside_short": dict(lens=[9000, 1, 0, 30, 5000, 64, 64], H=20, page=48),
    "many_short": dict(lens=[(7 * i) % 131 for i in range(400)], H=8, page=16),
    "large_scores": dict(lens=[3000, 70, 1], H=32, qgain=30.0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_decode(lib, name):
    Setup(seed=len(name), **CASES[name]).run().check()


@pytest.mark.parametrize("H", [16, 128])
def test_rising_scores(lib, H):
    """Each tile's scores lie above the last one's, so the reference moves in every tile."""
    s = Setup([64 * 40 + 5], H, seed=2)
    n = s.lens_l[0]
    ramp = torch.linspace(0.0, 6.0, n, device="cuda")
    for i, p in enumerate(s.table[0, :-(-n // 64)].tolist()):
        r = ramp[i * 64:(i + 1) * 64]
        s.cache[p, :r.numel(), 0] = r.to(torch.bfloat16)
    s.q[:, :, 0] = 100.0
    s.run().check()


@pytest.mark.parametrize("H", [16, 128])
def test_minus_infinity_scores(lib, H):
    """Rows whose scores are all -inf give zeros; -inf beside finite scores takes no part."""
    s = Setup([80, 80], H, seed=3)
    s.q[:, :, 0] = 1.0
    rows = [s.table[b, j].item() for b in (0, 1) for j in (0, 1)]
    s.cache[rows[0], :, 0] = -float("inf")
    s.cache[rows[1], :16, 0] = -float("inf")     # sequence 0: all of its tokens
    s.cache[rows[2], 10:, 0] = -float("inf")     # sequence 1: tokens 10..63 of 80
    s.run()
    # 0 * inf in the values makes column 0 NaN, as the formula does; the others are the softmax's
    assert (s.att.lse[0] == -float("inf")).all() and not s.att.out[0, :, 1:].any()
    k = s.rows(1)
    keep = torch.tensor([j for j in range(80) if j < 10 or j >= 64], device="cuda")
    sc = s.q[1].double() @ k[keep].T * s.scale
    want = torch.softmax(sc, 1) @ k[keep][:, 1:512]
    assert (s.att.out[1, :, 1:].double() - want).norm() <= U * want.norm()
    assert (s.att.lse[1].double() - torch.logsumexp(sc, 1)).abs().max() < 1e-4


@pytest.mark.parametrize("H", [16, 128])
def test_nan_stays_in_its_sequence(lib, H):
    s = Setup([100, 100, 100], H, seed=4)
    p = s.table[1, 1].item()
    s.cache[p, 3, 500] = float("nan")
    s.run()
    assert torch.isnan(s.att.lse[1]).all() and torch.isnan(s.att.out[1]).all()
    assert torch.isfinite(s.att.out[[0, 2]].float()).all()


@pytest.mark.parametrize("H", [20, 70])
def test_pitched_queries_and_shared_pages(lib, H):
    s = Setup([300, 200], H, latent=256, rope=64, seed=5)
    s.table[1, :3] = s.table[0, :3]              # a common prefix of 192 tokens
    big = torch.full((2, H + 11, 400), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 3:H + 3, 8:328] = s.q
    s.q = big[:, 3:H + 3, 8:328]
    s.run().check()


def test_interleaved_shapes_share_a_stream(lib):
    """Calls of several shapes, one after another without waiting, with workspaces of their own."""
    sets = [Setup([900, 5, 130], 16, seed=1), Setup([2000, 64], 128, seed=2), Setup([300] * 9, 48, seed=3, page=24)]
    for _ in range(5):
        for s in sets:
            s.att.decode(s.q, s.cache, s.table, s.lens)
    torch.cuda.synchronize()
    for s in sets:
        s.att.check_status()
        s.check()


@pytest.mark.parametrize("H", [16, 128])
def test_repeats_give_the_same_bytes(lib, H):
    s = Setup([3000, 77, 1500], H, seed=6).run()
    a, b = s.att.out.clone(), s.att.lse.clone()
    for _ in range(3):
        s.run()
        assert torch.equal(s.att.out, a) and torch.equal(s.att.lse, b)


@pytest.mark.parametrize("H", [16, 128])
def test_cache_past_32_bit_offsets(lib, H):
    """Pages whose elements start past 2^31, and whose bytes start past 2^32."""
    Setup([700, 64, 129], H, seed=7, num_pages=70000).run().check()


@pytest.mark.parametrize("H", [16, 128])
def test_graph_replay_reads_new_lengths(lib, H):
    s = Setup([400, 900, 64], H, seed=8)
    full = list(s.lens_l)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.att.decode(s.q, s.cache, s.table, s.lens, stream=st.cuda_stream)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st, capture_error_mode="thread_local"):
        s.att.decode(s.q, s.cache, s.table, s.lens, stream=st.cuda_stream)
    for lens in ([1, 0, 63], [399, 65, 0], full):
        s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        s.lens_l = lens
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s.att.check_status()
        s.check()


@pytest.mark.parametrize("H", [16, 128])
def test_out_of_range_lengths_and_pages_are_reported(lib, H):
    s = Setup([100, 100, 100], H, seed=9)
    cap = s.att.max_pages * s.page
    s.lens.copy_(torch.tensor([100, -5, 100], dtype=torch.int32))
    s.att.decode(s.q, s.cache, s.table, s.lens)
    torch.cuda.synchronize()
    assert s.att.status() == (lib.MOE_ERR_BOUNDS, 60) and s.att.status() == (0, 0)
    assert not s.att.out[1].any() and (s.att.lse[1] == -float("inf")).all()
    s.lens.copy_(torch.tensor([100, cap + 1, 100], dtype=torch.int32))
    s.table[1, :] = s.table[1, 0].item()         # every page of the clamped length is valid
    s.att.decode(s.q, s.cache, s.table, s.lens)
    torch.cuda.synchronize()
    assert s.att.status() == (lib.MOE_ERR_BOUNDS, 60)
    for bad in (-1, s.att.num_pages, 2 ** 31 - 1):
        s = Setup([100, 100], H, seed=9)
        s.table[1, 1] = bad
        s.att.decode(s.q, s.cache, s.table, s.lens)
        torch.cuda.synchronize()
        assert s.att.status() == (lib.MOE_ERR_BOUNDS, 62)
        assert torch.isfinite(s.att.out.float()).all()


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("latent,rope,page,n,norm,rot", [
    (512, 64, 64, 1, True, True), (512, 64, 24, 300, True, True), (128, 8, 8, 33, True, True),
    (256, 32, 16, 77, False, True), (384, 48, 40, 50, True, False), (512, 64, 64, 9, False, False)])
def test_append(lib, latent, rope, page, n, norm, rot):
    from moe_layer_dsv3_gb300.attention import LatentAttention
    g = torch.Generator(device="cuda").manual_seed(n)
    B, width = 3, -(-n // page) + 1
    pool = B * width + 2
    att = LatentAttention(B, 16, latent, rope, page, pool, width, 1.0)
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(n))[:B * width].view(B, width).int().cuda()
    cache = torch.randn(pool, page, latent + rope, generator=g, device="cuda").to(torch.bfloat16)
    before = cache.clone()
    kv = torch.randn(n, latent + rope + 24, generator=g, device="cuda").to(torch.bfloat16)[:, 8:8 + latent + rope]
    gamma = (1 + 0.3 * torch.randn(latent, generator=g, device="cuda")).to(torch.bfloat16) if norm else None
    seq = (torch.arange(n) % B).int().cuda()
    pos = (torch.arange(n) // B + 3).int().cuda()
    pos[n // 2] = -1                             # a padding token writes nothing
    angle = torch.arange(n + 8, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float().cuda() if rot else None
    att.append(kv, cache, table, seq, pos, gamma=gamma, eps=EPS, cos_sin=cs)
    torch.cuda.synchronize()
    att.check_status()
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for i in range(n):
        p, b = pos[i].item(), seq[i].item()
        if p < 0:
            continue
        x = kv[i].double()
        c, r = x[:latent], x[latent:]
        tc = torch.zeros_like(c)
        if norm:
            c = c / torch.sqrt((c * c).mean() + EPS) * gamma.double()
            tc = U * (1 + 2.0 ** -6) * c.abs()
        tr = torch.zeros_like(r)
        if rot:
            co, si = cs[p].double().chunk(2)
            ev, od = r[0::2], r[1::2]
            size = (ev.abs() + od.abs()).repeat_interleave(2)
            r = torch.stack([ev * co - od * si, ev * si + od * co], 1).flatten()
            tr = U * r.abs() + 2.0 ** -22 * size
        page_id = table[b, p // page].item()
        want[page_id, p % page] = torch.cat([c, r])
        tol[page_id, p % page] = torch.cat([tc, tr])
    assert ((cache.double() - want).abs() <= tol).all()


def test_append_out_of_range_is_reported(lib):
    from moe_layer_dsv3_gb300.attention import LatentAttention
    att = LatentAttention(2, 16, 128, 32, 8, 6, 2, 1.0)
    table = torch.tensor([[0, 1], [2, 99]], dtype=torch.int32, device="cuda")
    kv = torch.ones(2, 160, dtype=torch.bfloat16, device="cuda")
    cs = torch.ones(12, 32, device="cuda")
    for seq, pos, site in ((2, 0, 65), (-1, 0, 65), (0, 16, 65), (0, 2 ** 31 - 1, 65), (0, 12, 65), (1, 9, 66)):
        cache = att.new_cache()
        att.append(kv, cache, table, torch.tensor([0, seq], dtype=torch.int32, device="cuda"),
                   torch.tensor([2, pos], dtype=torch.int32, device="cuda"), cos_sin=cs)
        torch.cuda.synchronize()
        assert att.status() == (lib.MOE_ERR_BOUNDS, site), (seq, pos)
        assert cache[0, 2].any() and cache.ne(0).any(2).sum() == 1     # the good token alone


def test_append_then_decode(lib):
    """Tokens written one step at a time are the ones the next decode sees."""
    s = Setup([5, 64, 0], 16, seed=12, fill=0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(3):
        kv = torch.randn(3, 576, generator=g, device="cuda").to(torch.bfloat16)
        seq = torch.arange(3, dtype=torch.int32, device="cuda")
        room = [n for n in s.lens_l]
        # sequences 0 and 1 have a page for their next token only where the setup gave them one
        pos = torch.tensor([room[0], -1, -1], dtype=torch.int32, device="cuda")
        s.att.append(kv, s.cache, s.table, seq, pos)
        s.lens_l[0] += 1
        s.lens.copy_(torch.tensor(s.lens_l, dtype=torch.int32))
        s.run().check()
        assert torch.equal(s.rows(0)[-1], kv[0].double())


def test_no_sequences_and_no_tokens(lib):
    cfg = lib.mla_config(0, 16, 512, 64, 64, 4, 4, 1.0)
    ws = torch.zeros(lib.moe_mla_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    cache = torch.zeros(4, 64, 576, dtype=torch.bfloat16, device="cuda")
    lib.moe_mla_decode(cfg, 0, 576, 576, cache.data_ptr(), 0, 0, 0, 0, ws.data_ptr())
    lib.moe_mla_append(cfg, 0, 0, 576, 0, 1e-6, 0, 0, 0, 0, 0, cache.data_ptr(), ws.data_ptr())
    torch.cuda.synchronize()
    assert lib.moe_mla_status(cfg, ws.data_ptr()) == (0, 0)


def test_failed_tensor_map_launches_nothing(lib):
    s = Setup([100], 16, seed=13)
    for _ in range(2):
        s.att.out.fill_(7.0)
        lib.moe_debug_fail_tensor_maps(1)
        with pytest.raises(lib.MoeError) as e:
            s.att.decode(s.q, s.cache, s.table, s.lens)
        lib.moe_debug_fail_tensor_maps(0)
        torch.cuda.synchronize()
        assert e.value.code == lib.MOE_ERR_CUDA and (s.att.out == 7.0).all()
    s.run().check()


@pytest.mark.parametrize("bad", [-1, -7, 400, 2 ** 31 - 1])
def test_append_bad_page_among_many_tokens(lib, bad):
    """Every token of a bad page is left out and the status set; all others are written, whatever their warp's next."""
    from moe_layer_dsv3_gb300.attention import LatentAttention
    n = 6000                                       # several tokens a warp
    B, page, width = 2, 24, 200
    att = LatentAttention(B, 16, 128, 32, page, B * width, width, 1.0)
    table = torch.arange(B * width, dtype=torch.int32).view(B, width).cuda()
    table[1, 3] = bad                              # 400 = the number of pages
    cache = att.new_cache()
    kv = torch.randn(n, 160, device="cuda").to(torch.bfloat16)
    seq = (torch.arange(n) % B).int().cuda()
    pos = (torch.arange(n) // B).int().cuda()
    att.append(kv, cache, table, seq, pos)
    torch.cuda.synchronize()
    assert att.status() == (lib.MOE_ERR_BOUNDS, 66)
    want = torch.zeros_like(cache)
    good = ~((seq == 1) & (pos // page == 3))
    want[(seq.long() * width + pos.long() // page)[good], (pos.long() % page)[good]] = kv[good]
    assert torch.equal(cache, want)
