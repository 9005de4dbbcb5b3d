"""The norm, append and decode read what the kernel just before them on the stream wrote: lengths, tables, positions,
weights, rows. Each is launched early and waits on the device, so a chain of writes and calls without a host wait has
to give the bytes of the same calls with a wait before each."""
import pytest
import torch

from tests.test_gpu_mla import Setup

pytestmark = pytest.mark.gpu

N = 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _both(body):
    """body(i, sync) for i < N, without and with a wait before each call."""
    got = []
    for sync in ((lambda: None), torch.cuda.synchronize):
        torch.cuda.synchronize()
        got.append([body(i, sync) for i in range(N)])
        torch.cuda.synchronize()
    for a, b in zip(*got):
        for x, y in zip(a, b):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("H", [16, 128])
def test_decode(H):
    s = Setup([300, 64, 1, 900, 129], H, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    full = s.lens.clone()
    lens = [(full * torch.rand(5, generator=g, device="cuda")).int() for _ in range(N)]
    # sequences change places: lengths, pages and queries move together
    order = [torch.randperm(5, generator=g, device="cuda") for _ in range(N)]
    table = s.table.clone()
    q = [torch.randn(s.q.shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(N)]

    def body(i, sync):
        out, lse = torch.empty_like(s.att.out), torch.empty_like(s.att.lse)
        s.lens.copy_(lens[i][order[i]])
        s.table.copy_(table[order[i]])
        s.q.copy_(q[i])
        sync()
        s.att.decode(s.q, s.cache, s.table, s.lens, out=out, lse=lse)
        return out, lse

    _both(body)
    s.att.check_status()


def test_append():
    from moe_layer_dsv3_gb300.attention import LatentAttention
    B, n, page, width = 4, 600, 24, 9
    att = LatentAttention(B, 16, 256, 32, page, B * width, width, 1.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    perm = [torch.randperm(B * width, generator=g, device="cuda").view(B, width).int() for _ in range(N)]
    where = [torch.randperm(B * width * page, generator=g, device="cuda")[:n] for _ in range(N)]
    kvs, gammas, tables = [r(n, 288).to(torch.bfloat16) for _ in range(N)], [r(256).to(torch.bfloat16) for _ in range(N)], \
        [r(width * page, 32) for _ in range(N)]
    kv, gamma, cs = kvs[0].clone(), gammas[0].clone(), tables[0].clone()
    table = perm[0].clone()
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")

    def body(i, sync):
        cache = att.new_cache()
        kv.copy_(kvs[i])
        cs.copy_(tables[i])
        table.copy_(perm[i])
        seq.copy_(where[i] // (width * page))
        pos.copy_(where[i] % (width * page))
        gamma.copy_(gammas[i])
        sync()
        att.append(kv, cache, table, seq, pos, gamma=gamma, cos_sin=cs)
        return (cache,)

    _both(body)
    att.check_status()


@pytest.mark.parametrize("T,d", [(3, 512), (700, 1024), (300, 7168)])
def test_norm(T, d):
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    n = AddRMSNorm(T, d, mx=True)
    xs, dys = [r(T, d) for _ in range(4)], [r(T, d) for _ in range(4)]
    gammas = [r(d) for _ in range(N)]
    x, dy, gamma = xs[0].clone(), dys[0].clone(), gammas[0].clone()

    def body(i, sync):
        x.copy_(xs[i % 4])
        dy.copy_(dys[(i + i // 4) % 4])
        gamma.copy_(gammas[i])
        sync()
        y = n.forward(x, gamma, residual=dy)
        sync()
        n.backward(dy, gamma, dres=x)
        return y.clone(), n.codes.clone(), n.scales.clone(), n.rstd.clone(), n.dx.clone(), n.dgamma.clone()

    _both(body)
