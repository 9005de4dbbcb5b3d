"""A serving step with drafted tokens, its operators run together: page plans, the append, the attention of the drafted
trees and the MoE layer of the few tokens.

The example's stream is held to 2e-2 of the 64-bit one: about ten roundings to bf16
(2^-9 relative on average each). Without a host wait, on another stream and in a
graph the same calls give the same bytes.
"""
import random

import pytest
import torch

from tests.test_gpu_example import _example

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_speculate():
    assert _example().speculate(4, verbose=False) < 2e-2


class Step:
    """Everything of one step in preallocated buffers, so that it can be captured."""

    def __init__(self, B=3, n=4, H=16, d=256):
        from moe_layer_dsv3_gb300.attention import LatentAttention
        from moe_layer_dsv3_gb300.few import FewTokenMoE
        from moe_layer_dsv3_gb300.norm import AddRMSNorm
        from moe_layer_dsv3_gb300.pages import PagePlan
        g = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
        self.B, self.n, self.g = B, n, g
        self.att = LatentAttention(B, H, 128, 32, 8, 40, 12, 160 ** -0.5, drafts=n)
        self.cache = self.att.new_cache()
        self.plan = PagePlan(B, 8, 40, 12, B * n)
        self.table, self.free, self.count, self.lens = self.plan.new_pool()
        self.target = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.kv, self.q = rnd(B * n, 160), rnd(B, n, H, 160)
        self.tree = torch.tensor([[1, 3, 7, 9]] * B, dtype=torch.int64, device="cuda")
        self.drafts = torch.full((B,), n, dtype=torch.int32, device="cuda")
        self.norm = AddRMSNorm(B * n, H * 128, 1e-6)
        self.gamma = rnd(H * 128)
        self.few = FewTokenMoE(B * n, H * 128, 12, 3, 1, 1, 128, 1)
        self.few.quantize_weights(rnd(12, 256, H * 128) * 0.02, rnd(12, H * 128, 128) * 0.05, rnd(1, 256, H * 128) * 0.02,
                                  rnd(1, H * 128, 128) * 0.05)
        self.w_router, self.bias = rnd(12, H * 128) * 0.05, torch.zeros(12, device="cuda")

    def run(self, stream=0, wait=lambda: None):
        p = self.plan
        p.update(self.lens, self.target, self.table, self.free, self.count, stream=stream)
        wait()
        self.att.append(self.kv, self.cache, self.table, p.seq, p.pos, stream=stream)
        wait()
        o = self.att.decode_tree(self.q, self.cache, self.table, self.lens, tree=self.tree, drafts=self.drafts, stream=stream)
        wait()
        y = self.norm.forward(o.view(self.B * self.n, -1), self.gamma, stream=stream)
        wait()
        self.few.forward(y, self.w_router, self.bias, stream=stream)
        wait()

    def results(self):
        return [t.clone() for t in (self.few.y, self.few.topk_idx, self.att.tree_out, self.att.tree_lse, self.plan.slot, self.table,
                                    self.free, self.count, self.lens, self.cache)]

    def targets(self, steps):
        r, lens, out = random.Random(2), [0] * self.B, []
        for s in range(steps):
            lens = [min(90, max(0, v + (self.n if s % 2 == 0 else -r.randint(0, self.n)))) for v in lens]
            out.append(torch.tensor(lens, dtype=torch.int32, device="cuda"))
        return out


def _rounds(how, steps=24):
    s = Step()
    st = torch.cuda.Stream() if how in ("stream", "graph") else None
    graph = None
    got = []
    for i, t in enumerate(s.targets(steps)):
        gen = torch.Generator(device="cuda").manual_seed(100 + i)
        s.kv.copy_(torch.randn(s.kv.shape, generator=gen, device="cuda"))
        s.q.copy_(torch.randn(s.q.shape, generator=gen, device="cuda"))
        s.target.copy_(t)
        s.drafts.copy_(torch.minimum(t, torch.full_like(t, s.n)))
        if how == "waits":
            s.run(wait=torch.cuda.synchronize)
        elif how == "queue":
            s.run()
        else:
            st.wait_stream(torch.cuda.current_stream())
            if how == "stream" or i == 0:
                s.run(st.cuda_stream)
            else:
                if graph is None:
                    st.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=st, capture_error_mode="thread_local"):
                        s.run(st.cuda_stream)
                with torch.cuda.stream(st):
                    graph.replay()
            torch.cuda.current_stream().wait_stream(st)
        got.append(s.results())
    torch.cuda.synchronize()
    assert s.plan.status() == (0, 0) and s.att.status() == (0, 0) and s.few.status() == (0, 0)
    return got


@pytest.mark.parametrize("how", ["queue", "stream", "graph"])
def test_the_same_bytes_without_waits(how):
    for a, b in zip(_rounds("waits"), _rounds(how)):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
