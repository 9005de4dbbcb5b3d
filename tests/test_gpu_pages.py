"""moe_pages_update against a stack kept in Python: whole numbers, equal in every place."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """A table, a pool and lengths, on the host and on the GPU."""

    def __init__(self, batch, page, num_pages, max_pages, max_new, seed=0):
        from moe_layer_dsv3_gb300.pages import PagePlan
        r = random.Random(seed)
        self.page, self.max_pages, self.max_new = page, max_pages, max_new
        self.plan = PagePlan(batch, page, num_pages, max_pages, max_new)
        self.lens = [0] * batch
        self.free = list(range(num_pages))
        r.shuffle(self.free)
        self.count = num_pages
        self.table = [[-1000 - b] * max_pages for b in range(batch)]
        self.g = dict(table=i32(self.table), free=i32(self.free), count=i32([num_pages]), lens=i32(self.lens))

    def expect(self, target):
        """The step on the host: what it leaves and the maps of its tokens."""
        table, free = [list(t) for t in self.table], list(self.free)
        stack = free[:self.count]
        starts, seq, pos, slot = [0], [], [], []
        for b, (n, m) in enumerate(zip(self.lens, target)):
            for j in range(-(-m // self.page), -(-n // self.page)):
                stack.append(table[b][j])
        for b, (n, m) in enumerate(zip(self.lens, target)):
            for j in range(-(-n // self.page), -(-m // self.page)):
                table[b][j] = stack.pop()
            for p in range(n, m):
                seq.append(b)
                pos.append(p)
                slot.append(table[b][p // self.page] * self.page + p % self.page)
            starts.append(len(pos))
        for i in range(self.count, len(stack)):
            free[i] = stack[i]
        pad = self.max_new - len(pos)
        return dict(table=table, free=free, count=len(stack), lens=list(target), starts=starts, seq=seq + [0] * pad,
                    pos=pos + [-1] * pad, slot=slot + [-1] * pad)

    def call(self, target, **kw):
        t = target if torch.is_tensor(target) else i32(target)
        self.plan.update(self.g["lens"], t, self.g["table"], self.g["free"], self.g["count"], **kw)

    def compare(self, e):
        torch.cuda.synchronize()
        assert self.g["table"].tolist() == e["table"]
        assert self.g["free"].tolist() == e["free"]
        assert self.g["count"].tolist() == [e["count"]]
        assert self.g["lens"].tolist() == e["lens"]
        for n in ("starts", "seq", "pos", "slot"):
            assert getattr(self.plan, n).tolist() == e[n], n

    def step(self, target):
        e = self.expect(target)
        self.call(target)
        assert self.plan.status() == (0, 0)
        self.compare(e)
        self.table, self.free, self.count, self.lens = e["table"], e["free"], e["count"], e["lens"]


@pytest.mark.parametrize("batch,page,steps,most", [
    (1, 1, 6, 5), (1, 64, 8, 200), (3, 8, 12, 40), (37, 24, 10, 300), (96, 64, 6, 3), (255, 16, 5, 50), (256, 16, 5, 50),
    (257, 16, 5, 50), (1000, 7, 4, 30), (8192, 16, 3, 20), (5, 16, 4, 40000)])
def test_steps(lib, batch, page, steps, most):
    """Growing, shrinking, emptied and untouched sequences, in place, step after step."""
    r = random.Random(batch * 1000 + page)
    width = -(-(most * steps) // page) + 1
    m = Model(batch, page, batch * (-(-most * 2 // page) + 1) + 3, width, batch * most, seed=batch)
    for s in range(steps):
        target = []
        for n in m.lens:
            kind = r.random()
            n = 0 if kind < 0.1 else n if kind < 0.3 else max(0, n - r.randint(0, most)) if kind < 0.5 else min(n + r.randint(0, most), 2 * most)
            target.append(n)
        m.step(target)


def test_takes_what_was_just_left(lib):
    """More pages left than taken, the other way round, and as many of both, with an empty pool before the step."""
    for sizes, target in (([16, 32], [40, 0]), ([48, 8], [8, 16]), ([24, 24], [0, 48]), ([8, 40], [16, 32])):
        m = Model(2, 8, 7, 8, 64)
        m.step(sizes)
        m.step(target)
        m.step([0, 0])
        assert m.count == 7


def test_exact_fit_and_full_buffer(lib):
    m = Model(4, 8, 8, 4, 62)
    m.step([16, 16, 15, 15])                   # every page, and as many new tokens as the buffer holds
    assert m.count == 0
    m.step([16, 16, 16, 16])                   # no page left to take, none needed
    m.step([0, 0, 0, 0])


def test_refused_steps_change_nothing(lib):
    m = Model(3, 8, 6, 5, 32)
    m.step([10, 0, 7])
    def refuse(target, code, **other):
        before = {k: v.clone() for k, v in m.g.items()}
        for k, v in other.items():
            m.g[k].copy_(v)
        held = {k: v.clone() for k, v in m.g.items()}
        m.call(target)
        torch.cuda.synchronize()
        assert m.plan.status()[0] == code
        for k in m.g:
            assert torch.equal(m.g[k], held[k]), k
            m.g[k].copy_(before[k])
        assert m.plan.pos.tolist() == [-1] * 32 and m.plan.slot.tolist() == [-1] * 32 and m.plan.seq.tolist() == [0] * 32
        assert m.plan.starts.tolist() == [0] * 4
    refuse([24, 17, 7], lib.MOE_ERR_PAGES)     # four pages where three are free
    refuse([10, 33, 7], lib.MOE_ERR_BOUNDS)    # one token more than the buffer holds
    refuse([10, 0, -1], lib.MOE_ERR_BOUNDS)
    refuse([41, 0, 0], lib.MOE_ERR_BOUNDS)     # past the table
    refuse([2 ** 31 - 1] * 3, lib.MOE_ERR_BOUNDS)
    refuse([10, 0, 7], lib.MOE_ERR_BOUNDS, lens=i32([10, -3, 7]))
    refuse([10, 0, 7], lib.MOE_ERR_BOUNDS, lens=i32([10, 41, 7]))
    refuse([10, 0, 7], lib.MOE_ERR_BOUNDS, count=i32([-1]))
    refuse([10, 0, 7], lib.MOE_ERR_BOUNDS, count=i32([7]))
    refuse([0, 0, 0], lib.MOE_ERR_BOUNDS, count=i32([5]))     # more pages left than the pool has room for
    m.step([24, 16, 8])                        # and the next good one is made


def test_bad_pages_are_told(lib):
    m = Model(2, 8, 6, 4, 32)
    m.step([12, 3])
    m.g["table"][0, 1] = 6                     # the page that the next tokens of sequence 0 go to
    m.call([14, 4])
    torch.cuda.synchronize()
    assert m.plan.status()[0] == lib.MOE_ERR_BOUNDS
    assert m.plan.slot.tolist()[:2] == [-1, -1] and m.plan.slot.tolist()[2] >= 0
    m.g["free"][m.count - 1] = -5
    m.call([14, 12])
    torch.cuda.synchronize()
    assert m.plan.status()[0] == lib.MOE_ERR_BOUNDS
    assert m.plan.slot.tolist()[4:8] == [-1] * 4


def test_separate_outputs_leave_the_inputs(lib):
    m = Model(3, 8, 20, 6, 40)
    m.step([10, 20, 0])
    lens_out, count_out = torch.empty_like(m.g["lens"]), torch.empty_like(m.g["count"])
    target = [4, 30, 17]
    e = m.expect(target)
    for _ in range(3):                         # the same step again and again: the same answer
        m.call(target, lens_out=lens_out, count_out=count_out)
        torch.cuda.synchronize()
        assert m.g["lens"].tolist() == [10, 20, 0] and m.g["count"].tolist() == [m.count]
        assert lens_out.tolist() == target and count_out.tolist() == [e["count"]]
        assert m.g["table"].tolist() == e["table"] and m.plan.slot.tolist() == e["slot"]


def test_lengths_into_the_wanted_ones(lib):
    """lens_out may be any of the two."""
    m = Model(2, 8, 9, 4, 20)
    t = i32([9, 3])
    e = m.expect([9, 3])
    m.call(t, lens_out=t)
    torch.cuda.synchronize()
    assert t.tolist() == [9, 3] and m.g["lens"].tolist() == [0, 0] and m.plan.slot.tolist() == e["slot"]


def test_no_sequences_and_no_tokens(lib):
    from moe_layer_dsv3_gb300.pages import PagePlan
    p = PagePlan(0, 8, 4, 2, 5)
    table, free, count, lens = p.new_pool()
    p.update(lens, lens.clone(), table, free, count)
    torch.cuda.synchronize()
    assert p.pos.tolist() == [-1] * 5 and p.starts.tolist() == [0] and count.tolist() == [4]
    p = PagePlan(3, 8, 6, 2, 0)
    table, free, count, lens = p.new_pool()
    p.update(lens, i32([0, 0, 0]), table, free, count)
    assert p.status() == (0, 0) and p.starts.tolist() == [0] * 4
    p.update(lens, i32([0, 1, 0]), table, free, count)
    assert p.status()[0] == lib.MOE_ERR_BOUNDS


def test_captured_steps_replay(lib):
    """In a graph on a stream of its own: every replay takes the lengths of the time."""
    m = Model(6, 8, 60, 12, 60)
    target = i32([0] * 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.call(target, stream=s.cuda_stream)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
        m.call(target, stream=s.cuda_stream)
    r = random.Random(5)
    for _ in range(20):
        t = [min(80, max(0, n + r.randint(-8, 9))) for n in m.lens]
        e = m.expect(t)
        target.copy_(i32(t))
        g.replay()
        m.compare(e)
        m.table, m.free, m.count, m.lens = e["table"], e["free"], e["count"], e["lens"]
    assert m.plan.status() == (0, 0)
