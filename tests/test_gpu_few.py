"""moe_few_forward against the layer's formulas in 64 bits.

Tolerances of y, an element at a time, from its roundings. MX(x) is exact on both
sides (powers of two and one rounding of the same bf16 values). g and u are fp32 sums of d
products, each addition off by 2^-23 of the sum of magnitudes at most (the tensor
core may truncate); silu(g) u adds 2^-20 of itself for the exponential, the quotient
and the product. So h is known within dh, and MX(h) may be any value that a block
within dh quantises to: the largest distance of those from MX(h) times |Wd|, summed
over I, bounds what that does to o. The sums over I and over the experts are fp32
again, gates carry 2^-21 (a sum of at most 8 scores and a quotient), and y is rounded
to bf16 once: 2^-8. A logit is summed by 256 threads, 8 products of every 2048 columns
each, and joined by 5 + 7 additions: that many roundings of 2^-24, through a sigmoid of slope 1/4.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F = torch.float64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def scale_exp(top):
    """Exponent of the E8M0 scale of blocks with these largest magnitudes."""
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(torch.exp2(e) > top, e - 1, e)
    return e.clamp(min=-119.0) - 8


def on_grid(v, e):
    """v rounded to E4M3 values times 2^e."""
    u = v / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(u / step) * step).clamp(-448.0, 448.0) * torch.exp2(e)


def mx(v):
    w = v.reshape(*v.shape[:-1], -1, 32)
    return on_grid(w, scale_exp(w.abs().amax(-1, keepdim=True))).reshape(v.shape)


def mx_reach(h, dh):
    """How far MX of a value within dh of h may be from MX(h)."""
    w, dw = h.reshape(*h.shape[:-1], -1, 32), dh.reshape(*h.shape[:-1], -1, 32)
    at = on_grid(w, scale_exp(w.abs().amax(-1, keepdim=True)))
    far = torch.zeros_like(w)
    for top in ((w.abs() - dw).clamp(min=0).amax(-1, keepdim=True), (w.abs() + dw).amax(-1, keepdim=True)):
        e = scale_exp(top)
        for v in (w - dw, w + dw):
            far = torch.maximum(far, (on_grid(v, e) - at).abs())
    return far.reshape(h.shape)


class Case:
    def __init__(self, T, d, E, k, G=1, kept=1, I=128, S=0, seed=0, xgain=1.0, bias=0.0, same=False):
        from moe_layer_dsv3_gb300.few import FewTokenMoE
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.T, self.d, self.E, self.k, self.G, self.kept, self.I, self.S = T, d, E, k, G, kept, I, S
        x = xgain * rnd(1 if same else T, d)
        self.x = x.expand(T, d).to(torch.bfloat16).contiguous()
        self.w_router = (rnd(E, d) * 0.05).to(torch.bfloat16)
        self.bias = bias * rnd(E)
        self.gu = (rnd(E + S, 2 * I, d) * 0.5 / d ** 0.5).to(torch.bfloat16)
        self.down = (rnd(E + S, d, I) * 0.5 / I ** 0.5).to(torch.bfloat16)
        self.few = FewTokenMoE(T, d, E, k, G, kept, I, S)
        self.few.quantize_weights(self.gu[:E], self.down[:E], self.gu[E:], self.down[E:])

    def run(self, **kw):
        y = self.few.forward(self.x, self.w_router, self.bias, **kw)
        torch.cuda.synchronize()
        assert self.few.status() == (0, 0)
        return y

    def choice(self):
        """The choice in 64 bits and, a token at a time, whether no comparison it rests on is closer than the scores' error."""
        logits = self.x.to(F) @ self.w_router.to(F).T
        err = (-(-self.d // 2048) * 8 + 12) * 2.0 ** -24 * (self.x.to(F).abs() @ self.w_router.to(F).abs().T).amax(1) / 4 + 2.0 ** -21
        s = torch.sigmoid(logits)
        v = s + self.bias.to(F)
        sure = torch.ones(self.T, dtype=torch.bool, device="cuda")
        if self.G > 1:
            best = v.reshape(self.T, self.G, -1).sort(dim=2, descending=True).values[:, :, :2].sum(2)
            order = best.sort(dim=1, descending=True)
            if self.kept < self.G:
                sure &= order.values[:, self.kept - 1] - order.values[:, self.kept] > 4 * err
            keep = torch.zeros(self.T, self.G, dtype=torch.bool, device="cuda").scatter_(1, order.indices[:, :self.kept], True)
            v = torch.where(keep.repeat_interleave(self.E // self.G, 1), v, -torch.inf)
        top = v.sort(dim=1, descending=True)
        near = top.values[:, :min(self.k + 1, self.E)]
        if near.shape[1] > 1:
            sure &= ((near[:, :-1] - near[:, 1:]).amin(1) > 2 * err)
        idx = top.indices[:, :self.k]
        w = s.gather(1, idx)
        return idx, w / w.sum(1, keepdim=True), sure, err

    def reference(self, idx):
        """y for the given choice, and its tolerance."""
        s = torch.sigmoid(self.x.to(F) @ self.w_router.to(F).T).gather(1, idx)
        w = s / s.sum(1, keepdim=True)
        xq = mx(self.x.to(F))
        y, tol, mag = (torch.zeros(self.T, self.d, dtype=F, device="cuda") for _ in range(3))
        for e in range(self.E + self.S):
            t, j = torch.nonzero(idx == e, as_tuple=True) if e < self.E else (torch.arange(self.T, device="cuda"), None)
            if len(t) == 0:
                continue
            W, D = mx(self.gu[e].to(F)), mx(self.down[e].to(F))
            a, da = xq[t] @ W.T, self.d * 2.0 ** -23 * (xq[t].abs() @ W.abs().T)
            g, u, dg, du = a[:, :self.I], a[:, self.I:], da[:, :self.I], da[:, self.I:]
            sig = torch.sigmoid(g)
            h = g * sig * u
            # |silu'| <= 1.1
            dh = 1.1 * dg * (u.abs() + du) + (g * sig).abs() * du + 2.0 ** -20 * h.abs()
            hq = mx(h)
            o, m = hq @ D.T, hq.abs() @ D.abs().T
            to = mx_reach(h, dh) @ D.abs().T + self.I * 2.0 ** -23 * m
            f = 1.0 if j is None else w[t, j, None]
            y[t] += f * o
            tol[t] += f * to + (0.0 if j is None else 2.0 ** -21 * f * o.abs())
            mag[t] += f * o.abs()
        # partial sums of pieces and experts: no more additions than experts and pieces, 24 in all
        return y, tol + 24 * 2.0 ** -24 * mag + 2.0 ** -8 * (y.abs() + tol)

    def magnitude(self, idx):
        """Sum of w |o| over a token's experts, element by element."""
        s = torch.sigmoid(self.x.to(F) @ self.w_router.to(F).T).gather(1, idx)
        w = s / s.sum(1, keepdim=True)
        xq, mag = mx(self.x.to(F)), torch.zeros(self.T, self.d, dtype=F, device="cuda")
        for e in range(self.E + self.S):
            t, j = torch.nonzero(idx == e, as_tuple=True) if e < self.E else (torch.arange(self.T, device="cuda"), None)
            a = xq[t] @ mx(self.gu[e].to(F)).T
            o = mx(torch.nn.functional.silu(a[:, :self.I]) * a[:, self.I:]) @ mx(self.down[e].to(F)).T
            mag[t] += o.abs() * (1.0 if j is None else w[t, j, None])
        return mag

    def check(self, y=None):
        y = self.run() if y is None else y
        idx, w, sure, err = self.choice()
        got = self.few.topk_idx[:self.T].long()
        assert torch.equal(got[sure], idx[sure])
        assert sure.float().mean() > 0.5
        ref, tol = self.reference(got)
        logit_err = 4 * err[:, None]                        # a gate moves with its own score and with the sum
        s = torch.sigmoid(self.x.to(F) @ self.w_router.to(F).T).gather(1, got)
        assert ((self.few.topk_w[:self.T].to(F) - s / s.sum(1, keepdim=True)).abs() <= logit_err + 2.0 ** -21).all()
        tol = tol + logit_err * ref.abs()
        bad = (y.to(F) - ref).abs() > tol
        assert not bad.any(), (bad.sum().item(), ((y.to(F) - ref).abs() / tol).max().item())


# T, d, E, k, G, kept, I, S
SHAPES = [
    (1, 128, 1, 1, 1, 1, 128, 0),              # one tile of everything
    (1, 256, 8, 2, 1, 1, 128, 1),
    (2, 384, 8, 2, 4, 2, 256, 1),              # odd tile counts
    (3, 128, 4, 4, 1, 1, 896, 0),              # every expert chosen by every token
    (5, 896, 16, 3, 1, 1, 128, 0),
    (8, 256, 32, 8, 8, 4, 128, 1),
    (9, 512, 12, 5, 1, 1, 384, 1),
    (16, 256, 24, 2, 4, 1, 256, 0),
    (17, 640, 10, 8, 1, 1, 256, 1),
    (31, 256, 64, 8, 8, 3, 128, 0),
    (32, 1024, 6, 2, 3, 2, 512, 1),
    (33, 256, 512, 8, 1, 1, 128, 1),           # the most experts
    (47, 384, 40, 1, 1, 1, 256, 0),
    (64, 256, 8, 8, 1, 1, 128, 1),             # every expert has all tokens
    (64, 768, 96, 6, 32, 5, 256, 1),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_against_the_formula(lib, shape):
    T, d, E, k, G, kept, I, S = shape
    Case(T, d, E, k, G, kept, I, S, seed=sum(shape), bias=0.1 if G > 1 else 0.0).check()


def test_wide_layer(lib):
    """Many tiles a CTA, ranges that cut inside a reduction, the ring walked around many times."""
    Case(6, 4096, 8, 4, 1, 1, 1024, 1, seed=3).check()


def test_as_the_layer(lib):
    """The layer's own forward pass on the same weights: the same choice, and y within both calls' tolerances (the layer rounds
    each expert's output to bf16 before it sums them: 2^-8 of each)."""
    from moe_layer_dsv3_gb300.few import FewTokenMoE
    from moe_layer_dsv3_gb300.layer import MoELayer
    T, d, E, k, I = 40, 512, 16, 4, 256
    c = Case(T, d, E, k, 4, 2, I, 1, seed=5, bias=0.1)
    layer = MoELayer(T, d, E, k, 4, 2, I, 1, 128)
    layer.quantize_weights(c.gu[:E], c.down[:E], c.gu[E:], c.down[E:])
    y = layer.forward(c.x, c.w_router, c.bias)
    few = FewTokenMoE(T, d, E, k, 4, 2, I, 1, wq=layer.wq)
    c.few = few
    z = c.run()
    c.check(z)
    idx, _, sure, _ = c.choice()
    assert torch.equal(layer.topk_idx.long()[sure], few.topk_idx.long()[sure])
    ref, tol = c.reference(few.topk_idx.long())
    same = (layer.topk_idx == few.topk_idx).all(1)
    assert same.sum() >= sure.sum()
    # sum of w |o| <= the largest |o|, here bounded by the tolerance's own scale: 2^-8 of each term
    terms = c.magnitude(few.topk_idx.long())
    assert ((y.to(F) - ref).abs() <= 2 * tol + 2.0 ** -8 * terms)[same].all()


def test_fewer_tokens_than_the_buffers(lib):
    """Calls of every size in turn on one workspace, each as if it were the only one."""
    c = Case(64, 256, 12, 3, 1, 1, 256, 1, seed=6)
    x = c.x
    order = [64, 1, 17, 2, 16, 33, 8, 9, 64, 7]
    for t in order:
        c.T, c.x = t, x[:t]
        y = c.few.forward(c.x, c.w_router, c.bias)
        torch.cuda.synchronize()
        assert c.few.status() == (0, 0)
        c.check(y)
        assert y.data_ptr() == c.few.y.data_ptr() and y.shape == (t, 256)
    c.few.y.fill_(3.0)
    c.few.forward(x[:5], c.w_router, c.bias)
    torch.cuda.synchronize()
    assert (c.few.y[5:] == 3.0).all()                      # rows behind the last token stay
    empty = c.few.forward(x[:0], c.w_router, c.bias)
    assert empty.shape == (0, 256)


@pytest.mark.parametrize("T", [1, 12, 64])
def test_the_same_bytes_every_time(lib, T):
    """Which CTA takes a piece, and what the workspace held, change nothing."""
    c = Case(T, 1024, 8, 4, 1, 1, 512, 1, seed=7)
    y = c.run().clone()
    head = 16 + 4 * 64
    for i in range(20):
        c.few.ws[1024 * (-(-head // 1024)):].fill_((37 * i) % 256)
        assert torch.equal(c.run(), y)


def test_all_tokens_to_the_same_experts(lib):
    """One expert with 64 tokens beside ones without any: the longest and the shortest columns."""
    Case(64, 512, 40, 2, 1, 1, 256, 0, seed=8, same=True).check()
    Case(64, 512, 40, 2, 1, 1, 256, 1, seed=8, same=True).check()


@pytest.mark.parametrize("gain", [1e-4, 1e4, 1e15])
def test_small_and_large_inputs(lib, gain):
    """Scales far from 1 on the way: MX blocks near both ends, and silu at both of its limits."""
    c = Case(7, 256, 8, 2, 1, 1, 128, 1, seed=9, xgain=gain)
    if gain > 1e10:                                        # the products of h stay finite in fp32
        c.gu.mul_(1e-12)
        c.few.quantize_weights(c.gu[:8], c.down[:8], c.gu[8:], c.down[8:])
    # scores at both ends of the sigmoid tie: the choice is not what is looked at
    c.w_router.mul_(min(1.0, 1.0 / gain))
    c.check()


def test_zero_tokens_values(lib):
    c = Case(3, 256, 8, 2, 1, 1, 128, 1, seed=10)
    c.x[1].zero_()
    y = c.run()
    assert (y[1] == 0).all() and c.few.topk_idx[1].tolist() == c.bias.sort(descending=True, stable=True).indices[:2].tolist()
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("shared", [0, 1])
def test_a_nan_token_stays_alone(lib, shared):
    c = Case(9, 256, 8, 2, 1, 1, 128, shared, seed=11)
    y = c.run().clone()
    keep = torch.arange(9, device="cuda") != 4
    c.x[4, 100] = float("nan")
    z = c.run()                                            # (a score of NaN counts as the lowest, by the sigmoid's clamp)
    assert torch.isnan(z[4].float()).all()
    assert torch.isfinite(z[keep].float()).all()
    c.T, c.x = 8, c.x[keep].contiguous()
    idx = c.few.topk_idx[keep].long()
    ref, tol = c.reference(idx)
    assert ((z[keep].to(F) - ref).abs() <= tol + 2.0 ** -12 * ref.abs() + 2.0 ** -8 * (z[keep].float() - y[keep].float()).abs()).all()


@pytest.mark.parametrize("shared", [0, 1])
def test_no_choice_is_told(lib, shared):
    """A bias that is NaN for every expert, and for all but one of them where two are wanted."""
    c = Case(5, 256, 8, 2, 1, 1, 128, shared, seed=16)
    for good in (0, 1):
        c.bias.fill_(float("nan"))
        c.bias[:good] = 0.0
        z = c.few.forward(c.x, c.w_router, c.bias)
        torch.cuda.synchronize()
        assert c.few.status()[0] == lib.MOE_ERR_BOUNDS and torch.isnan(z.float()).all()
    c.bias.zero_()
    c.check()


def test_equal_scores_go_to_the_lower_experts(lib):
    c = Case(5, 256, 64, 8, 1, 1, 128, 0, seed=12)
    c.w_router[:] = c.w_router[0]
    c.bias.zero_()
    c.run()
    assert (c.few.topk_idx == torch.arange(8, device="cuda", dtype=torch.int32)).all()
    # a sum of 8 equal scores (3, 5, 6 and 7 times one are rounded) and a quotient: at most 8 roundings of 2^-24
    assert ((c.few.topk_w - 0.125).abs() <= 0.125 * 2.0 ** -21).all()


def test_captured_on_another_stream(lib):
    """Two graphs of one workspace and a call between their replays; each takes the inputs of the time."""
    c = Case(6, 512, 16, 3, 1, 1, 256, 1, seed=13)
    other = Case(6, 512, 16, 3, 1, 1, 256, 1, seed=14)
    x, small = c.x.clone(), c.x[:2].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty(2, 512, dtype=torch.bfloat16, device="cuda")
    calls = [lambda: c.few.forward(x, c.w_router, c.bias, stream=s.cuda_stream),
             lambda: c.few.forward(small, c.w_router, c.bias, stream=s.cuda_stream, y=y2)]
    graphs = []
    for f in calls:
        with torch.cuda.stream(s):
            f()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            f()
        graphs.append(g)
    want6 = c.run(y=torch.empty_like(x)).clone()
    for src in (c.x, other.x):
        x.copy_(src)
        small.copy_(src[:2])
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                graphs[0].replay()
                graphs[1].replay()
        s.synchronize()
        assert c.few.status() == (0, 0)
        got6, got2 = c.few.y.clone(), y2.clone()
        keep = c.x
        c.x = src
        assert torch.equal(c.run(y=torch.empty_like(x)), got6)
        c.x = src[:2].contiguous()
        assert torch.equal(c.few.forward(c.x, c.w_router, c.bias), got2)
        c.x = keep
    assert torch.equal(c.run(), want6)


def test_refused_tensors(lib):
    c = Case(4, 256, 8, 2, seed=15)
    f = c.few
    bad = lambda *a, **k: pytest.raises(lib.MoeError, f.forward, *a, **k)
    wide = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    bad(wide, c.w_router, c.bias)                          # more tokens than the buffers hold
    bad(c.x.float(), c.w_router, c.bias)
    bad(c.x.cpu(), c.w_router, c.bias)
    bad(c.x[:, ::2], c.w_router, c.bias)
    bad(torch.zeros(256, 8, dtype=torch.bfloat16, device="cuda").T[:4], c.w_router, c.bias)
    bad(c.x, c.w_router[:7], c.bias)
    bad(c.x, c.w_router, c.bias.double())
    bad(c.x, c.w_router, c.bias, y=wide)
    with pytest.raises(lib.MoeError):
        f.quantize_weights(c.gu[:7], c.down[:8])


def test_two_layers_at_once(lib):
    """Calls on two streams, each with a workspace of its own: their CTAs share the SMs, and neither waits for one that has none."""
    a, b = Case(16, 2048, 24, 4, 1, 1, 512, 1, seed=17), Case(30, 1024, 24, 4, 1, 1, 1024, 0, seed=18)
    want = [a.run().clone(), b.run().clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(40):
        for c, s in zip((a, b), streams):
            c.few.forward(c.x, c.w_router, c.bias, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        assert c.few.status() == (0, 0)
        assert torch.equal(c.few.y, w)
