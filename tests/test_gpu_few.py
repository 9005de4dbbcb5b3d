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
import numpy as np
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
