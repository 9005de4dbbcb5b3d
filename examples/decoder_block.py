"""One DeepSeek-V3-style decoder block, served and trained with this library.

Serving: a prompt's latent rows are appended to a paged cache, then each step
appends one token a sequence, attends over the cache (absorbed latent
attention), and runs add + RMSNorm -> MoE layer, the layer reading the norm's
MXFP8 codes from its workspace. Training: the norm and the layer forward and
backward. Projections are plain torch products; weights are random.

    python examples/decoder_block.py [--steps 4]

Every step is checked against the same block in 64 bits (the MoE layer's output
is taken as given: its own tests hold it to its oracle).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_layer_dsv3_gb300 import MOE_FLAG_X_QUANTIZED  # noqa: E402
from moe_layer_dsv3_gb300.attention import LatentAttention  # noqa: E402
from moe_layer_dsv3_gb300.layer import MoELayer  # noqa: E402
from moe_layer_dsv3_gb300.norm import AddRMSNorm  # noqa: E402

EPS = 1e-6


def rope_table(positions, rope):
    freq = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def rotate(x, cs):
    """Rotate neighbouring columns of x [..., rope] by the angles of cs [..., rope] (cosines, then sines)."""
    co, si = cs.to(x.dtype).chunk(2, -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)


class DecoderBlock:
    """norm -> latent attention -> add + norm -> MoE, one new token a sequence."""

    def __init__(self, batch, d=1024, heads=16, nope=128, rope=64, latent=512, experts=16, topk=4, inner=256,
                 page_size=64, num_pages=64, max_pages=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)
        self.B, self.d, self.H, self.nope, self.rope, self.latent = batch, d, heads, nope, rope, latent
        gain = lambda n: (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
        self.g_in, self.g_kv, self.g_out = gain(d), gain(latent), gain(d)
        self.w_q = w(heads * (nope + rope), d)
        self.w_kv = w(latent + rope, d)
        self.w_uk, self.w_uv = w(heads, nope, latent), w(heads, nope, latent)   # keys, values from a latent row
        self.w_o = w(d, heads * nope)
        self.cos_sin = rope_table(page_size * max_pages, rope)
        self.norm_in, self.norm_out = AddRMSNorm(batch, d, EPS), AddRMSNorm(batch, d, EPS)
        self.att = LatentAttention(batch, heads, latent, rope, page_size, num_pages, max_pages, (nope + rope) ** -0.5)
        self.cache = self.att.new_cache()
        self.moe = MoELayer(batch, d, experts, topk, 1, 1, inner, 1, 128, flags=MOE_FLAG_X_QUANTIZED)
        self.w_router, self.bias = w(experts, d), torch.zeros(experts, device="cuda")
        self.moe.quantize_weights(w(experts, 2 * inner, d), w(experts, d, inner), w(1, 2 * inner, d), w(1, d, inner))

    def prefill(self, x, block_table, seq, pos):
        """Cache the tokens x [n][d] (the input stream) at positions pos of sequences seq."""
        n = AddRMSNorm(x.shape[0], self.d, EPS)
        kv = n.forward(x, self.g_in) @ self.w_kv.T
        self.att.append(kv, self.cache, block_table, seq, pos, gamma=self.g_kv, eps=EPS, cos_sin=self.cos_sin)

    def step(self, x, block_table, pos):
        """One new token a sequence: x [batch][d] at positions pos. Returns the block's output."""
        B, H = self.B, self.H
        y = self.norm_in.forward(x, self.g_in)
        self.att.append(y @ self.w_kv.T, self.cache, block_table, torch.arange(B, dtype=torch.int32, device="cuda"), pos,
                        gamma=self.g_kv, eps=EPS, cos_sin=self.cos_sin)
        q = (y @ self.w_q.T).view(B, H, self.nope + self.rope)
        q_lat = torch.einsum("bhn,hnc->bhc", q[..., :self.nope], self.w_uk)                  # absorb the key projection
        q_rot = rotate(q[..., self.nope:].float(), self.cos_sin[pos.long()][:, None]).to(torch.bfloat16)
        o = self.att.decode(torch.cat([q_lat, q_rot], 2), self.cache, block_table, pos + 1)
        attn = torch.einsum("bhc,hnc->bhn", o, self.w_uv).reshape(B, -1) @ self.w_o.T
        z = self.norm_out.forward(attn, self.g_out, residual=x, layer=self.moe)
        return self.norm_out.h + self.moe.forward(z, self.w_router, self.bias)

    def reference(self, x, streams, pos):
        """The block's residual stream after attention and the MoE's input in 64 bits, from each sequence's whole stream."""
        f = torch.float64
        norm = lambda v, g: v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * g.to(f)
        out = []
        for b, s in enumerate(streams):                       # s [tokens][d]: every token so far, the new one last
            y = norm(s.to(f), self.g_in)
            kv = y @ self.w_kv.to(f).T
            c, r = norm(kv[:, :self.latent], self.g_kv), rotate(kv[:, self.latent:], self.cos_sin[:len(s)])
            q = (y[-1] @ self.w_q.to(f).T).view(self.H, -1)
            k = torch.einsum("tc,hnc->htn", c, self.w_uk.to(f))
            v = torch.einsum("tc,hnc->htn", c, self.w_uv.to(f))
            qr = rotate(q[:, self.nope:], self.cos_sin[int(pos[b])][None])
            sc = (torch.einsum("hn,htn->ht", q[:, :self.nope], k) + qr @ r.T) * (self.nope + self.rope) ** -0.5
            out.append(torch.einsum("ht,htn->hn", torch.softmax(sc, 1), v).flatten() @ self.w_o.to(f).T)
        h = x.to(f) + torch.stack(out)
        return h, norm(h, self.g_out)


def serve(steps, verbose=True):
    B, page, max_pages = 5, 64, 8
    blk = DecoderBlock(B, page_size=page, max_pages=max_pages, num_pages=B * max_pages)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(B * max_pages, generator=torch.Generator().manual_seed(2)).int().view(B, max_pages).cuda()
    lens = [1, 63, 64, 200, 130]
    streams = [torch.randn(n, blk.d, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).int().cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    blk.prefill(torch.cat(streams), table, seq, pos)
    worst = 0.0
    for _ in range(steps):
        x = torch.randn(B, blk.d, generator=g, device="cuda").to(torch.bfloat16)
        streams = [torch.cat([s, x[b:b + 1]]) for b, s in enumerate(streams)]
        p = torch.tensor([len(s) - 1 for s in streams], dtype=torch.int32, device="cuda")
        blk.step(x, table, p)
        torch.cuda.synchronize()
        blk.att.check_status()
        blk.moe.check_status()
        h, z = blk.reference(x, streams, p)
        err = max(float((blk.norm_out.h.double() - h).norm() / h.norm()), float((blk.norm_out.y.double() - z).norm() / z.norm()))
        worst = max(worst, err)
    if verbose:
        print("served %d steps of %d sequences, largest relative error %.1e" % (steps, B, worst))
    return worst


def train(verbose=True):
    """add + norm -> MoE forward and backward; the gradients of the norm's inputs join the residual path's."""
    T, d = 256, 512
    blk = MoELayer(T, d, 8, 2, 1, 1, 128, 1, 128, flags=MOE_FLAG_X_QUANTIZED)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    w = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)
    blk.quantize_weights(w(8, 256, d), w(8, d, 128), w(1, 256, d), w(1, d, 128))
    norm, gamma = AddRMSNorm(T, d, EPS), r(d)
    y = norm.forward(r(T, d), gamma, residual=r(T, d), layer=blk)
    out = norm.h + blk.forward(y, w(8, d), torch.zeros(8, device="cuda"))
    dout = r(T, d)
    dx = norm.backward(blk.backward(dout), gamma, dres=dout)
    torch.cuda.synchronize()
    blk.check_status()
    # the norm's own gradient in 64 bits, from the layer's input gradient
    h, gy, rs = norm.h.double(), blk.dx.double() * gamma.double(), norm.rstd.double()[:, None]
    want = rs * (gy - h * rs * (gy * h * rs).mean(1, keepdim=True)) + dout.double()
    err = float((dx.double() - want).norm() / want.norm())
    if verbose:
        print("trained one step, output %s, relative error of the norm's gradient %.1e" % (tuple(out.shape), err))
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    serve(a.steps)
    train()
