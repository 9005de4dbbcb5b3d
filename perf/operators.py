"""Measured cases of the operators beside the MoE layer, each with a plain form.

Operators (entry points in include/moe.h, wrappers in moe_layer_dsv3_gb300):

norm_fwd   moe_add_rmsnorm: h = x + r, y = h rstd gamma, rstd = (mean(h^2) + eps)^(-1/2),
           with MX(y) (E4M3 codes, one E8M0 scale per 32 values) beside y.
norm_bwd   moe_add_rmsnorm_backward: the gradients of both inputs (one tensor, they are
           equal) and of gamma.
append     moe_mla_append: normalise and rotate the latent rows of new tokens and write
           them into a paged cache.
decode     moe_mla_decode: attention of one new token a sequence over the paged cache of
           latent rows that all heads share (absorbed form), split over the cache's
           length and joined.

``run`` computes the plain form (elementary torch operations in 32 bits) where ``own`` is
false and calls this package where it is true.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token's residual stream ahead of the experts, the layer's benchmark width
        dict(name="norm_fwd_token", op="norm_fwd", T=1, d=7168, residual=True, mx=True),
        # a ragged prefill chunk at an odd width, the first norm of a network (no residual yet)
        dict(name="norm_fwd_chunk", op="norm_fwd", T=1037, d=2016, residual=False, mx=True),
        # the layer's benchmark batch: 16384 tokens of width 7168, codes for the experts' products
        dict(name="norm_fwd_batch", op="norm_fwd", T=16384, d=7168, residual=True, mx=True),
        # a small training batch without a second path into the residual stream
        dict(name="norm_bwd_small", op="norm_bwd", T=301, d=1024, residual=False),
        # the layer's benchmark batch, gradient of the residual stream added
        dict(name="norm_bwd_batch", op="norm_bwd", T=16384, d=7168, residual=True),
        # one decoding step of 96 sequences: a row each, at scattered places
        dict(name="append_step", op="append", n=96, batch=96, mean=1500, latent=512, rope=64, page=64, salt=1),
        # a prefill of 32768 tokens over 9 sequences
        dict(name="append_prefill", op="append", n=32768, batch=9, mean=0, latent=512, rope=64, page=64, salt=2),
        # one short conversation on a shard of 16 heads: latency counts
        dict(name="decode_one", op="decode", batch=1, heads=16, mean=1500, ragged=False, empty=0, latent=512,
             rope=64, page=64, salt=3),
        # a mixed serving batch, odd head count, pages that end inside a tile, two empty slots
        dict(name="decode_mixed", op="decode", batch=37, heads=20, mean=700, ragged=True, empty=2, latent=512,
             rope=64, page=24, salt=4),
        # a full serving batch with all 128 heads on one GPU
        dict(name="decode_batch", op="decode", batch=128, heads=128, mean=4096, ragged=True, empty=0, latent=512,
             rope=64, page=64, salt=5),
        # two long documents: few rows, the work has to be split over the length
        dict(name="decode_long", op="decode", batch=2, heads=128, mean=131072, ragged=False, empty=0, latent=512,
             rope=64, page=64, salt=6),
        # long contexts on a shard of 16 heads: the cache's bytes bound it
        dict(name="decode_shard", op="decode", batch=64, heads=16, mean=16384, ragged=True, empty=0, latent=512,
             rope=64, page=128, salt=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "append", "decode", "decode"])
    salt = rng.randrange(1 << 30)
    if op in ("norm_fwd", "norm_bwd"):
        d = 32 * _log(rng, 4, 256)
        T = _log(rng, 1, min(16384, 16384 * 7168 // d))
        case = dict(op=op, T=T, d=d, residual=rng.random() < 0.6)
        if op == "norm_fwd":
            case["mx"] = rng.random() < 0.7
            if not case["mx"]:
                case["d"] -= 8 * rng.randrange(4)
        return case
    latent = rng.choice([128, 256, 384, 512, 512, 512])
    rope = rng.choice([32, 64, 64])
    page = rng.choice([8, 16, 24, 48, 64, 64, 128, 256])
    if op == "append":
        batch = _log(rng, 1, 128)
        step = rng.random() < 0.5
        return dict(op=op, n=batch if step else max(batch, _log(rng, 32, 32768)), batch=batch,
                    mean=_log(rng, 1, 4000) if step else 0, latent=latent, rope=rope, page=page, salt=salt)
    batch = _log(rng, 1, 192)
    heads = rng.choice([1, 8, 16, 16, 32, 40, 64, 128, 128, rng.randint(1, 128)])
    # no more cache rows than the listed cases hold, and no more products than the largest of them
    most = min(1 << 20, (1 << 19) * 128 // heads)
    mean = _log(rng, 1, max(2, min(131072, most // batch)))
    return dict(op=op, batch=batch, heads=heads, mean=mean, ragged=rng.random() < 0.7,
                empty=rng.choice([0, 0, 1]) if batch > 1 else 0, latent=latent, rope=rope, page=page, salt=salt)


def _lens(case):
    """Cached tokens of each sequence (decode), or already cached ones (append)."""
    r = random.Random(case["salt"])
    n, mean = case["batch"], case["mean"]
    if case.get("ragged", True):
        lens = [max(0 if mean == 0 else 1, int(mean * r.uniform(0.5, 1.5))) for _ in range(n)]
    else:
        lens = [mean] * n
    for i in r.sample(range(n), min(n, case.get("empty", 0))):
        lens[i] = 0
    return lens


def _new_tokens(case):
    """New tokens of each sequence (append): one each in a decoding step, else ragged with sum n."""
    n, b = case["n"], case["batch"]
    r = random.Random(case["salt"] + 1)
    w = [r.uniform(0.2, 1.8) for _ in range(b)]
    got = [1 + int((n - b) * x / sum(w)) for x in w]
    got[0] += n - sum(got)
    return got


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _paged(case, lens, seed):
    """Block table over a shuffled pool of pages with a few spare ones; unused entries are -1."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(1, max(need))
    num_pages = total + 3
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table.to(DEV), num_pages, width


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("norm_fwd", "norm_bwd"):
        T, d = case["T"], case["d"]
        # residual streams carry a few channels far above the rest
        chan = 1.0 + 19.0 * (torch.rand(d, generator=g, device=DEV) < 0.004).float()
        st["gamma"] = (1.0 + 0.2 * _randn(g, d, dtype=torch.float32)).to(torch.bfloat16)
        if op == "norm_fwd":
            st["x"] = _randn(g, T, d)
            st["residual"] = (_randn(g, T, d) * chan).to(torch.bfloat16) if case["residual"] else None
        else:
            st["h"] = (_randn(g, T, d) * chan).to(torch.bfloat16)
            st["dy"] = _randn(g, T, d)
            st["dres"] = _randn(g, T, d) if case["residual"] else None
            st["rstd"] = (st["h"].float().square().mean(1) + EPS).rsqrt()
        if own:
            from moe_layer_dsv3_gb300.norm import AddRMSNorm
            st["norm"] = AddRMSNorm(T, d, eps=EPS, mx=case.get("mx", False))
        return st
    lens = _lens(case)
    new = _new_tokens(case) if op == "append" else [0] * case["batch"]
    table, num_pages, width = _paged(case, [a + b for a, b in zip(lens, new)], seed)
    latent, rope, page = case["latent"], case["rope"], case["page"]
    st["table"] = table
    st["cache"] = _randn(g, num_pages, page, latent + rope)
    if op == "append":
        st["kv"] = _randn(g, case["n"], latent + rope)
        st["gamma"] = (1.0 + 0.2 * _randn(g, latent, dtype=torch.float32)).to(torch.bfloat16)
        st["seq"] = torch.tensor([b for b, k in enumerate(new) for _ in range(k)], dtype=torch.int32, device=DEV)
        st["pos"] = torch.tensor([lens[b] + i for b, k in enumerate(new) for i in range(k)], dtype=torch.int32,
                                 device=DEV)
        freq = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
        ang = torch.arange(max(a + b for a, b in zip(lens, new)), dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
    else:
        st["q"] = _randn(g, case["batch"], case["heads"], latent + rope)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["scale"] = (128 + rope) ** -0.5
    if own:
        from moe_layer_dsv3_gb300.attention import LatentAttention
        st["att"] = LatentAttention(case["batch"], case.get("heads", 1), latent=latent, rope=rope, page_size=page,
                                    num_pages=num_pages, max_pages=width, scale=st.get("scale", 1.0))
    return st


# ---------------------------------------------------------------- plain forms (32 bits, rounded once at the end)
def _mx(y):
    """E4M3 codes and E8M0 scales of the bf16 rows y, blocks of 32 along the row."""
    v = y.float().unflatten(1, (-1, 32))
    amax = v.abs().amax(2)
    exp = torch.frexp(amax)[1] - 1                                  # floor(log2 amax)
    byte = torch.where(amax > 0, (exp - 8 + 127).clamp(0, 254), 0)
    codes = torch.ldexp(v, (127 - byte).unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.flatten(1), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm_fwd(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    rstd = (h.square().mean(1) + EPS).rsqrt()
    y = (h * rstd[:, None] * st["gamma"].float()).to(torch.bfloat16)
    out = dict(y=y, rstd=rstd)
    if st["residual"] is not None:
        out["h"] = h.to(torch.bfloat16)
    if st["case"]["mx"]:
        out["codes"], out["scales"] = _mx(y)
    return out


def _plain_norm_bwd(st):
    h, dy, rstd = st["h"].float(), st["dy"].float(), st["rstd"]
    xhat = h * rstd[:, None]
    gdy = dy * st["gamma"].float()
    dx = (gdy - xhat * (gdy * xhat).mean(1, keepdim=True)) * rstd[:, None]
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return dict(dx=dx.to(torch.bfloat16), dgamma=(dy * xhat).sum(0))


def _plain_append(st):
    case = st["case"]
    latent, page = case["latent"], case["page"]
    kv = st["kv"].float()
    c = kv[:, :latent]
    c = c * (c.square().mean(1, keepdim=True) + EPS).rsqrt() * st["gamma"].float()
    pos = st["pos"].long()
    cos, sin = st["cos_sin"][pos].chunk(2, 1)
    even, odd = kv[:, latent::2], kv[:, latent + 1::2]
    rot = torch.stack([even * cos - odd * sin, even * sin + odd * cos], 2).flatten(1)
    rows = st["table"][st["seq"].long(), pos // page].long() * page + pos % page
    st["cache"].view(-1, kv.shape[1])[rows] = torch.cat([c, rot], 1).to(torch.bfloat16)
    return st["cache"]


def _plain_decode(st):
    latent = st["case"]["latent"]
    k = st["cache"][st["table"].long()].flatten(1, 2).float()                         # [B, L, latent + rope]
    seen = torch.arange(k.shape[1], device=DEV) < st["lens"][:, None]
    k = torch.where(seen[:, :, None], k, 0.0)
    s = torch.matmul(st["q"].float(), k.transpose(1, 2)) * st["scale"]                 # [B, H, L]
    s = torch.where(seen[:, None, :], s, -math.inf)
    m = s.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(2, keepdim=True)
    o = torch.matmul(p, k[:, :, :latent]) / torch.where(l > 0, l, 1.0)
    return dict(out=o.to(torch.bfloat16), lse=(m + torch.log(l)).squeeze(2))


_PLAIN = dict(norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd, append=_plain_append, decode=_plain_decode)


# ---------------------------------------------------------------- the framework's calls
def _own_norm_fwd(st):
    n = st["norm"]
    n.forward(st["x"], st["gamma"], st["residual"])
    out = dict(y=n.y, rstd=n.rstd)
    if st["residual"] is not None:
        out["h"] = n.h
    if st["case"]["mx"]:
        out["codes"] = n.codes.view(torch.float8_e4m3fn)
        out["scales"] = n.scales.view(torch.float8_e8m0fnu)
    return out


def _own_norm_bwd(st):
    n = st["norm"]
    n.backward(st["dy"], st["gamma"], st["dres"], h=st["h"], rstd=st["rstd"])
    return dict(dx=n.dx, dgamma=n.dgamma)


def _own_append(st):
    st["att"].append(st["kv"], st["cache"], st["table"], st["seq"], st["pos"], gamma=st["gamma"], eps=EPS,
                     cos_sin=st["cos_sin"])
    return st["cache"]


def _own_decode(st):
    att = st["att"]
    att.decode(st["q"], st["cache"], st["table"], st["lens"])
    return dict(out=att.out, lse=att.lse)


_OWN = dict(norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd, append=_own_append, decode=_own_decode)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what each cannot do without
def work(case):
    op = case["op"]
    if op == "norm_fwd":
        T, d = case["T"], case["d"]
        n = T * d
        by = 2 * n + 2 * n + 2 * d + 4 * T                      # x, y, gamma, rstd
        if case["residual"]:
            by += 4 * n                                         # residual in, h out
        if case["mx"]:
            by += n + n // 32                                   # codes, scales
        return dict(bytes=by, flops=6 * n)
    if op == "norm_bwd":
        T, d = case["T"], case["d"]
        n = T * d
        return dict(bytes=(8 if case["residual"] else 6) * n + 2 * d + 4 * d + 4 * T, flops=12 * n)
    row = 2 * (case["latent"] + case["rope"])
    if op == "append":
        n = case["n"]
        # rows in, rows out, sequence, position, page number; the rotation's rows are shared by sequences
        rot = 4 * case["rope"] * (max(_new_tokens(case)) if case["mean"] == 0 else n)
        return dict(bytes=n * (2 * row + 12) + rot + 2 * case["latent"], flops=n * (4 * case["latent"] + 6 * case["rope"]))
    lens, H = _lens(case), case["heads"]
    tokens, b = sum(lens), case["batch"]
    by = tokens * row + b * H * (row + 2 * case["latent"] + 4) + 4 * b + 4 * sum(-(-n // case["page"]) for n in lens)
    return dict(bytes=by, flops=2 * H * tokens * (2 * case["latent"] + case["rope"]))


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "norm_fwd":
        h = st["x"].to(f)
        if case["residual"]:
            h += st["residual"].to(f)
        rstd = 1.0 / torch.sqrt(torch.sum(h * h, 1) / case["d"] + EPS)
        y = torch.einsum("td,t,d->td", h, rstd, st["gamma"].to(f))
        out = dict(y=y, rstd=rstd)
        if case["residual"]:
            out["h"] = h
        if case["mx"]:
            # codes before their rounding to 8 bits; a scale is a choice of power of two, not a computed number
            top = y.to(torch.bfloat16).to(f).reshape(case["T"], -1, 32).abs().max(2).values
            e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 8
            out["codes"] = (y.reshape(case["T"], -1, 32) / torch.exp2(e)[:, :, None]).clamp(-448, 448).reshape(y.shape)
            out["scales"] = None
        return out
    if op == "norm_bwd":
        h, dy, g = st["h"].to(f), st["dy"].to(f), st["gamma"].to(f)
        r = st["rstd"].to(f)
        # y_i = h_i r g_i with dr/dh_j = -r^3 h_j / d
        dot = torch.einsum("td,td,d->t", dy, h, g)
        dx = torch.einsum("td,d,t->td", dy, g, r) - h * (r ** 3 * dot / case["d"])[:, None]
        if case["residual"]:
            dx += st["dres"].to(f)
        return dict(dx=dx, dgamma=torch.einsum("td,td,t->d", dy, h, r))
    latent, rope, page = case["latent"], case["rope"], case["page"]
    if op == "append":
        kv = st["kv"].to(f)
        cache = st["cache"].to(f)
        c = kv[:, :latent]
        c = c / torch.sqrt(torch.mean(c * c, 1) + EPS)[:, None] * st["gamma"].to(f)
        z = torch.view_as_complex(kv[:, latent:].reshape(-1, rope // 2, 2).contiguous())
        cs = st["cos_sin"].to(f)[st["pos"].long()]
        z = torch.view_as_real(z * torch.complex(cs[:, :rope // 2], cs[:, rope // 2:])).reshape(-1, rope)
        p = st["pos"].long()
        cache[st["table"].long()[st["seq"].long(), torch.div(p, page, rounding_mode="floor")], p % page] = torch.cat([c, z], 1)
        return cache
    B, H = case["batch"], case["heads"]
    out = torch.zeros(B, H, latent, dtype=f, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=f, device=DEV)
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        k = st["cache"][st["table"][b, :-(-n // page)].long()].reshape(-1, latent + rope)[:n].to(f)
        s = st["q"][b].to(f) @ k.T * st["scale"]
        lse[b] = torch.logsumexp(s, 1)
        out[b] = torch.softmax(s, 1) @ k[:, :latent]
    return dict(out=out, lse=lse)
