"""Measured cases of the operators of a serving step with drafted tokens, each with a plain form.

Operators (entry points in include/moe.h, wrappers in moe_layer_dsv3_gb300):

few        moe_few_forward: the whole MoE layer for up to 64 tokens. logits = x Wr^T,
           s = sigmoid(logits), v = s + bias, the k best v of the best groups, w = s / sum(s);
           [g | u] = MX(x) Wgu^T, h = silu(g) u, o = MX(h) Wd^T with MX weights, and
           y = sum over a token's experts of w o, plus the shared expert's o.
tree       moe_mla_decode_tree: attention of a tree of drafted tokens a sequence over the paged
           cache of latent rows. The drafted tokens are the sequence's last ones in the cache;
           each sees all tokens before them and those of them that its mask names.
pages      moe_pages_update: block tables and slot maps from request lengths. Pages of
           sequences that shrink go on a stack of free pages, sequences that grow take theirs
           from its top, and every new token gets its sequence, position and cache row.

``run`` computes the plain form (elementary torch operations in 32 bits, whole numbers in 64) where
``own`` is false and calls this package where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one conversation through a layer of wide experts with a shared one: latency counts
        dict(name="few_one", op="few", T=1, d=7168, E=64, k=8, groups=8, kept=4, inner=2048, shared=1, salt=1),
        # five drafted tokens through many narrow experts
        dict(name="few_small", op="few", T=5, d=2048, E=128, k=8, groups=1, kept=1, inner=768, shared=0, salt=2),
        # a decoding step of 16 sequences, most experts in use
        dict(name="few_batch", op="few", T=16, d=7168, E=64, k=8, groups=8, kept=4, inner=2048, shared=1, salt=3),
        # 8 sequences with 8 drafted tokens each: the most that one call takes, every expert in use
        dict(name="few_most", op="few", T=64, d=7168, E=64, k=8, groups=8, kept=4, inner=2048, shared=1, salt=4),
        # four drafted tokens of one short conversation on a shard of 16 heads: latency counts
        dict(name="tree_one", op="tree", batch=1, heads=16, drafts=4, mean=1500, ragged=False, padded=False, empty=0,
             latent=512, rope=64, page=64, salt=5),
        # a mixed serving batch: odd counts, pages that end inside a tile, fewer drafts in some, an empty slot
        dict(name="tree_mixed", op="tree", batch=23, heads=20, drafts=7, mean=700, ragged=True, padded=True, empty=1,
             latent=512, rope=64, page=24, salt=6),
        # a serving batch with all 128 heads on one GPU
        dict(name="tree_batch", op="tree", batch=32, heads=128, drafts=8, mean=4096, ragged=True, padded=False, empty=0,
             latent=512, rope=64, page=64, salt=7),
        # long contexts on a shard of 16 heads
        dict(name="tree_shard", op="tree", batch=48, heads=16, drafts=5, mean=8192, ragged=True, padded=True, empty=0,
             latent=512, rope=64, page=128, salt=8),
        # two long documents with wide trees
        dict(name="tree_long", op="tree", batch=2, heads=128, drafts=16, mean=65536, ragged=False, padded=False, empty=0,
             latent=512, rope=64, page=64, salt=9),
        # one decoding step of 96 sequences: a token each, a page now and then
        dict(name="pages_step", op="pages", batch=96, page=64, mean=1500, least=1, most=1, salt=10),
        # a verified step of 512 sequences: rejected drafts leave, new ones come
        dict(name="pages_verify", op="pages", batch=512, page=16, mean=700, least=-7, most=9, salt=11),
        # prompts of 37 requests, half a million tokens in all
        dict(name="pages_prefill", op="pages", batch=37, page=64, mean=0, least=500, most=28000, salt=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "tree", "tree", "tree", "pages"])
    salt = rng.randrange(1 << 30)
    if op == "few":
        d, inner = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 16)
        most = min(512, 65 * 7168 * 2048 // (d * inner))            # no more weights than the largest listed case
        groups, kept = rng.choice([(1, 1), (1, 1), (4, 2), (8, 4), (8, 3)])
        per = _log(rng, 2, most // groups)
        return dict(op=op, T=_log(rng, 1, 64), d=d, E=groups * per, k=rng.randint(1, min(8, kept * per)), groups=groups, kept=kept,
                    inner=inner, shared=rng.choice([0, 1]), salt=salt)
    if op == "pages":
        batch = _log(rng, 1, 1024)
        page = 8 * rng.choice([1, 2, 2, 3, 4, 8, 8, 16])
        if rng.random() < 0.6:
            return dict(op=op, batch=batch, page=page, mean=_log(rng, 1, 4000), least=rng.choice([1, 0, -1, -8, -60]),
                        most=_log(rng, 1, 64), salt=salt)
        batch = _log(rng, 1, 128)
        return dict(op=op, batch=batch, page=page, mean=0, least=_log(rng, 1, 200), most=_log(rng, 200, 700000 // batch), salt=salt)
    batch = _log(rng, 1, 64)
    heads = rng.choice([1, 8, 16, 16, 32, 40, 64, 128, rng.randint(1, 128)])
    drafts = _log(rng, 1, 64 if rng.random() < 0.5 else 12)
    # no more products, cache rows and scores than the largest listed cases
    most = min(1 << 19, (1 << 17) * 2048 // (heads * drafts))
    mean = _log(rng, 1, max(2, min(65536, most // batch)))
    return dict(op=op, batch=batch, heads=heads, drafts=drafts, mean=mean, ragged=rng.random() < 0.7,
                padded=rng.random() < 0.5, empty=rng.choice([0, 0, 1]) if batch > 1 else 0,
                latent=rng.choice([128, 256, 384, 512, 512, 512]), rope=rng.choice([32, 64, 64]),
                page=rng.choice([8, 16, 24, 48, 64, 64, 128, 256]), salt=salt)


def _lens(case):
    """Cached tokens of each sequence, the drafted ones included (tree), or before the step (pages)."""
    r = random.Random(case["salt"])
    n, mean, drafts = case["batch"], case["mean"], case.get("drafts", 0)
    if case.get("ragged", True):
        lens = [int(mean * r.uniform(0.5, 1.5)) + drafts for _ in range(n)]
    else:
        lens = [mean + drafts] * n
    for i in r.sample(range(n), min(n, case.get("empty", 0))):
        lens[i] = 0
    return lens


def _drafted(case):
    """Drafted tokens of each sequence."""
    r = random.Random(case["salt"] + 1)
    return [min(n, r.randint(1, case["drafts"]) if case["padded"] else case["drafts"]) for n in _lens(case)]


def _wanted(case):
    """Tokens of each sequence after the step."""
    r = random.Random(case["salt"] + 1)
    return [max(0, n + r.randint(case["least"], case["most"])) for n in _lens(case)]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _choose(logits, bias, case, f):
    """The router's choice from logits, in type f: experts in order of their value, gates, and the least gap of any choice made."""
    E, k, G = case["E"], case["k"], case["groups"]
    s = 1.0 / (1.0 + torch.exp(-logits.to(f)))
    v = s + bias.to(f)
    gap = torch.full((len(v),), math.inf, dtype=f, device=v.device)
    if G > 1:
        gs = v.view(-1, G, E // G).topk(2, 2).values.sum(2).sort(dim=1, descending=True, stable=True)
        if case["kept"] < G:
            gap = gs.values[:, case["kept"] - 1] - gs.values[:, case["kept"]]
        keep = torch.zeros_like(gs.values, dtype=torch.bool).scatter_(1, gs.indices[:, :case["kept"]], True)
        v = torch.where(keep.repeat_interleave(E // G, 1), v, -math.inf)
    top = v.sort(dim=1, descending=True, stable=True)
    near = top.values[:, :min(k + 1, E)]
    if near.shape[1] > 1:
        gap = torch.minimum(gap, (near[:, :-1] - near[:, 1:]).amin(1))
    idx = top.indices[:, :k]
    chosen = s.gather(1, idx)
    return idx, chosen / chosen.sum(1, keepdim=True), gap


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


def _mx(v):
    """E4M3 codes and E8M0 scale bytes of rows v, in blocks of 32 along the last dimension."""
    w = v.unflatten(-1, (-1, 32))
    amax = w.abs().amax(-1)
    exp = torch.frexp(amax)[1] - 1                                  # floor(log2 amax)
    byte = torch.where(amax > 0, (exp - 8 + 127).clamp(0, 254), 0)
    codes = torch.ldexp(w, (127 - byte).unsqueeze(-1)).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)
    return codes.flatten(-2), byte.to(torch.uint8)


def _unmx(codes, byte, f=torch.float32):
    return torch.ldexp(codes.to(f).unflatten(-1, (-1, 32)), byte.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)


def _few_inputs(case, g):
    T, d, E, inner = case["T"], case["d"], case["E"], case["inner"]
    w_router = (_randn(g, E, d, dtype=torch.float32) * 0.02).to(torch.bfloat16)
    bias = _randn(g, E, dtype=torch.float32) * (0.1 if case["groups"] > 1 else 0.0)
    # A choice that hangs on the last bits of a 32-bit sum is nobody's to make: such tokens are drawn again.
    kept, have = [], 0
    while have < T:
        x = _randn(g, T + 16, d)
        gap = _choose(x.double() @ w_router.double().T, bias, case, torch.float64)[2]
        kept.append(x[gap > 2e-5])
        have += len(kept[-1])
    gu = _randn(g, E + case["shared"], 2 * inner, d).mul_(0.5 / math.sqrt(d))
    down = _randn(g, E + case["shared"], d, inner).mul_(0.5 / math.sqrt(d))
    return torch.cat(kept)[:T].contiguous(), w_router, bias, gu, down


def _prepare_few(case, st, g):
    st["x"], st["w_router"], st["bias"], gu, down = _few_inputs(case, g)
    E = case["E"]
    if own:
        from moe_layer_dsv3_gb300.few import FewTokenMoE
        st["few"] = FewTokenMoE(case["T"], case["d"], E, case["k"], case["groups"], case["kept"], case["inner"], case["shared"])
        st["few"].quantize_weights(gu[:E], down[:E], gu[E:], down[E:])
    else:
        for name, w in (("gu", gu), ("down", down)):
            parts = [_mx(w[e].float()) for e in range(len(w))]
            st[name] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _prepare_tree(case, st, g, seed):
    lens, drafts = _lens(case), case["drafts"]
    latent, rope, page = case["latent"], case["rope"], case["page"]
    st["table"], num_pages, width = _paged(case, lens, seed)
    st["cache"] = _randn(g, num_pages, page, latent + rope)
    st["q"] = _randn(g, case["batch"], drafts, case["heads"], latent + rope)
    st["lens"], st["drafts"] = _int(lens), _int(_drafted(case))
    st["scale"] = (128 + rope) ** -0.5
    r = random.Random(seed)
    masks = []
    for _ in range(case["batch"]):
        seen = []
        for i in range(drafts):
            parent = r.randint(max(-1, i - 4), i - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        masks.append([m - (1 << 64) if m >> 63 else m for m in seen])
    st["tree"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
    if own:
        from moe_layer_dsv3_gb300.attention import LatentAttention
        st["att"] = LatentAttention(case["batch"], case["heads"], latent=latent, rope=rope, page_size=page,
                                    num_pages=num_pages, max_pages=width, scale=st["scale"], drafts=drafts)


def _pages_inputs(case, seed):
    page, lens, want = case["page"], _lens(case), _wanted(case)
    old, new = [-(-n // page) for n in lens], [-(-n // page) for n in want]
    width = max(1, max(old + new))
    spare = sum(max(0, b - a) for a, b in zip(old, new)) + 5
    num_pages = sum(old) + spare
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = spare
    for b, k in enumerate(old):
        table[b, :k] = perm[at:at + k]
        at += k
    free = torch.full((num_pages,), -1, dtype=torch.int32)
    free[:spare] = perm[:spare]
    total = sum(max(0, b - a) for a, b in zip(lens, want)) + 3                # a buffer a little larger than the step needs
    return table, free, spare, total


def _prepare_pages(case, st, seed):
    table, free, spare, st["new"] = _pages_inputs(case, seed)
    st["table"], st["free"], st["count"] = table.to(DEV), free.to(DEV), _int([spare])
    st["lens"], st["want"] = _int(_lens(case)), _int(_wanted(case))
    if own:
        from moe_layer_dsv3_gb300.pages import PagePlan
        st["plan"] = PagePlan(case["batch"], case["page"], len(free), table.shape[1], st["new"])
        st["lens_out"], st["count_out"] = torch.empty_like(st["lens"]), torch.empty_like(st["count"])


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "few":
        _prepare_few(case, st, g)
    elif case["op"] == "tree":
        _prepare_tree(case, st, g, seed)
    else:
        _prepare_pages(case, st, seed)
    return st


# ---------------------------------------------------------------- plain forms
def _plain_few(st):
    case = st["case"]
    E, inner = case["E"], case["inner"]
    x = st["x"].float()
    idx, w, _ = _choose(x @ st["w_router"].float().T, st["bias"], case, torch.float32)
    xq = _unmx(*_mx(x))

    def ffn(rows, gu, down):
        gu = rows @ _unmx(*gu).T
        g, u = gu[:, :inner], gu[:, inner:]
        return _unmx(*_mx(g / (1.0 + torch.exp(-g)) * u)) @ _unmx(*down).T

    gu, down = st["gu"], st["down"]
    y = torch.zeros_like(x)
    if idx.numel() < E:                                             # the experts of each assignment, read where they are
        flat = idx.flatten()
        for a in range(len(flat)):
            at = flat[a:a + 1]
            t = a // case["k"]
            o = ffn(xq[t:t + 1], [v.index_select(0, at)[0] for v in gu], [v.index_select(0, at)[0] for v in down])
            y[t] += w.flatten()[a] * o[0]
    else:
        dense = torch.zeros(len(x), E, device=DEV).scatter_(1, idx, w)
        for e in range(E):
            y += dense[:, e:e + 1] * ffn(xq, [v[e] for v in gu], [v[e] for v in down])
    if case["shared"]:
        y += ffn(xq, [v[E] for v in gu], [v[E] for v in down])
    return dict(y=y.to(torch.bfloat16), idx=idx.to(torch.int32), w=w)


def _seen(st, L):
    """What each drafted token sees: [batch, drafts, L]. Tokens past a sequence's own drafted ones see nothing."""
    n = st["case"]["drafts"]
    j = torch.arange(L, device=DEV)
    first = (st["lens"] - st["drafts"])[:, None, None]
    at = j - first                                                  # [B, 1, L]: which drafted token
    bit = (st["tree"][:, :, None] >> at.clamp(0, 63)) & 1 == 1
    seen = (at < 0) | ((j < st["lens"][:, None, None]) & bit)
    return seen & (torch.arange(n, device=DEV) < st["drafts"][:, None])[:, :, None]


def _plain_tree(st):
    latent = st["case"]["latent"]
    B, n, H, row = st["q"].shape
    k = st["cache"][st["table"].long()].flatten(1, 2).float()                         # [B, L, latent + rope]
    L = k.shape[1]
    k = torch.where((torch.arange(L, device=DEV) < st["lens"][:, None])[:, :, None], k, 0.0)
    s = torch.matmul(st["q"].float().flatten(1, 2), k.transpose(1, 2)) * st["scale"]   # [B, n H, L]
    s = torch.where(_seen(st, L)[:, :, None, :], s.view(B, n, H, L), -math.inf)
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(B, n * H, L), k[:, :, :latent]).view(B, n, H, latent) / torch.where(l > 0, l, 1.0)
    return dict(out=o.to(torch.bfloat16), lse=(m + torch.log(l)).squeeze(3))


def _plain_pages(st):
    page, n = st["case"]["page"], st["new"]
    lens, want, count = st["lens"].long(), st["want"].long(), st["count"].long()
    table, free = st["table"].long(), st["free"].long()
    B, width = table.shape
    old, new = (lens + page - 1) // page, (want + page - 1) // page
    grow, drop = (new - old).clamp(min=0), (old - new).clamp(min=0)
    G, F = grow.sum(), drop.sum()
    j = torch.arange(width, device=DEV)
    taken = (grow.cumsum(0) - grow)[:, None] + j - old[:, None]     # how many pages are taken before this one
    left = (drop.cumsum(0) - drop)[:, None] + j - new[:, None]
    is_new = (j >= old[:, None]) & (j < new[:, None])
    is_left = (j >= new[:, None]) & (j < old[:, None])
    stack = torch.cat([free, free.new_zeros(B * width + 1)])
    stack[torch.where(is_left, count + left, len(stack) - 1).flatten()] = table.flatten()
    table = torch.where(is_new, stack[(count + F - 1 - taken).clamp(0, len(stack) - 1)], table)
    at = torch.arange(len(free), device=DEV)
    free = torch.where((at >= count) & (at < count + F - G), stack[:len(free)], free)
    add = (want - lens).clamp(min=0)
    ends = add.cumsum(0)
    i = torch.arange(n, device=DEV)
    seq = torch.searchsorted(ends, i, right=True)
    live = seq < B
    seq = torch.where(live, seq, 0)
    pos = lens[seq] + i - (ends - add)[seq]
    slot = table[seq, torch.where(live, pos, 0) // page] * page + pos % page
    i32 = torch.int32
    return dict(table=table.to(i32), free=free.to(i32), count=(count + F - G).to(i32), lens=want.to(i32),
                starts=torch.cat([ends.new_zeros(1), ends]).to(i32), seq=seq.to(i32),
                pos=torch.where(live, pos, -1).to(i32), slot=torch.where(live, slot, -1).to(i32))


_PLAIN = dict(few=_plain_few, tree=_plain_tree, pages=_plain_pages)


# ---------------------------------------------------------------- the framework's calls
def _own_few(st):
    few = st["few"]
    few.forward(st["x"], st["w_router"], st["bias"])
    return dict(y=few.y, idx=few.topk_idx, w=few.topk_w)


def _own_tree(st):
    att = st["att"]
    att.decode_tree(st["q"], st["cache"], st["table"], st["lens"], tree=st["tree"], drafts=st["drafts"])
    return dict(out=att.tree_out, lse=att.tree_lse)


def _own_pages(st):
    p = st["plan"]
    p.update(st["lens"], st["want"], st["table"], st["free"], st["count"], lens_out=st["lens_out"], count_out=st["count_out"])
    return dict(table=st["table"], free=st["free"], count=st["count_out"], lens=st["lens_out"], starts=p.starts, seq=p.seq,
                pos=p.pos, slot=p.slot)


_OWN = dict(few=_own_few, tree=_own_tree, pages=_own_pages)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what each cannot do without
def work(case):
    op = case["op"]
    if op == "few":
        T, d, E, k, inner, S = (case[n] for n in ("T", "d", "E", "k", "inner", "shared"))
        # experts that some token chooses, if all are as likely: E (1 - (1 - k / E)^T)
        used = max(min(E, k), E * (1.0 - (1.0 - k / E) ** T)) + S
        by = int(used * 3 * d * inner * 33 / 32) + 2 * E * d + 4 * E + T * (4 * d + 8 * k)
        return dict(bytes=by, flops=6 * d * inner * T * (k + S) + 2 * T * E * d)
    lens = _lens(case)
    if op == "tree":
        n, H, b = case["drafts"], case["heads"], case["batch"]
        row, latent = case["latent"] + case["rope"], case["latent"]
        by = 2 * sum(lens) * row + b * n * H * (2 * row + 2 * latent + 4) + 8 * b * n + 8 * b
        by += 4 * sum(-(-x // case["page"]) for x in lens)
        # a drafted token's products: every token before the drafted ones, and about half of those
        pairs = sum(m * (x - m) + m * (m + 1) // 2 for x, m in zip(lens, _drafted(case)))
        return dict(bytes=by, flops=2 * H * pairs * (row + latent))
    want, page = _wanted(case), case["page"]
    new = sum(max(0, b - a) for a, b in zip(lens, want))
    moved = sum(abs(-(-b // page) - -(-a // page)) for a, b in zip(lens, want))
    return dict(bytes=12 * (new + 3) + 8 * moved + 16 * len(lens) + 12, flops=8 * (new + len(lens)))


# ---------------------------------------------------------------- 64 bits, from the definitions
def _round_mx(v):
    """MX of rows v (64 bits): each value on its block's grid of E4M3 values, as the values they stand for."""
    w = v.reshape(*v.shape[:-1], -1, 32)
    top = w.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(torch.exp2(e) > top, e - 1, e).clamp(min=-119.0) - 8             # the scale's exponent
    u = w / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)     # 3 bits after the leading one
    u = (torch.round(u / step) * step).clamp(-448.0, 448.0)
    return (u * torch.exp2(e)).reshape(v.shape)


def exact(case, seed):
    f = torch.float64
    if case["op"] == "pages":
        return _exact_pages(case, seed)
    if case["op"] == "few":
        x, w_router, bias, gu, down = _few_inputs(case, _gen(seed))
        x = x.to(f)
        E, k, G, inner = case["E"], case["k"], case["groups"], case["inner"]
        s = torch.sigmoid(x @ w_router.to(f).T)
        v = s + bias.to(f)
        if G > 1:
            best = v.reshape(-1, G, E // G).sort(2, descending=True).values[:, :, :2].sum(2)
            low = best.argsort(1, descending=True)[:, case["kept"]:]
            v = v.reshape(-1, G, E // G).clone()
            for t in range(len(x)):
                v[t, low[t]] = -math.inf
            v = v.reshape(-1, E)
        idx = v.argsort(1, descending=True)[:, :k]
        w = s.gather(1, idx)
        w = w / w.sum(1, keepdim=True)
        xq = _round_mx(x)
        y = torch.zeros_like(x)
        for e in range(E + case["shared"]):
            t, j = torch.nonzero(idx == e, as_tuple=True) if e < E else (torch.arange(len(x), device=DEV), None)
            if len(t) == 0:
                continue
            a = torch.einsum("td,id->ti", xq[t], _round_mx(gu[e].to(f)))
            h = torch.nn.functional.silu(a[:, :inner]) * a[:, inner:]
            o = torch.einsum("ti,di->td", _round_mx(h), _round_mx(down[e].to(f)))
            y[t] += o if j is None else o * w[t, j, None]
        return dict(y=y, idx=idx.to(torch.int32), w=w)
    st = prepare(case, seed)
    latent, rope = case["latent"], case["rope"]
    B, n, H, _ = st["q"].shape
    out = torch.zeros(B, n, H, latent, dtype=f, device=DEV)
    lse = torch.full((B, n, H), -math.inf, dtype=f, device=DEV)
    for b, (L, m) in enumerate(zip(_lens(case), _drafted(case))):
        if L == 0 or m == 0:
            continue
        k = st["cache"][st["table"][b, :-(-L // case["page"])].long()].reshape(-1, latent + rope)[:L].to(f)
        for i in range(m):
            mask = int(st["tree"][b, i]) & ((1 << m) - 1)
            rows = [L - m + j for j in range(m) if mask >> j & 1]
            ki = torch.cat([k[:L - m], k[rows]]) if rows else k[:L - m]
            if len(ki) == 0:
                continue
            s = st["q"][b, i].to(f) @ ki.T * st["scale"]
            lse[b, i] = torch.logsumexp(s, 1)
            out[b, i] = torch.softmax(s, 1) @ ki[:, :latent]
    return dict(out=out, lse=lse)


def _exact_pages(case, seed):
    page = case["page"]
    table, free, count, total = _pages_inputs(case, seed)
    table, free, lens, want = table.tolist(), free.tolist(), _lens(case), _wanted(case)
    stack = free[:count]
    for b, (a, z) in enumerate(zip(lens, want)):
        for j in range(-(-z // page), -(-a // page)):
            stack.append(table[b][j])
    starts, seq, pos, slot = [0], [], [], []
    for b, (a, z) in enumerate(zip(lens, want)):
        for j in range(-(-a // page), -(-z // page)):
            table[b][j] = stack.pop()
        for p in range(a, z):
            seq.append(b)
            pos.append(p)
            slot.append(table[b][p // page] * page + p % page)
        starts.append(len(pos))
    for i in range(count, len(stack)):
        free[i] = stack[i]
    pad = total - len(pos)
    return dict(table=_int(table), free=_int(free), count=_int([len(stack)]), lens=_int(want), starts=_int(starts),
                seq=_int(seq + [0] * pad), pos=_int(pos + [-1] * pad), slot=_int(slot + [-1] * pad))
