"""Model of the latent decode's work split: every tile has one worker, and every cut sequence one complete list of pieces.

The device finds a worker's range, its pieces and the join's entries from the
lengths with the integer arithmetic written here (csrc/mla.cuh: find_range, Walk,
owner_of, join_entry).
"""
import random

import pytest


def _split(lens, tile, W, min_tiles):
    tiles = [-(-n // tile) for n in lens]
    total = sum(tiles)
    most = -(-total // min_tiles)
    W = min(W, most if most > 0 else 1)
    begin = lambda w: total * w // W
    starts = [sum(tiles[:b]) for b in range(len(lens))]
    pieces, entries = [], []
    for w in range(W):
        f0, f1 = begin(w), begin(w + 1)
        mine = []
        for b, (s, n) in enumerate(zip(starts, tiles)):
            lo, hi = max(f0, s), min(f1, s + n)
            if lo < hi:
                mine.append((b, lo - s, hi - lo))
        pieces.append(mine)
        entry = None
        if mine and mine[0][1] > 0:
            b, t0, _ = mine[0]
            s0 = f0 - t0
            if s0 + tiles[b] <= f1:
                w0 = ((s0 + 1) * W - 1) // total           # owner_of
                entry = (b, 0 if begin(w0) == s0 else 1, w0, w - w0 + 1)
        entries.append(entry)
    return tiles, pieces, entries


@pytest.mark.parametrize("seed", range(40))
def test_split(seed):
    r = random.Random(seed)
    tile, min_tiles = r.choice([(64, 3), (128, 2)])
    n = r.choice([1, 2, 7, 40, 300])
    lens = [r.choice([0, 1, tile, r.randint(1, 5000), r.randint(1, 100)]) for _ in range(n)]
    W = r.choice([1, 2, 76, 152])
    tiles, pieces, entries = _split(lens, tile, W, min_tiles)
    seen = {b: [] for b, k in enumerate(tiles) if k}
    sizes = []
    for w, mine in enumerate(pieces):
        sizes.append(sum(k for _, _, k in mine))
        for at, (b, t0, k) in enumerate(mine):
            seen[b].append((t0, k, w, 0 if at == 0 else 1))
    assert max(sizes) - min(sizes) <= 1
    joined = {e[0]: e for e in entries if e}
    assert len(joined) == sum(e is not None for e in entries)
    for b, got in seen.items():
        got.sort()
        assert got[0][0] == 0 and sum(k for _, k, _, _ in got) == tiles[b]
        assert all(x[0] + x[1] == y[0] for x, y in zip(got, got[1:]))
        if len(got) == 1:
            assert b not in joined                          # written whole by its worker
        else:
            _, first_slot, w0, count = joined[b]
            # consecutive workers, each with its range's first piece after the first one
            assert [w for _, _, w, _ in got] == list(range(w0, w0 + count))
            assert got[0][3] == first_slot and all(s == 0 for _, _, _, s in got[1:])


def test_range_begin_in_32_bits():
    """range_begin: total * w / W from the quotient and the remainder of total / W."""
    r = random.Random(1)
    for _ in range(20000):
        W = r.randint(1, 160)
        total, w = r.choice([r.randrange(2 ** 31), r.randrange(1, 2000), W, 2 ** 31 - 1]), r.randint(0, W)
        q, rest = divmod(total, W)
        assert rest * w < 2 ** 32 and q * w + rest * w // W == total * w // W


def test_page_of_a_token_by_multiplication():
    """BoxRows: token / page as the high word of a product, for every page size and token the library takes."""
    r = random.Random(2)
    pages = list(range(8, 2049, 8)) + [2 ** k + d for k in range(5, 31) for d in (-8, 0, 8)] + [2 ** 31 - 8]
    for page in pages:
        log = 3
        while 2 ** log < page:
            log += 1
        mul = 2 ** (31 + log) // page + 1
        assert mul < 2 ** 32
        some = [r.randrange(2 ** 31 // page + 1) * page + d for d in (-1, 0, 1) for _ in range(20)]
        for tok in [0, 1, page - 1, page, 2 ** 31 - 1] + [t for t in some if 0 <= t < 2 ** 31]:
            assert ((tok * mul) >> 32) >> (log - 1) == tok // page
