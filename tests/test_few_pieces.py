"""The list of pieces of moe_few_forward and the room for their parts, as a model on the host.

Every step of every unit is in one piece, a piece's row ranges lie in the weights, and whatever the router
chooses, the parts of g, u and o fit the workspace.
"""
import random

import pytest

m = pytest.importorskip("moe_layer_dsv3_gb300")

UP, DOWN, MIN_STEPS, MAX_SMS, MAX_T = 1, 2, 2, 160, 64


def parts_of(units, steps, ctas, want):
    return min(-(-ctas * want // units), max(steps // MIN_STEPS, 1))


def cut_at(steps, i, n):
    return min(steps, (steps + 1) // 2 * i // n * 2)


def pieces(slots, d, inner, ctas):
    KA, KI = d // 128, inner // 128
    NB, RP = KI, (KA + 1) // 2
    PU, PD = parts_of(slots * NB, KA, ctas, UP), parts_of(slots * RP, KI, ctas, DOWN)
    nup = slots * NB * PU
    for p in range(nup + slots * RP * PD):
        if p < nup:
            u, part = divmod(p, PU)
            yield "up", u // NB, u % NB, part, cut_at(KA, part, PU), cut_at(KA, part + 1, PU)
        else:
            u, part = divmod(p - nup, PD)
            yield "down", u // RP, u % RP, part, cut_at(KI, part, PD), cut_at(KI, part + 1, PD)


@pytest.mark.parametrize("slots,d,inner", [(1, 128, 128), (1, 128, 4096), (1, 7168, 128), (9, 7168, 2048), (3, 384, 640), (38, 2048, 768),
                                           (513, 256, 128), (2, 896, 1152), (5, 1152, 896), (65, 7168, 2048)])
@pytest.mark.parametrize("ctas", [152, 148, 7])
def test_every_step_once(slots, d, inner, ctas):
    seen, last = {}, None
    for kind, s, b, part, k0, k1 in pieces(slots, d, inner, ctas):
        assert 0 <= s < slots and k0 < k1
        assert k0 % 2 == 0                                  # a cut lies between two whole pairs of steps
        assert not (last == "down" and kind == "up")
        last = kind
        seen.setdefault((kind, s, b), []).append((part, k0, k1))
    KA, KI = d // 128, inner // 128
    assert set(seen) == {("up", s, b) for s in range(slots) for b in range(KI)} | \
        {("down", s, b) for s in range(slots) for b in range((KA + 1) // 2)}
    for (kind, s, b), parts in seen.items():
        assert [p for p, _, _ in parts] == list(range(len(parts)))
        assert parts[0][1] == 0 and parts[-1][2] == (KA if kind == "up" else KI)
        assert all(x[2] == y[1] for x, y in zip(parts, parts[1:]))


def _room(T, d, E, k, inner, S):
    """The workspace's size, part by part as the library lays it out."""
    up = lambda n: -(-n // 1024) * 1024
    slots, rows = min(T * k, E) + S, T * (k + S)
    I128, d128 = inner // 128, d // 128

    def bound(steps, blocks, want):
        return min(T * (-(-MAX_SMS * want // blocks) + k + S), rows * max(steps // MIN_STEPS, 1))
    gu, o = bound(d128, I128, UP), bound(I128, (d128 + 1) // 2, DOWN)
    total = up(16 + 4 * MAX_T) + up(4 * (2 + slots + slots * I128)) + up(4 * T * E) + up(MAX_T * d) + up(d128 * 512) + \
        up((rows + 16) * inner) + up(slots * I128 * 512) + up(gu * I128 * 256 * 4) + up(o * d * 4)
    return total, gu, o


def test_parts_fit_whatever_is_chosen():
    r = random.Random(1)
    for _ in range(400):
        T, k = r.randint(1, 64), r.randint(1, 8)
        E = r.choice([k, r.randint(k, 40), r.randint(k, 512), 512])
        d, inner, S = 128 * r.choice([1, 2, 3, 7, 16, 56, 112]), 128 * r.choice([1, 2, 5, 6, 16, 31]), r.randint(0, 1)
        total, gu, o = _room(T, d, E, k, inner, S)
        assert m.moe_few_workspace_size(m.config(T, d, E, k, 1, 1, inner, S)) == total
        most = min(T * k, E) + S
        for slots in {1, 2, k, k + S, k + S + 1, most // 2, most - 1, most}:
            if not 1 <= slots <= most:
                continue
            rows = min(T * (k + S), slots * T)
            for ctas in (MAX_SMS, 152, 148, 20, 1):
                pu = parts_of(slots * (inner // 128), d // 128, ctas, UP)
                pd = parts_of(slots * ((d // 128 + 1) // 2), inner // 128, ctas, DOWN)
                assert pu == 1 or rows * pu <= gu
                assert rows * pd <= o
