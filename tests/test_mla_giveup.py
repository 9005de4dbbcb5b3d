"""Model of the pair decode kernel's softmax threads after a wait that gave up: the kernel still ends.

Two CTAs of eight threads (four warps of two lanes) walk tiles as csrc/k_mla_pair.cu does: a wait for the scores, the
barrier that hands out `grow`, the word sent to the other CTA, the wait for its word, and, where a reference moved,
the exchange of factors; at the end of a piece the barrier over the sums and the exchange of 1 / sum. Any wait on a
memory barrier may run out, in any lane, at any time. Checked for each order of steps tried: every thread reaches the
end (CTA barriers, votes and warp barriers have no limit), and no memory barrier gets more arrivals than it expects.
"""
import os
import random
import re

import pytest

WARPS, LANES = 4, 2
FIRST = (0, 1)                       # warps that speak for the heads
SPEAKER = (2, 0)                     # warp and lane that send the word


class Bar:
    """Memory barrier: `count` arrivals and all expected bytes end a phase."""

    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than the barrier expects"
        self.tx += tx
        self.pending -= 1
        self._turn()

    def deliver(self, n):
        self.tx -= n
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.pending, self.phase = self.count, self.phase + 1


class Cta:
    def __init__(self):
        self.gx, self.gf = [Bar(1), Bar(1)], [Bar(len(FIRST)), Bar(len(FIRST))]
        self.moved = [0, 0]


def softmax_thread(rank, warp, lane, ctas, grows, pieces, net):
    """Yields ("wait", bar, phase) -> whether it ended, ("barrier", flag) -> OR, ("vote", flag) -> any, ("warp",)."""
    me, other = ctas[rank], ctas[rank ^ 1]
    ok, swaps, tile = True, 0, 0

    def wait(bar, phase):
        nonlocal ok
        if ok:
            ok = yield ("wait", bar, phase)

    def exchange():
        nonlocal swaps
        k = swaps & 1
        if warp in FIRST:
            if ok:
                net.append((other.gf[k], None, 1))
            yield ("warp",)
            if lane == 0 and ok:
                me.gf[k].arrive(LANES)
        yield from wait(me.gf[k], swaps >> 1)
        swaps += 1

    for n, whole in pieces:
        for ti in range(n):
            par = tile & 1
            yield from wait(None, 0)                       # the scores: an event that comes, or does not
            grow = yield ("barrier", grows[rank][tile])
            if (warp, lane) == SPEAKER and ok:
                me.gx[par].arrive(1)
                net.append((other.gx[par], (other, par, grow), 1))
            yield from wait(me.gx[par], tile >> 1)
            theirs = me.moved[par]
            if (yield ("vote", grow or theirs)) and ti > 0:
                yield from exchange()
            tile += 1
        yield ("barrier", False)
        if whole:
            yield from exchange()


def run(seed, give_up):
    r = random.Random(seed)
    pieces = [(r.randint(1, 4), r.random() < 0.7) for _ in range(r.randint(1, 3))]
    tiles = sum(n for n, _ in pieces)
    grows = [[r.random() < 0.5 for _ in range(tiles)] for _ in range(2)]
    ctas, net = [Cta(), Cta()], []
    threads = {(c, w, l): softmax_thread(c, w, l, ctas, grows, pieces, net)
               for c in range(2) for w in range(WARPS) for l in range(LANES)}
    at = {t: next(g) for t, g in threads.items()}

    def step(t, answer):
        try:
            at[t] = threads[t].send(answer)
        except StopIteration:
            at[t] = ("end",)

    gave_up = 0
    while True:
        todo = []                                          # (weight, action)
        for i, (bar, word, n) in enumerate(net):
            todo.append((1.0, ("deliver", i)))
        for t, a in at.items():
            if a[0] == "wait":
                done = a[1] is None or a[1].phase > a[2]
                if done:
                    todo.append((1.0, ("go", t, True)))
                if give_up:
                    todo.append((0.02, ("go", t, False)))
        for c in range(2):
            group = [t for t in at if t[0] == c]
            if all(at[t][0] == "barrier" for t in group):
                todo.append((1.0, ("all", group, any(at[t][1] for t in group))))
            for w in range(WARPS):
                warp = [t for t in group if t[1] == w]
                for kind in ("vote", "warp"):
                    if all(at[t][0] == kind for t in warp):
                        todo.append((1.0, ("all", warp, any(at[t][1] for t in warp if len(at[t]) > 1))))
        if not todo:
            break
        what = r.choices([x for _, x in todo], [x for x, _ in todo])[0]
        if what[0] == "deliver":
            # words still under way when all threads are done: only where a thread gave up, and both CTAs then stay a while
            assert gave_up or any(a[0] != "end" for a in at.values()), seed
            bar, word, n = net.pop(what[1])
            if word is not None:
                word[0].moved[word[1]] = word[2]
            bar.deliver(n)
        elif what[0] == "go":
            gave_up += not what[2]
            step(what[1], what[2])
        else:
            for t in what[1]:
                step(t, what[2])
    stuck = {t: a[0] for t, a in at.items() if a[0] != "end"}
    assert not stuck, (seed, stuck)
    return gave_up


@pytest.mark.parametrize("part", range(8))
def test_every_thread_ends_after_a_wait_that_gave_up(part):
    assert sum(run(1000 * part + i, True) for i in range(150)) > 0


def test_every_wait_ends_where_none_gives_up():
    for seed in range(300):
        assert run(seed, False) == 0


def _source(name):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "moe_layer_dsv3_gb300", "csrc", name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_cta_barrier_depends_on_what_the_other_cta_sent():
    """The exchange holds no CTA barrier, and one answer a warp leads into it, as the model has it."""
    src = _source("k_mla_pair.cu")
    body = re.search(r"auto exchange = \[&\].*?\n    };", src, re.S).group(0)
    assert "named_barrier" not in body and "barrier_or" not in body and "__syncthreads" not in body
    read = src.index("&c.moved[par]) != 0u")
    lead = src[read:src.index("exchange(fac", read)]
    assert "__any_sync" in lead


@pytest.mark.parametrize("name,raw", [("k_mla.cu", "mbar_arrive("), ("k_mla_pair.cu", "mbar_arrive_remote(")])
def test_softmax_threads_arrive_only_while_their_waits_hold(name, raw):
    """Arrivals of a thread that runs ahead without waiting could be more than a barrier expects, or start a product early."""
    src = _source(name)
    soft = src[src.index("auto wait = [&]"):src.rindex("tmem_dealloc(tmem")]
    arrive = re.search(r"auto arrive = \[&\].*?\n    };", soft, re.S).group(0)
    assert re.search(r"if \([^;]*\bok\b[^;]*\) " + re.escape(raw), arrive)
    assert raw not in soft.replace(arrive, "")


@pytest.mark.parametrize("name", ["k_mla.cu", "k_mla_pair.cu"])
def test_a_cta_stays_after_a_wait_that_gave_up(name):
    """Between the last barrier of all roles and the release of TMEM, if any thread gave up."""
    src = _source(name)
    end = src[:src.rindex("tmem_dealloc(tmem")]
    assert "drain_pause()" in end[end.rindex("tc_fence_before()"):]
