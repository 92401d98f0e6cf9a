"""The barrier protocol of the pass over K that adds up weights (scored attention of more
than 8 query rows per KV head), checked on the CPU.

A CTA walks items, each of some tiles of positions and some blocks of query rows; a block
goes through all the item's tiles.  Roles: a thread that copies K tiles into a ring, one
that issues the products, two warps that bring a block's q and lse, and two groups of four
warps that take the tiles of a block in turns.  Copies and products complete some time
after they are issued, products in order.

The model runs random interleavings and checks that every read sees what it should: a
product its K tile and its block's q, a sum its tile's scores and its block's lse, and that
no warp arrives twice in one phase of a barrier and nobody waits for ever.  Its control: a
group that has no tile of a block must not run ahead of it (without the wait for the block's
q it arrives for later blocks in an earlier one's phase).
"""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.phase, self.who = count, 0, []

    def arrive(self, who):
        assert who not in self.who, "%s arrives twice in one phase" % (who,)
        self.who.append(who)
        if len(self.who) == self.count:
            self.who, self.phase = [], self.phase + 1

    def done(self, parity):
        # mbarrier.try_wait.parity: has the phase with this parity completed?
        return (self.phase & 1) != parity


def simulate(items, slots, buffers, q_buffers, seed, follow=True, steps=200000):
    """items: (tiles, blocks) each.  Returns the number of sums, or raises."""
    rng = random.Random(seed)
    kfull, kempty = ([Barrier(1) for _ in range(slots)] for _ in range(2))
    dfull, dfree = [Barrier(2) for _ in range(buffers)], [Barrier(4) for _ in range(buffers)]
    qready, lfree = [Barrier(2) for _ in range(2)], [Barrier(8) for _ in range(2)]
    qfree = [Barrier(1) for _ in range(q_buffers)]
    ring, scores, q, lse = {}, {}, {}, {}          # what stands where
    async_k, async_mma = [], []                    # copies in any order; products in theirs
    sums = []

    def blocks():
        nb = 0
        for item, (tiles, count) in enumerate(items):
            for _ in range(count):
                yield nb, item, tiles
                nb += 1

    def copies():
        n = 0
        for nb, _, tiles in blocks():
            for t in range(tiles):
                slot, use = n % slots, n // slots
                yield lambda: kempty[slot].done((use & 1) ^ 1)
                async_k.append((slot, (nb, t)))
                n += 1

    def land(i):
        slot, what = async_k.pop(i)
        ring[slot] = what
        kfull[slot].arrive("copy")

    def products():
        n, used, phase = 0, set(), [0] * buffers
        for nb, _, tiles in blocks():
            yield lambda: qready[nb & 1].done((nb >> 1) & 1)
            for t in range(tiles):
                buf, slot = t % buffers, n % slots
                if buf in used:
                    yield lambda: dfree[buf].done(phase[buf])
                    phase[buf] ^= 1
                yield lambda: kfull[slot].done((n // slots) & 1)
                used.add(buf)
                async_mma.append((nb, t, buf, slot, t + 1 == tiles))
                dfull[buf].arrive("issue")
                n += 1

    def execute():
        nb, t, buf, slot, last = async_mma.pop(0)
        assert ring[slot] == (nb, t), "K tile %s read as %s" % (ring[slot], (nb, t))
        assert q[nb % q_buffers] == nb, "q of block %d read as %d" % (q[nb % q_buffers], nb)
        scores[buf] = (nb, t)
        kempty[slot].arrive("commit")
        if last:
            qfree[nb % q_buffers].arrive("commit")
        dfull[buf].arrive("commit")

    def loader(w):
        for nb, _, _ in blocks():
            qb, use = nb % q_buffers, nb // q_buffers
            if use > 0:
                yield lambda: qfree[qb].done((use - 1) & 1)
            if nb > 1:
                yield lambda: lfree[nb & 1].done(((nb >> 1) - 1) & 1)
            q[qb] = nb
            lse[nb & 1] = nb
            yield lambda: True
            qready[nb & 1].arrive(w)

    def adder(w):
        group, phase = w // 4, [0] * buffers
        for nb, _, tiles in blocks():
            if follow:
                yield lambda: qready[nb & 1].done((nb >> 1) & 1)
            for t in range(group, tiles, 2):
                buf = t % buffers
                yield lambda: dfull[buf].done(phase[buf])
                phase[buf] ^= 1
                assert scores[buf] == (nb, t), "scores %s read as %s" % (scores[buf], (nb, t))
                assert lse[nb & 1] == nb, "lse of block %d read as %d" % (lse[nb & 1], nb)
                yield lambda: True
                assert scores[buf] == (nb, t) and lse[nb & 1] == nb
                dfree[buf].arrive(w)
                if w % 4 == 0:
                    sums.append((nb, t))
            yield lambda: True
            lfree[nb & 1].arrive(w)

    actors = [copies(), products(), loader(0), loader(1)] + [adder(w) for w in range(8)]
    waiting = {i: next(a, None) for i, a in enumerate(actors)}
    for _ in range(steps):
        live = [i for i, c in waiting.items() if c is not None]
        if not live and not async_k and not async_mma:
            break
        ready = [("actor", i) for i in live if waiting[i]()]
        ready += [("k", i) for i in range(len(async_k))] + ([("mma", 0)] if async_mma else [])
        assert ready, "nobody can go on: %d sums" % len(sums)
        kind, i = rng.choice(ready)
        if kind == "actor":
            waiting[i] = next(actors[i], None)
        elif kind == "k":
            land(i)
        else:
            execute()
    else:
        raise AssertionError("did not end")
    want = sorted((nb, t) for nb, _, tiles in blocks() for t in range(tiles))
    assert sorted(sums) == want
    return len(sums)


SHAPES = [
    [(1, 1)], [(1, 8)], [(1, 1)] * 7, [(2, 1), (1, 1), (3, 1)], [(1, 8), (1, 8)], [(2, 5)], [(3, 4)],
    [(5, 1), (4, 1), (1, 1), (6, 1)], [(1, 3), (2, 3), (5, 2)], [(9, 2), (1, 2)],
]


@pytest.mark.parametrize("buffers,q_buffers", [(4, 2), (2, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_every_read_sees_what_it_should(shape, buffers, q_buffers):
    """Four buffers of scores and two of q for up to 128 rows, two and one for more (only
    those have items of several blocks, but the protocol holds for any)."""
    for slots in (2, 3, 5, 12):
        for seed in range(15):
            simulate(SHAPES[shape], slots, buffers, q_buffers, seed)


def test_a_group_without_tiles_must_follow():
    caught = 0
    for seed in range(20):
        try:
            simulate([(1, 8)], 4, 2, 1, seed, follow=False)
        except AssertionError:
            caught += 1
    assert caught == 20
