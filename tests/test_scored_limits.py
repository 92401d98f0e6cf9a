"""What the limited waits of the pass over K that adds up weights (scored attention of more
than 8 query rows per KV head) may time, checked on the CPU.

That launch starts beside the merge before it: copies, q and the plan need nothing of the
merge, while lse and the weights do, behind a wait for the launches before (the dependency
wait, without a limit).  Waits on barriers give up after a second.  A limited wait that only
something behind the dependency wait can end would time the launches before: where those take
longer, the weights would be wrong without a fault of this launch.

The model lets the launches before end only when nothing else can go on, and checks that
nobody stands in a limited wait then.  Its control: the roles without their own dependency
waits.
"""
import itertools

import pytest


def stuck_in(items, slots, q_buffers, guard):
    """items: (tiles, blocks) each.  The roles that stand in a limited wait while the launches
    before have yet to end.  Until then there are no products and no sums."""
    done = set()                 # barriers whose phase has completed
    LIMITED, DEPENDS = True, False
    blocks = [(nb, tiles) for nb, tiles in enumerate(
        itertools.chain.from_iterable([t] * c for t, c in items))]

    def copies():
        for n in range(sum(tiles for _, tiles in blocks)):
            if guard and n == slots:
                yield DEPENDS, None
            if n >= slots:
                yield LIMITED, ("read", n - slots)       # by a product
            done.add(("tile", n))

    def products():
        if guard:
            yield DEPENDS, None
        n = 0
        for nb, tiles in blocks:
            yield LIMITED, ("q and lse", nb)
            for _ in range(tiles):
                yield LIMITED, ("tile", n)
                done.add(("read", n))
                n += 1
            done.add(("products", nb))

    def loader():
        for nb, _ in blocks:
            if nb >= q_buffers:
                yield LIMITED, ("products", nb - q_buffers)
            if nb == 0:
                yield DEPENDS, None
            done.add(("q and lse", nb))

    def adder():
        yield DEPENDS, None

    roles = {"copies": copies(), "products": products(), "loader": loader(), "adder": adder()}
    at = {k: next(r, None) for k, r in roles.items()}
    while True:
        ready = [k for k, w in at.items() if w and w[0] is LIMITED and w[1] in done]
        if not ready:
            return sorted(k for k, w in at.items() if w and w[0] is LIMITED)
        for k in ready:
            at[k] = next(roles[k], None)


SHAPES = [[(1, 1)], [(1, 8)], [(40, 1)], [(2, 5), (1, 1)], [(3, 1)] * 9, [(16, 4)]]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("slots,q_buffers", [(2, 1), (4, 2), (12, 2)])
def test_limits_time_this_launch_alone(shape, slots, q_buffers):
    assert stuck_in(SHAPES[shape], slots, q_buffers, guard=True) == []


def test_without_their_own_dependency_waits_two_roles_time_the_launches_before():
    assert stuck_in([(40, 1)], 4, 2, guard=False) == ["copies", "products"]
    assert stuck_in([(1, 1)], 4, 2, guard=False) == ["products"]
