"""What a kernel does before it ends after a wait that gave up, modelled on the CPU: an mbarrier as its phase, waits by
parity, arrivals that come when they like."""
import random


class Barrier:
    """An mbarrier whose phases are completed one after the other."""

    def __init__(self):
        self.phase = 0

    def complete(self):
        self.phase += 1

    def passes(self, parity):
        """Whether a wait for the phase of this parity returns at once."""
        return self.phase & 1 != parity


def test_last_products_are_waited_for_on_a_barrier_of_their_own():
    """The MMA thread commits what it has issued and waits for that commit before tensor memory is released. A wait for
    parity 0 on a barrier that tiles have gone through may pass before the commit has come; on a fresh one it does not."""
    early = []
    for tiles in range(6):
        used, fresh = Barrier(), Barrier()
        for _ in range(tiles):
            used.complete()
        early.append(used.passes(0))
        assert not fresh.passes(0)
        fresh.complete()  # the commit comes
        assert fresh.passes(0)
    assert early == [False, True, False, True, False, True]


def drain(first, g, stages):
    """(stage, parity) of the waits of the loading thread for the units first .. g - 1."""
    return [(h % stages, h // stages & 1) for h in range(first, g)]


def ring(stages, g, landed, end_marker):
    """The stages' barriers after `g` units, those below `landed` being there, and with the marker that tells the end."""
    bars = [Barrier() for _ in range(stages)]
    for h in range(landed):
        bars[h % stages].complete()
    if end_marker:
        bars[g % stages].complete()
    return bars


def test_copies_in_flight_are_waited_for_whoever_gave_up():
    """The loading thread may have issued its last copy before a consumer gives up. Whatever is still in flight then, its
    waits do not all pass, and once it has landed they all do, also where the stage after the last unit has served to
    tell the end (the unit that it held before was consumed)."""
    for stages in range(1, 7):
        for g in range(0, 4 * stages + 2):
            for told in (False, True):
                first = g - stages + (1 if told else 0) if g >= stages else 0
                for landed in range(first, g + 1):
                    bars = ring(stages, g, landed, told)
                    passes = all(bars[s].passes(p) for s, p in drain(first, g, stages))
                    assert passes == (landed == g), (stages, g, told, landed)


def test_the_stage_that_told_the_end_is_not_waited_for():
    """Its barrier is a phase further: a wait for the unit that it held would not pass any more."""
    for stages in range(1, 7):
        g = 3 * stages + 1
        bars = ring(stages, g, g, True)
        assert not all(bars[s].passes(p) for s, p in drain(g - stages, g, stages))


def pieces_of(items, cost, ctas):
    """The attention's work split: items of `cost` units and their blocks in one line, cut into equal ranges; per CTA the
    (item, first block, end) that it holds, and per CTA the item that it starts and does not end, with the last CTA of it."""
    total = sum(cost + n for n in items)
    ctas = min(ctas, total)
    held, joins = [], []
    for c in range(ctas):
        u0, u1 = total * c // ctas, total * (c + 1) // ctas
        mine, join, first = [], None, 0
        for i, n in enumerate(items):
            b0, b1 = max(0, u0 - first - cost), min(n, u1 - first - cost)
            if b1 > b0 and u1 > first and u0 < first + cost + n:
                mine.append((i, b0, b1))
                if b0 == 0 and b1 < n:
                    join = (i, ((first + cost + n) * ctas + total - 1) // total - 1)
            first += cost + n
        held.append(mine)
        joins.append(join)
    return held, joins


def test_an_item_with_a_missing_piece_is_not_joined():
    """A CTA that gave up leaves a mark in place of its own item to join; the joining block of an item looks for marks among
    the CTAs that hold its pieces. Items without a mark are complete, and what no mark touches is joined."""
    rng = random.Random(3)
    for _ in range(300):
        items = [rng.randint(1, rng.choice([2, 10, 200])) for _ in range(rng.randint(1, 30))]
        held, joins = pieces_of(items, rng.choice([2, 4]), rng.choice([2, 7, 148, 444]))
        gone = {c for c in range(len(held)) if rng.random() < 0.2}
        for c, join in enumerate(joins):
            if join is None:
                continue
            i, last = join
            blocks = sorted((b0, b1) for d in range(c, last + 1) for j, b0, b1 in held[d] if j == i)
            assert [b for b, _ in blocks] == [0] + [e for _, e in blocks[:-1]] and blocks[-1][1] == items[i]  # all pieces, in c .. last
            assert all(any(j == i for j, _, _ in held[d]) for d in range(c, last + 1))
            complete = not any(d in gone for d in range(len(held)) if any(j == i for j, _, _ in held[d]))
            assert complete == (c not in gone and not any(d in gone for d in range(c, last + 1)))


def test_a_cluster_whose_sums_are_not_all_there_finishes_no_rows():
    """The blocks of a cluster each hold a part of the sums, written by four warps. A warp that has none to write marks every
    block before they meet; behind the meeting a block finishes its rows if it has no mark."""
    rng = random.Random(4)
    for _ in range(500):
        blocks = rng.choice([1, 2, 4, 8])
        have = [[rng.random() < 0.95 for _ in range(4)] for _ in range(blocks)]
        marked = [False] * blocks
        for warps in have:
            for there in warps:
                if not there:
                    marked = [True] * blocks
        for b in range(blocks):
            assert (not marked[b]) == all(all(w) for w in have)
