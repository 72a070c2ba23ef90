"""How the consumer warps of the decode attention leave together when a wait has given up: the meeting of the four warps
modelled on the CPU, every interleaving with the producer warp, which may set the flag at any time."""
from functools import lru_cache

WARPS, ITEMS = 4, 2
READ, FIRST, LEAVE, SECOND, DONE = range(5)  # before a read of the flag, in the first barrier, past it, in the second


def stuck(vote):
    """Whether some interleaving ends with a warp in a barrier that never completes. An item: look at the flag, meet in the
    first barrier, leave if the flag says so, else meet in the second. With `vote` the look comes before the first barrier,
    which hands each warp the looks of all; without, each warp looks for itself behind the barrier."""

    @lru_cache(None)
    def run(flag, warps):  # warps: (place, what it brought or got, item)
        again = []
        if not flag:
            again.append((True, warps))  # the producer gives up
        for w, (place, saw, item) in enumerate(warps):
            def to(*state):
                again.append((flag, warps[:w] + (state,) + warps[w + 1:]))
            if place == READ:
                to(FIRST, flag if vote else False, item)
            elif place == LEAVE:
                if saw if vote else flag:
                    to(DONE, saw, item)
                else:
                    to(SECOND, False, item)
        for place, then in ((FIRST, LEAVE), (SECOND, READ)):
            if all(w[0] == place for w in warps):
                any_saw = any(w[1] for w in warps)
                item = warps[0][2] + (place == SECOND)
                again.append((flag, tuple((then if item < ITEMS else DONE, any_saw, item) for _ in warps)))
        again = [a for a in again if a[1] != warps or a[0] != flag]
        if not any(a[1] != warps for a in again) and any(w[0] != DONE for w in warps):
            if not again:
                return True  # nobody can go on, and not everybody has left
        return any(run(*a) for a in again)

    return run(False, ((READ, False, 0),) * WARPS)


def test_warps_that_vote_in_the_barrier_never_wait_for_one_that_left():
    assert not stuck(vote=True)


def test_warps_that_look_behind_the_barrier_may():
    assert stuck(vote=False)
