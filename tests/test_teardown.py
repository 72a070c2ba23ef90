"""What a kernel does before it ends after a wait that gave up, modelled on the CPU: an mbarrier as its phase, waits by
parity, arrivals that come when they like."""


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
