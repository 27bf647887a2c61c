"""Model check of the V ring of the tcgen05 absorbed decode where a view leaves pages partly seen (decode_tc.cu), on
CPU.  Such a page is copied on this CTA's own barrier, its unseen rows are cleared by the producer warp's other lanes,
and both CTAs report on the leader's tail barrier before the PV issuer reads it.  A view can make any page of any step
partly seen, also both pages of one step and pages of successive steps, so the local and the tail barrier are one per page
of the step.  Copies land, and lanes run, in random order.  mbarriers follow the hardware's phase rule, and arriving on a
phase that still waits for a copy's bytes is an error; one shared barrier for both pages does exactly that."""
import random

import pytest

NV = 2


class Bar:
    """An mbarrier: arrivals of the current phase and bytes that it still waits for."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, tx=0):
        assert self.pending > 0, "an arrival that the phase did not expect"
        self.pending -= 1
        self.tx += tx
        self._turn()

    def land(self, tx):
        self.tx -= tx
        self._turn()

    def passed(self, parity):
        return (self.phase & 1) != parity


def simulate(pages, seed, shared=False, skip_tail=False):
    """pages: per step the two pages' states: "whole", "part" or "none" (zero-filled).  Returns "ok" or "deadlock"."""
    rnd = random.Random(seed)
    own = lambda pg: 0 if shared else pg  # noqa: E731
    full, empty = [Bar(1) for _ in range(NV)], [Bar(1) for _ in range(2 * NV)]     # empty: per CTA and slot
    local = [Bar(1) for _ in range(2 * NV)]                                        # per CTA and slot
    tail = [Bar(2) for _ in range(NV)]                                             # the leader's
    slots = [[None] * NV for _ in range(2)]
    landing = []                                                                   # copies under way

    def producer(cta):
        for g, step in enumerate(pages):
            for pg in range(NV):
                yield empty[NV * cta + pg], (g & 1) ^ 1
                slots[cta][pg] = None
                if step[pg] == "part":
                    if cta == 0:
                        full[pg].arrive()
                    b = local[NV * cta + own(pg)]
                    b.arrive(1)
                    landing.append((b, cta, pg, (g, "stale")))
                else:
                    if cta == 0:
                        full[pg].arrive(2)
                    landing.append((full[pg], cta, pg, (g, "clean")))

    def clearer(cta):
        ph = [0] * NV
        for g, step in enumerate(pages):
            for pg in range(NV):
                if step[pg] != "part":
                    continue
                yield local[NV * cta + own(pg)], ph[own(pg)] & 1
                ph[own(pg)] += 1
                assert slots[cta][pg] == (g, "stale"), ("cleared too early", slots[cta][pg], g)
                slots[cta][pg] = (g, "clean")
                tail[own(pg)].arrive()

    def issuer():
        ph = [0] * NV
        for g, step in enumerate(pages):
            for pg in range(NV):
                yield full[pg], g & 1
                if step[pg] == "part":
                    if not skip_tail:
                        yield tail[own(pg)], ph[own(pg)] & 1
                    ph[own(pg)] += 1
                for cta in range(2):
                    assert slots[cta][pg] == (g, "clean"), (cta, pg, slots[cta][pg], g)
                for cta in range(2):
                    empty[NV * cta + pg].arrive()

    roles = [producer(0), producer(1), clearer(0), clearer(1), issuer()]
    waits = {}
    for r, co in enumerate(roles):
        try:
            waits[r] = next(co)
        except StopIteration:
            pass
    while waits or landing:
        ready = [r for r, (bar, parity) in waits.items() if bar.passed(parity)]
        choices = ready + ["land"] * (1 if landing else 0)
        if not choices:
            return "deadlock"
        c = rnd.choice(choices)
        if c == "land":
            bar, cta, pg, what = landing.pop(rnd.randrange(len(landing)))
            slots[cta][pg] = what
            bar.land(1)
            continue
        try:
            waits[c] = next(roles[c])
        except StopIteration:
            del waits[c]
    return "ok"


def _cases(n, seed):
    rnd = random.Random(seed)
    for s in range(n):
        yield [tuple(rnd.choice(["whole", "part", "part", "none"]) for _ in range(NV)) for _ in range(rnd.randint(1, 8))], seed + s


def test_partly_seen_pages_in_any_order():
    for pages, seed in _cases(400, 10):
        assert simulate(pages, seed) == "ok", (pages, seed)
    for seed in range(100):
        assert simulate([("part", "part")] * 6, seed) == "ok"


@pytest.mark.parametrize("mistake", [dict(shared=True), dict(skip_tail=True)])
def test_planted_mistakes_are_caught(mistake):
    outcomes = set()
    for pages, seed in _cases(200, 5000):
        try:
            outcomes.add(simulate(pages, seed, **mistake))
        except AssertionError:
            outcomes.add("error")
    assert outcomes - {"ok"}
