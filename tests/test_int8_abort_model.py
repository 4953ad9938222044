"""Host model of how the int8 GEMM kernels end when a wait has run out (gemm_int8.cuh, gemm_int8_wide.cuh): the token loaders of
one CTA, or of a pair whose copies all arrive on the leader's barrier, and a consumer that gives up at any time.  A
copy still in flight when the CTAs are gone would write into the next one's shared memory, so none may be.

What the kernels do comes through; what they did before, to wait only in a loader that had itself been stopped, and not
for what the peer alone had issued, is caught, which shows that the model can."""
import random

import pytest


class InFlight(Exception):
    pass


class Barrier:
    """One arrival and the bytes that it expects, in halves of a stage; bytes may come before the arrival."""

    def __init__(self):
        self.phase, self.arrived, self.bytes = 0, False, 0

    def _turn(self):
        if self.arrived and self.bytes == 0:
            self.phase, self.arrived = self.phase + 1, False

    def expect(self, halves):
        assert not self.arrived
        self.arrived, self.bytes = True, self.bytes + halves
        self._turn()

    def land(self):
        self.bytes -= 1
        self._turn()

    def done(self, parity):
        return (self.phase & 1) != parity


def simulate(seed, ranks, stages, total, always=True, tell=True):
    """always: a loader that was not stopped waits for its copies too.  tell: the peer tells what it has issued."""
    rng = random.Random(seed)
    full = [Barrier() for _ in range(stages)]
    empty = [[0] * stages for _ in range(ranks)]         # phases done
    abort = [False] * ranks
    flying, told = [], [None]
    give_up = rng.randrange(0, total + 1)                # the k-block at which the consumer stops; total: never
    late = []                                            # what one CTA does to another's memory

    def loader(rank):
        at, phase, issued, ok = 0, 0, {}, True
        for n in range(total):
            while (empty[rank][at] & 1) == (phase ^ 1):
                if abort[rank]:
                    ok = False
                    break
                yield
            if not ok:
                break
            if rank == 0:
                full[at].expect(ranks)
            flying.append(full[at])
            issued[at] = phase
            at += 1
            if at == stages:
                at, phase = 0, phase ^ 1
            yield
        else:
            n = total
        if rank == 1:
            if tell:
                late.append(lambda: told.__setitem__(0, n))
            return
        if ranks == 2 and tell:
            while told[0] is None:
                yield
            for _ in range(told[0] - n):
                full[at].expect(1)
                issued[at] = phase
                at += 1
                if at == stages:
                    at, phase = 0, phase ^ 1
        if ok and not always:
            return
        for s, ph in issued.items():
            idle = 0
            while not full[s].done(ph):   # the limit is far longer than a copy: it runs out when none is left
                idle = 0 if flying else idle + 1
                if idle > 50:
                    break
                yield

    def consumer():
        at, phase = 0, 0
        for n in range(total):
            if n == give_up:
                break
            while not full[at].done(phase):
                yield
            for r in range(ranks):
                def free(r=r, at=at):
                    empty[r][at] += 1
                late.append(free)
            at += 1
            if at == stages:
                at, phase = 0, phase ^ 1
            yield
        if give_up < total:
            order = list(range(ranks))
            rng.shuffle(order)
            for r in order:
                abort[r] = True
                for _ in range(rng.randrange(0, 8)):
                    yield

    actors = [loader(r) for r in range(ranks)] + [consumer()]
    speed = [rng.choice([1, 1, 4, 20]) for _ in actors] + [rng.choice([1, 3, 12]), rng.choice([1, 3, 12])]
    alive = [True] * len(actors)
    for _ in range(200000):
        if not any(alive):
            break
        pick = rng.choices(range(len(speed)), weights=speed)[0]
        if pick < len(actors):
            if alive[pick]:
                try:
                    next(actors[pick])
                except StopIteration:
                    alive[pick] = False
        elif pick == len(actors):
            if flying:
                flying.pop(rng.randrange(len(flying))).land()
        elif late:
            late.pop(0)()
    assert not any(alive), "a loader never ends"
    if flying:
        raise InFlight(f"{len(flying)} copies")


@pytest.mark.parametrize("ranks", [1, 2])
@pytest.mark.parametrize("stages,total", [(5, 3), (5, 40), (6, 17), (8, 1), (4, 9)])
def test_nothing_is_in_flight_at_the_end(ranks, stages, total):
    for seed in range(300):
        simulate(seed, ranks, stages, total)


@pytest.mark.parametrize("ranks,broken", [(1, dict(always=False)), (2, dict(always=False)), (2, dict(tell=False)), (2, dict(always=False, tell=False))], ids=str)
def test_broken_ends_are_caught(ranks, broken):
    with pytest.raises(InFlight):
        for seed in range(2000):
            simulate(seed, ranks, 5, 12, **broken)
